"""Rotary positions and the 4-bit cache in 64 bits on the CPU, written from the
header's text: rotation, storing, the page layout, attention."""
import math

import torch

F64 = torch.float64


def rotate(x, pos, spec, backward=False):
    """x [tokens][H][D] float64, pos [tokens]: the rotation of a binding.Rope."""
    s = spec.spec
    n = s.rotary_dim // 2
    a = pos.to(F64)[:, None] * torch.tensor(list(s.freq)[:n], dtype=F64)
    cos, sin = torch.cos(a)[:, None] * s.amplitude, torch.sin(a)[:, None] * s.amplitude * (-1 if backward else 1)
    i = torch.arange(n)
    u, v = (i, i + n) if s.layout == 0 else (2 * i, 2 * i + 1)
    y = x.clone()
    y[..., u] = x[..., u] * cos - x[..., v] * sin
    y[..., v] = x[..., v] * cos + x[..., u] * sin
    return y


def bf16_down(x):
    y = x.to(torch.bfloat16)
    lower = torch.nextafter(y, torch.full_like(y, -math.inf))
    return torch.where(y.to(F64) > x, lower, y)


def quantise(x):
    """x [..., D] float64 -> codes [..., D] int64, scale and minimum [..., D / 32] bfloat16."""
    g = x.unflatten(-1, (-1, 32))
    low = bf16_down(g.amin(-1))
    scale = -bf16_down(-(g.amax(-1) - low.to(F64)) / 15)
    s = scale.to(F64)[..., None]
    c = torch.where(s > 0, (g - low.to(F64)[..., None]) / torch.where(s > 0, s, 1.0), 0.0)
    return c.round().clamp(0, 15).flatten(-2).long(), scale, low


def value(codes, scale, low):
    g = codes.to(F64).unflatten(-1, (-1, 32))
    return (low.to(F64)[..., None] + g * scale.to(F64)[..., None]).to(torch.bfloat16).to(F64).flatten(-2)


def addresses(D):
    """Byte offsets in a block: (key codes, key scales, value codes, value scales) of token t and channel c; a key's
    minimum is 2 bytes after its scale, a value's 4."""
    t, c = torch.arange(16)[:, None], torch.arange(D)[None, :]
    g, w = c // 32, D // 8
    kc = t * (D // 2) + c // 2
    ks = 8 * D + (t * (D // 32) + g) * 4
    vc = 10 * D + (((t // 8 * 8 + c // w) * 4 + t % 8 // 2) * 2 + t % 2) * (w // 2) + c % w // 2
    vs = 18 * D + ((t // 8 * (D // 32) + g) * 4 + t % 8 // 2) * 8 + t % 2 * 2
    return kc, ks, vc, vs


class Pool:
    """The pages on the CPU, read and written one token at a time."""

    def __init__(self, n_pages, H_kv, D, P, seed=0):
        self.H, self.D, self.P = H_kv, D, P
        g = torch.Generator().manual_seed(seed)
        self.raw = torch.randint(0, 256, (n_pages, H_kv, P // 16, 20 * D), generator=g, dtype=torch.uint8)

    def bytes(self):
        return self.raw.reshape(self.raw.shape[0], -1)

    def _word(self, blk, at):
        lo, hi = blk[at].to(torch.int32), blk[at + 1].to(torch.int32)
        return (((hi << 8) | lo) << 16).view(torch.float32).to(torch.bfloat16)

    def read(self, page, row, h):
        """(key, value) [D] float64."""
        blk, (kc, ks, vc, vs), t = self.raw[page, h, row // 16], addresses(self.D), row % 16
        sh = 4 * (torch.arange(self.D) % 2)
        out = []
        for code, sc, low in ((kc[t], ks[t], ks[t] + 2), (vc[t], vs[t], vs[t] + 4)):
            c = (blk[code].long() >> sh) & 15
            out.append((self._word(blk, low).to(F64) + c.to(F64) * self._word(blk, sc).to(F64)).to(torch.bfloat16).to(F64))
        return out

    def write(self, page, row, h, k, v):
        blk, (kc, ks, vc, vs), t = self.raw[page, h, row // 16], addresses(self.D), row % 16
        for x, code, sc, dl in ((k, kc[t], ks[t], 2), (v, vc[t], vs[t], 4)):
            c, s, m = quantise(x)
            blk[code[0::2]] = (c[0::2] | (c[1::2] << 4)).to(torch.uint8)
            for g in range(self.D // 32):
                at = int(sc[32 * g])
                for a, w in ((at, s[g]), (at + dl, m[g])):
                    b = int(w.view(torch.int16)) & 0xffff
                    blk[a], blk[a + 1] = b & 255, b >> 8

    def history(self, table, n):
        """keys, values [n][H_kv][D] of the first n slots."""
        k = torch.zeros(n, self.H, self.D, dtype=F64)
        v = torch.zeros_like(k)
        for i in range(n):
            for h in range(self.H):
                k[i, h], v[i, h] = self.read(int(table[i // self.P]), i % self.P, h)
        return k, v

    def fill(self, table, n, seed, spread=1.0):
        """Normal keys (with channel offsets) and values in the first n slots, all at once."""
        g = torch.Generator().manual_seed(seed)
        kc, ks, vc, vs = addresses(self.D)
        pages = torch.as_tensor(table)[: -(-n // self.P)].long()
        shape = (len(pages), self.H, self.P // 16, 16, self.D)
        x = [torch.randn(shape, generator=g, dtype=F64) * spread + torch.randn(self.D, generator=g, dtype=F64),
             torch.randn(shape, generator=g, dtype=F64)]
        part = self.raw[pages]
        for y, code, sc, dl in ((x[0], kc, ks, 2), (x[1], vc, vs, 4)):
            c, s, m = quantise(y)
            part[..., code[:, 0::2].flatten()] = (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8).flatten(-2)
            for at, w in ((sc, s), (sc + dl, m)):
                b = w.contiguous().view(torch.int16).to(torch.int32) & 0xffff
                idx = at[:, ::32].flatten()
                part[..., idx], part[..., idx + 1] = (b & 255).to(torch.uint8).flatten(-2), (b >> 8).to(torch.uint8).flatten(-2)
        self.raw[pages] = part
        # after the last token: bytes that read as NaN and infinities
        for i in range(n, len(pages) * self.P):
            self.raw[int(pages[i // self.P]), :, i % self.P // 16, ks[i % 16, ::32] + 1] = 127
            self.raw[int(pages[i // self.P]), :, i % self.P // 16, ks[i % 16, ::32]] = 192
            for d in (0, 4):
                self.raw[int(pages[i // self.P]), :, i % self.P // 16, vs[i % 16, ::32] + d + 1] = 255
                self.raw[int(pages[i // self.P]), :, i % self.P // 16, vs[i % 16, ::32] + d] = 255

    def all(self, table, n):
        """history() without loops."""
        kc, ks, vc, vs = addresses(self.D)
        part = self.raw[torch.as_tensor(table)[: -(-n // self.P)].long()] if n else self.raw[:0]
        sh = 4 * (torch.arange(self.D) % 2)
        out = []
        for code, sc, dl in ((kc, ks, 2), (vc, vs, 4)):
            c = (part[..., code.flatten()].unflatten(-1, code.shape).long() >> sh) & 15
            w = [((part[..., a.flatten()].to(torch.int32) | (part[..., a.flatten() + 1].to(torch.int32) << 8)) << 16)
                 .view(torch.float32).to(F64).unflatten(-1, code.shape) for a in (sc, sc + dl)]
            x = (w[1] + c.to(F64) * w[0]).to(torch.bfloat16).to(F64)      # [pages][H][blocks][16][D]
            out.append(x.flatten(2, 3).transpose(1, 2).flatten(0, 1)[:n])
        return out


def attend(q, k, v, q_len, scale=None):
    """q [N][H][D], k, v [kv][H_kv][D] float64 -> of the first q_len rows: out [n][H][D], lse [n][H], the weighted
    magnitudes sum_j p_j |v_j| [n][H][D], and the largest sum_d |q_d k_d| scale of a visible key [n][H]."""
    N, H, D = q.shape
    kv, H_kv = k.shape[:2]
    out, lse = torch.zeros(q_len, H, D, dtype=F64), torch.full((q_len, H), -math.inf, dtype=F64)
    mag, big = torch.zeros_like(out), torch.zeros(q_len, H, dtype=F64)
    f = scale or D ** -0.5
    for n in range(q_len):
        m = kv - q_len + n + 1
        if m <= 0:
            continue
        for h in range(H):
            kk, vv = k[:m, h // (H // H_kv)], v[:m, h // (H // H_kv)]
            x = kk @ q[n, h] * f
            p = torch.softmax(x, 0)
            lse[n, h], out[n, h], mag[n, h] = torch.logsumexp(x, 0), p @ vv, p @ vv.abs()
            big[n, h] = (kk.abs() @ q[n, h].abs()).max() * f
    return out, lse, mag, big


def attend_bounds(dtype, kv, D, out, lse, mag, big):
    """How far out and lse may be off.  A logit is a float32 sum of D exact products, in any order, then scaled and
    subtracted: off by at most (D + 8) 2^-23 of sum |q_d k_d| (a truncating adder loses 2^-23 a step).  A probability
    is off by twice that, by 2^-20 for the exponential and 2^-8 for its rounding to bfloat16 (float32: 2^-20 too); the sums over kv
    keys lose 2^-23 a step of 8 keys or 64 partial sums; the output's own rounding is half a step."""
    e = (D + 8) * 2.0 ** -23 * big
    steps = (kv / 8 + 64) * 2.0 ** -23
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    p = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -20
    return ((2 * e + 2.0 ** -20 + p + 2 * steps)[..., None] * mag + half * out.abs() + 1e-30,
            2 * e + 2.0 ** -20 + steps + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0))
