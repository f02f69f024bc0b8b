"""Cases of the rotary-position and 4-bit-cache operators, with their plain forms.

A cache page holds, for each KV head, page_size / 16 blocks of 16 tokens.  A
block is 20 D bytes: the key codes (16 rows of D / 2 bytes, channel 2 j in the
low nibble of byte j), the keys' (scale, minimum) bfloat16 pairs per token and
group of 32 channels, the value codes and the values' pairs.  Values are laid
out as [half 2][slice 8][pair 4][odd 2][D / 16 bytes] (token = 8 half + 2 pair
+ odd, a slice is D / 8 channels), their pairs as [half 2][group][pair 4][scale,
minimum][odd 2].  A stored number is bfloat16(minimum + code * scale).
"""
import math

import torch

own = False

F = torch.float32
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases ----------------------------------------------------------------

def listed():
    full = dict(base=500000.0, layout="half", factor=1.0, original=0, amplitude=1.0)
    return [
        # one decode step's query rotation: latency only
        dict(name="rope_decode", op="rope", dtype="bf16", b=64, n=1, heads=32, d=128, rot=128, reach=131072,
             backward=False, **full),
        # training on long sequences: the gradient of interleaved, partly rotated, rescaled positions
        dict(name="rope_backward", op="rope", dtype="bf16", b=4, n=2047, heads=32, d=128, rot=64, reach=1048576,
             backward=True, base=10000.0, layout="interleaved", factor=8.0, original=8192, amplitude=1.0),
        # a decode step of 64 sequences: rotate the queries, store one key and value each
        dict(name="append_decode", op="append", dtype="bf16", b=64, n=1, heads=32, kv=8, d=128, page=16, lo=1, hi=8192,
             rot=128, **full),
        # prompts of unequal length enter the cache (the padded rows are not stored)
        dict(name="append_prompts", op="append", dtype="bf16", b=3, n=1999, heads=32, kv=8, d=128, page=64, lo=1000,
             hi=4096, rot=128, base=10000.0, layout="half", factor=16.0, original=4096, amplitude=1.2772588722239782),
        # the history of a few sequences, read back for the knowledge-graph attention
        dict(name="read_history", op="read", dtype="bf16", b=4, kv=8, d=128, page=64, lo=9000, hi=16384),
        # short histories with one KV head
        dict(name="read_short", op="read", dtype="bf16", b=16, kv=1, d=64, page=16, lo=3, hi=513),
        # a single sequence's decode step: latency
        dict(name="attend_one", op="attend", dtype="bf16", b=1, n=1, heads=32, kv=8, d=128, page=16, lo=513, hi=513),
        # serving: 64 sequences of unequal length
        dict(name="attend_batch", op="attend", dtype="bf16", b=64, n=1, heads=32, kv=8, d=128, page=64, lo=700,
             hi=8192),
        # two very long sequences, every head on one KV head
        dict(name="attend_long_mqa", op="attend", dtype="bf16", b=2, n=1, heads=32, kv=1, d=128, page=128, lo=131109,
             hi=262144),
        # float32 queries, a few drafted tokens to verify
        dict(name="attend_draft_f32", op="attend", dtype="f32", b=8, n=5, heads=16, kv=4, d=64, page=32, lo=5,
             hi=2051),
        # the benchmark's 64-token queries over sequences of about 1024
        dict(name="attend_queries", op="attend", dtype="bf16", b=16, n=64, heads=32, kv=8, d=128, page=16, lo=960,
             hi=1088),
        # a long prompt's last chunks: bound by the tensor cores
        dict(name="attend_prompt", op="attend", dtype="bf16", b=2, n=2048, heads=32, kv=8, d=128, page=64, lo=6001,
             hi=8192),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "attend", "attend", "attend"])
    d = rng.choice([64, 128, 128])
    kv, heads = rng.choice([(8, 32), (1, 32), (4, 16), (2, 6), (8, 8), (1, 1)])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    page = rng.choice([16, 32, 64, 128])
    scaled = rng.choice([True, False])
    rope = dict(base=rng.choice([10000.0, 500000.0]), layout=rng.choice(["half", "interleaved"]),
                rot=16 * rng.randint(1, d // 16), factor=rng.choice([2.0, 8.0, 32.0]) if scaled else 1.0,
                original=rng.choice([0, 4096, 8192]) if scaled else 0, amplitude=rng.choice([1.0, 1.2]))
    if op == "rope":
        b = _log(rng, 1, 256)
        most = (8000 if dtype == "bf16" else 4000) // b
        return dict(op=op, dtype=dtype, b=b, n=_log(rng, 1, most), heads=heads, d=d,
                    reach=_log(rng, 1000, 2000000), backward=rng.choice([True, False]), **rope)
    if op == "append":
        b = _log(rng, 1, 256)
        n = _log(rng, 1, (5000 if dtype == "bf16" else 2500) // b)
        hi = _log(rng, max(2, n), 8192)
        return dict(op=op, dtype=dtype, b=b, n=n, heads=heads, kv=kv, d=d, page=page, lo=max(1, hi // 3), hi=hi, **rope)
    if op == "read":
        b = _log(rng, 1, 64)
        hi = _log(rng, 1, 60000 // b)
        return dict(op=op, dtype="bf16", b=b, kv=kv, d=d, page=page, lo=max(1, hi // 2), hi=hi)
    b = _log(rng, 1, 256)
    hi = _log(rng, 1, 262144 // b // (8 if kv == 8 else 1))
    n = _log(rng, 1, max(1, min(2048, hi, 800000000 // (b * hi * heads))))
    return dict(op=op, dtype=dtype, b=b, n=n, heads=heads, kv=kv, d=d, page=page, lo=max(1, hi // 3), hi=hi)


def _lens(c):
    """The sequences' lengths (spread between lo and hi) and their new tokens, on the host."""
    kv = [c["lo"] + int((c["hi"] - c["lo"]) * ((0.61803398875 * i + 0.999) % 1.0) + 0.5) for i in range(c["b"])]
    if c["op"] == "read":
        return kv, kv
    n = c["n"]
    # every third sequence brings fewer new tokens than the padded batch has rows
    new = [min(k, n - (n // 3 if i % 3 == 1 else 0)) for i, k in enumerate(kv)]
    return kv, new


def work(c):
    d, e = c["d"], 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "rope":
        x = c["b"] * c["n"] * c["heads"] * d
        return {"bytes": 2 * x * e + 4 * c["b"] * c["n"], "flops": 3 * c["b"] * c["n"] * c["heads"] * c["rot"]}
    kv, new = _lens(c)
    row = 20 * d // 16 * c["kv"]   # stored bytes of a token: keys and values with their scales
    if c["op"] == "read":
        return {"bytes": sum(kv) * (row + 2 * c["kv"] * d * e), "flops": sum(kv) * 4 * c["kv"] * d}
    if c["op"] == "append":   # queries in and out, keys and values in, codes out and in again, values out
        t = sum(new)
        return {"bytes": t * (2 * c["heads"] * d * e + 2 * c["kv"] * d * e + 2 * row + 2 * c["kv"] * d * 2),
                "flops": t * (3 * (c["heads"] + c["kv"]) * c["rot"] + 12 * c["kv"] * d)}
    seen = sum(m * k - m * (m - 1) // 2 for k, m in zip(kv, new))
    return {"bytes": sum(kv) * row + sum(new) * c["heads"] * (2 * d * e + 4), "flops": 4 * d * c["heads"] * seen}


# ---- the plain forms ------------------------------------------------------------

def _freqs(c, device):
    """Radians per position: base^(-2 i / rot), divided by `factor` for the frequencies that turn less than once
    in `original` positions (all of them without it), kept for those that turn more than 32 times, a ramp between."""
    f = c["base"] ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=device) / c["rot"])
    keep = ((c["original"] * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0) if c["original"] else torch.zeros_like(f)
    return keep * f + (1.0 - keep) * f / c["factor"]


def _rotate(x, pos, c, back=False):
    """x [..., heads, d] in 32 bits, pos [...]: pairs of channels turned by pos * frequency."""
    a = pos.double()[..., None, None] * _freqs(c, x.device)
    cos, sin = (torch.cos(a) * c["amplitude"]).to(F), (torch.sin(a) * c["amplitude"]).to(F)
    sin = -sin if back else sin
    r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["layout"] == "half":
        u, v = r[..., :c["rot"] // 2], r[..., c["rot"] // 2:]
        return torch.cat([u * cos - v * sin, v * cos + u * sin, rest], -1)
    u, v = r[..., 0::2], r[..., 1::2]
    return torch.cat([torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2), rest], -1)


def _views(pages, c):
    """The codes and (scale, minimum) pairs of pages [n, kv, blocks, 20 d], as views: token dimensions, then the row."""
    d = c["d"]
    half = pages.view(torch.bfloat16)
    kc = pages[..., :8 * d].unflatten(-1, (16, d // 2))
    ks = half[..., 4 * d:5 * d].unflatten(-1, (16, d // 32, 2))
    vc = pages[..., 10 * d:18 * d].unflatten(-1, (2, 8, 4, 2, d // 16)).permute(0, 1, 2, 3, 5, 6, 4, 7)
    vs = half[..., 9 * d:].unflatten(-1, (2, d // 32, 4, 2, 2)).permute(0, 1, 2, 3, 5, 7, 4, 6)
    return kc, ks, vc, vs


def _bf16_toward(x, up):
    """x in 64 bits rounded to bfloat16 toward +infinity (up) or -infinity."""
    near = (x.to(F).view(torch.int32) & -65536).view(F)   # toward zero, or the next where 32 bits reached it
    past = (x > near.double()) if up else (x < near.double())
    away = (near.view(torch.int32) + 65536).view(F)
    return torch.where(past, away, near).to(torch.bfloat16)


def _quantise(x):
    """x [..., d] in 32 bits -> packed codes [..., d / 2] and (scale, minimum) pairs [..., d / 32, 2].  The quotients
    are taken in 64 bits: keys and values in bfloat16 often lie on the border of two codes."""
    g = x.unflatten(-1, (-1, 32)).double()
    low = _bf16_toward(g.amin(-1), False)
    step = _bf16_toward((g.amax(-1) - low.double()) / torch.full((), 15.0, dtype=torch.float64, device=x.device), True)
    wide = torch.where(step > 0, step.double(), 1.0)[..., None]
    code = torch.round((g - low.double()[..., None]) / wide).clamp(0, 15).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.stack([step, low], -1)


def _value(codes, pairs):
    """Packed codes and pairs -> the stored numbers, in 32 bits."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(F).unflatten(-1, (-1, 32))
    p = pairs.to(F)
    return (n * p[..., 0:1] + p[..., 1:2]).flatten(-2).to(torch.bfloat16).to(F)


def _slots(s):
    """[b, n]: the cache slot of each query token, and whether the token is there."""
    c, dev = s["case"], s["kv_len"].device
    n = torch.arange(s["rows"], device=dev)
    slot = (s["kv_len"] - s["q_len"])[:, None] + n
    return slot, (n < s["q_len"][:, None]) & (slot >= 0)


def _history(s):
    """The pages of every sequence, gathered: keys and values [b, slots, kv, d] in 32 bits."""
    c = s["case"]
    blocks = s["pages"].view(-1, c["kv"], c["page"] // 16, 20 * c["d"])[s["table"].long().flatten()]
    kc, ks, vc, vs = _views(blocks, c)
    k = _value(kc, ks).flatten(2, 3)
    v = _value(vc.flatten(3, 5).flatten(-2), vs.flatten(3, 5)).flatten(2, 3)
    return tuple(x.unflatten(0, (c["b"], -1)).transpose(2, 3).flatten(1, 2) for x in (k, v))


def _plain_rope(s):
    y = _rotate(s["x"].to(F), s["pos"], s["case"], s["case"]["backward"])
    return y.to(s["x"].dtype)


def _places(s):
    """The new tokens' (sequence, row), slot, and place in the views: of a key row, of a value row."""
    c = s["case"]
    slot, there = _slots(s)
    bi, ni = torch.nonzero(there, as_tuple=True)
    at = slot[bi, ni]
    page = s["table"][bi, at // c["page"]].long()
    sub, tok = at % c["page"] // 16, at % 16
    return bi, ni, at, (page, slice(None), sub, tok), (page, slice(None), sub, tok // 8, tok % 8 // 2, tok % 2)


def _plain_append(s):
    c = s["case"]
    slot, there = _slots(s)
    q = torch.where(there[..., None, None], _rotate(s["q"].to(F), slot, c).to(s["q"].dtype), s["q_out"])
    bi, ni, at, key, val = _places(s)
    kc, ks, vc, vs = _views(s["pages"].view(-1, c["kv"], c["page"] // 16, 20 * c["d"]), c)
    kc[key], ks[key] = _quantise(_rotate(s["k"][bi, ni].to(F), at, c))
    codes, vs[val] = _quantise(s["v"][bi, ni].to(F))
    vc[val] = codes.unflatten(-1, (8, -1))
    k, v = _plain_read(s)
    return q, k, v


def _plain_read(s):
    """The stored numbers of each sequence's last q_len slots; the rows behind them stay as they were."""
    c = s["case"]
    bi, ni, _, key, val = _places(s)
    kc, ks, vc, vs = _views(s["pages"].view(-1, c["kv"], c["page"] // 16, 20 * c["d"]), c)
    k, v = s["k_out"].clone(), s["v_out"].clone()
    k[bi, ni] = _value(kc[key], ks[key]).to(k.dtype)
    v[bi, ni] = _value(vc[val].flatten(-2), vs[val]).to(v.dtype)
    return k, v


def _plain_attend(s):
    c = s["case"]
    k, v = _history(s)
    slot, there = _slots(s)
    q = s["q"].to(F).unflatten(2, (c["kv"], -1))                                    # [b, n, kv, g, d]
    key = torch.arange(k.shape[1], device=k.device)
    v = torch.where((key < s["kv_len"][:, None])[..., None, None], v, 0.0)
    logit = torch.einsum("bnhgd,bthd->bhgnt", q, k) / math.sqrt(c["d"])
    logit = logit.masked_fill_((key > slot[..., None])[:, None, None], -math.inf)
    top = logit.amax(-1, keepdim=True)
    p = torch.exp(logit.sub_(torch.where(torch.isinf(top), 0.0, top)))
    total = p.sum(-1)
    out = torch.einsum("bhgnt,bthd->bnhgd", p, v) / total.permute(0, 3, 1, 2)[..., None].clamp_min(1e-30)
    lse = (top[..., 0] + torch.log(total)).permute(0, 3, 1, 2)
    there = there[..., None]
    return (torch.where(there[..., None], out.flatten(2, 3).to(s["q"].dtype), s["out"]),
            torch.where(there, lse.flatten(2, 3), s["lse"]))


# ---- the state and a pass ---------------------------------------------------------

def prepare(case, seed):
    c = dict(case)
    dev, dt = torch.device("cuda"), DT[c["dtype"]]
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    s = {"case": c}
    if c["op"] == "rope":
        s["x"] = normal(c["b"], c["n"], c["heads"], c["d"]).to(dt)
        s["pos"] = torch.randint(0, c["reach"], (c["b"], c["n"]), generator=g, device=dev, dtype=torch.int32)
        s["y"] = torch.empty_like(s["x"])
    else:
        kv, new = _lens(c)
        s["rows"] = c["n"] if "n" in c else max(kv)
        s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=dev)
        s["q_len"] = torch.tensor(new, dtype=torch.int32, device=dev)
        width = -(-max(kv) // c["page"])
        n_pages = c["b"] * width + 3
        s["table"] = torch.randperm(n_pages, generator=g, device=dev)[:c["b"] * width].view(c["b"], width).to(torch.int32)
        # a pool filled from normal keys and values: channels with offsets of their own, as rotated keys have
        s["pages"] = torch.empty((n_pages, c["kv"] * c["page"] // 16 * 20 * c["d"]), dtype=torch.uint8, device=dev)
        tokens, most = c["page"] * c["kv"], 1 << 26
        shift = torch.randn(c["kv"], 1, 1, c["d"], generator=g, device=dev)
        for p0 in range(0, n_pages, max(1, most // (tokens * c["d"]))):
            part = s["pages"][p0:p0 + max(1, most // (tokens * c["d"]))]
            kc, ks, vc, vs = _views(part.view(-1, c["kv"], c["page"] // 16, 20 * c["d"]), c)
            kc[...], ks[...] = _quantise(normal(len(part), c["kv"], c["page"] // 16, 16, c["d"]) + shift)
            codes, pairs = _quantise(normal(len(part), c["kv"], c["page"] // 16, 16, c["d"]))
            vc[...] = codes.unflatten(-1, (8, -1)).unflatten(3, (2, 4, 2))
            vs[...] = pairs.unflatten(3, (2, 4, 2))
    if c["op"] in ("append", "attend"):
        s["q"] = normal(c["b"], c["n"], c["heads"], c["d"]).to(dt)
    if c["op"] == "append":
        s["k"] = (normal(c["b"], c["n"], c["kv"], c["d"])).to(dt)
        s["v"] = normal(c["b"], c["n"], c["kv"], c["d"]).to(dt)
        s["q_out"] = torch.zeros_like(s["q"])
    if c["op"] in ("append", "read"):
        s["k_out"] = torch.zeros((c["b"], s["rows"], c["kv"], c["d"]), dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.zeros_like(s["k_out"])
    if c["op"] == "attend":
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((c["b"], c["n"], c["heads"]), device=dev)
    if own:   # the handles and the workspace that a program keeps
        from hierarchical_kv_pruning_b200 import binding
        if c["op"] in ("rope", "append"):
            s["rope"] = binding.Rope(c["rot"], base=c["base"], interleaved=c["layout"] == "interleaved",
                                     factor=c["factor"], original_len=c["original"], amplitude=c["amplitude"])
        if c["op"] != "rope":
            s["cache"] = binding.KvCache(s["pages"], c["kv"], c["d"], c["page"])
        if c["op"] == "attend":
            s["workspace"] = torch.empty(s["cache"].workspace_size(dt, c["b"], c["n"], c["heads"]), dtype=torch.uint8,
                                         device=dev)
    return s


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "read": _plain_read, "attend": _plain_attend}[op](s)
    from hierarchical_kv_pruning_b200 import binding
    if op == "rope":
        return binding.rope(s["x"], s["pos"], s["rope"], out=s["y"], backward=s["case"]["backward"])
    cache, seqs = s["cache"], (s["table"], s["kv_len"], s["q_len"])
    if op == "append":
        cache.append(s["k"], s["v"], *seqs, rope=s["rope"], q=s["q"], q_out=s["q_out"])
        k, v = cache.read(s["rows"], *seqs, k_out=s["k_out"], v_out=s["v_out"])
        return s["q_out"], k, v
    if op == "read":
        return cache.read(s["rows"], *seqs, k_out=s["k_out"], v_out=s["v_out"])
    return cache.attend(s["q"], *seqs, out=s["out"], lse=s["lse"], workspace=s["workspace"])


# ---- the definition in 64 bits ------------------------------------------------------

def _turned(x, pos, c, back=False):
    """x [heads, d] rows of one token each, in 64 bits: complex multiplication by amplitude * exp(+-i pos f)."""
    i = torch.arange(c["rot"] // 2, device=x.device, dtype=torch.float64)
    f = torch.exp(-2.0 * i / c["rot"] * math.log(c["base"]))
    turns = c["original"] * f / (2 * math.pi)
    keep = torch.where(turns < 1, 0.0, torch.where(turns > 32, 1.0, (turns - 1) / 31)) if c["original"] else 0.0 * f
    f = f * (keep + (1 - keep) / c["factor"])
    z = torch.polar(torch.full_like(f, c["amplitude"]).expand(pos.shape[0], -1).contiguous(),
                    pos.double()[:, None] * f * (-1 if back else 1))[:, None]
    i = i.long()
    first, second = (i, i + c["rot"] // 2) if c["layout"] == "half" else (2 * i, 2 * i + 1)
    w = torch.complex(x[..., first], x[..., second]) * z
    y = x.clone()
    y[..., first], y[..., second] = w.real, w.imag
    return y


def _stored(x):
    """What a cache holds of rows x [..., d] in 64 bits, from the definition."""
    def rounded(t, up):
        n = t.to(torch.bfloat16).double()
        step = torch.where(n == 0, 2.0 ** -133, torch.exp2(torch.floor(torch.log2(n.abs().clamp_min(2.0 ** -126))) - 7))
        if up:
            return torch.where(n < t, (n + step).to(torch.bfloat16).double(), n)
        return torch.where(n > t, (n - step).to(torch.bfloat16).double(), n)
    g = x.reshape(*x.shape[:-1], -1, 32)
    low = rounded(g.min(-1, keepdim=True).values, False)
    step = rounded((g.max(-1, keepdim=True).values - low) / 15, True)
    code = ((g - low) / step.clamp_min(1e-300)).round().clamp(0, 15)
    return (low + code * step).to(torch.bfloat16).double().reshape(x.shape)


def _read_slots(s, b, slots):
    """Keys and values [slots, kv, d] of sequence b in 64 bits, byte by byte from the layout."""
    c, d = s["case"], s["case"]["d"]
    dev = slots.device
    page, tok = s["table"][b].long()[slots // c["page"]], slots % c["page"]
    base = ((page[:, None] * c["kv"] + torch.arange(c["kv"], device=dev)) * (c["page"] // 16) + (tok // 16)[:, None]) * 20 * d
    raw, ch, t = s["pages"].view(-1), torch.arange(d, device=dev), (tok % 16)[:, None, None]

    def pair(byte):   # the bfloat16 number at a byte address
        bits = (raw[byte].to(torch.int32) | (raw[byte + 1].to(torch.int32) << 8)) << 16
        return bits.view(torch.float32).double()

    def number(code_byte, scale_byte, low_byte):
        code = (raw[code_byte] >> (4 * (ch % 2)).to(torch.uint8)) & 15
        return (code.double() * pair(scale_byte) + pair(low_byte)).to(torch.bfloat16).double()

    at = base[:, :, None]
    k = number(at + t * (d // 2) + ch // 2, at + 8 * d + (t * (d // 32) + ch // 32) * 4, at + 8 * d + (t * (d // 32) + ch // 32) * 4 + 2)
    w = d // 8
    vc = (((t // 8 * 8 + ch // w) * 4 + t % 8 // 2) * 2 + t % 2) * (w // 2) + ch % w // 2
    vs = ((t // 8 * (d // 32) + ch // 32) * 4 + t % 8 // 2) * 8 + t % 2 * 2
    v = number(at + 10 * d + vc, at + 18 * d + vs, at + 18 * d + vs + 4)
    return k, v


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        x = s["x"].double().flatten(0, 1)
        return _turned(x, s["pos"].flatten(), c, c["backward"]).view(s["x"].shape)
    kv, new = _lens(c)
    dev = s["pages"].device
    if c["op"] == "append":
        q, k, v = (torch.zeros(s[n].shape, dtype=torch.float64, device=dev) for n in ("q_out", "k_out", "v_out"))
        for b in range(c["b"]):
            at = torch.arange(kv[b] - new[b], kv[b], device=dev)
            q[b, :new[b]] = _turned(s["q"][b, :new[b]].double(), at, c)
            k[b, :new[b]] = _stored(_turned(s["k"][b, :new[b]].double(), at, c))
            v[b, :new[b]] = _stored(s["v"][b, :new[b]].double())
        return q, k, v
    if c["op"] == "read":
        k, v = (torch.zeros(s[n].shape, dtype=torch.float64, device=dev) for n in ("k_out", "v_out"))
        for b in range(c["b"]):
            k[b, :kv[b]], v[b, :kv[b]] = _read_slots(s, b, torch.arange(kv[b], device=dev))
        return k, v
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=dev)
    group = c["heads"] // c["kv"]
    for b in range(c["b"]):
        k, v = _read_slots(s, b, torch.arange(kv[b], device=dev))
        past = torch.arange(kv[b], device=dev)[None, :] > torch.arange(kv[b] - new[b], kv[b], device=dev)[:, None]
        for h in range(c["heads"]):
            x = (s["q"][b, :new[b], h].double() @ k[:, h // group].T) * c["d"] ** -0.5
            x[past] = -math.inf
            lse[b, :new[b], h] = torch.logsumexp(x, 1)
            out[b, :new[b], h] = torch.softmax(x, 1) @ v[:, h // group]
    return out, lse
