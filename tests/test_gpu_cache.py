"""Rotary positions and the 4-bit paged cache on the GPU against the 64-bit
reference: each operator at the sizes and masks where it can go wrong, what it
must leave alone, and a decode loop of all of them."""
import math

import pytest
import torch

from hierarchical_kv_pruning_b200 import binding
from hierarchical_kv_pruning_b200.binding import AtlaskvError, KvCache, Rope
from tests import _cache_ref as ref

pytestmark = pytest.mark.gpu
F64, BF, F32 = torch.float64, torch.bfloat16, torch.float32
HALF_STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def normal(seed, *shape, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype)


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def tables(lens, P, n_pages, seed, width=None):
    """Distinct random pages for each sequence; -1 past its length."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // P) for n in lens]
    ids = torch.randperm(n_pages, generator=g).tolist()
    t = torch.full((len(lens), width or max(1, *need)), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        t[b, :n] = torch.tensor([ids.pop() for _ in range(n)], dtype=torch.int32)
    return t


# ---- rotary positions -----------------------------------------------------------

def check_rotated(y, x, pos, spec, backward=False):
    """cos and sin are off by at most 4e-7 (the angle's rounding to float32 within a half turn, the functions' 2 ulp, the
    amplitude's product), products and their sum by three roundings."""
    want = ref.rotate(x.to(F64), pos, spec, backward)
    other = ref.rotate(x.to(F64).abs(), torch.zeros_like(pos), spec).abs()
    n = spec.spec.rotary_dim
    pair = torch.zeros_like(want)
    i = torch.arange(n // 2)
    u, v = (i, i + n // 2) if spec.spec.layout == 0 else (2 * i, 2 * i + 1)
    pair[..., u] = pair[..., v] = other[..., u] + other[..., v]
    tol = pair * (4e-7 + 3 * 2.0 ** -24) + HALF_STEP[y.dtype] * want.abs()
    assert bool(((y.to(F64) - want).abs() <= tol).all())
    assert torch.equal(y[..., n:], x[..., n:])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,rot,inter,H,B,N", [
    (128, 128, False, 32, 3, 1), (128, 64, True, 5, 1, 7), (64, 64, False, 1, 2, 33), (64, 16, False, 3, 1, 1),
    (128, 48, False, 7, 2, 3), (128, 112, True, 32, 1, 2500), (64, 64, True, 9, 1, 801), (128, 16, True, 1, 1, 1),
])
def test_rope(dtype, D, rot, inter, H, B, N):
    spec = Rope(rot, base=500000.0, interleaved=inter, factor=8.0, original_len=4096, amplitude=1.1)
    x = normal(rot + N, B, N, H, D, dtype=dtype)
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(-1000, 2 ** 31 - 1, (B, N), generator=g, dtype=torch.int64)
    pos[0, 0] = 2 ** 31 - 1
    for backward in (False, True):
        y = binding.rope(x.cuda(), i32(pos), spec, backward=backward).cpu()
        check_rotated(y.flatten(0, 1), x.flatten(0, 1), pos.flatten(), spec, backward)


def test_rope_in_place_strided_and_empty():
    spec, D, H = Rope(64, interleaved=False), 128, 4
    wide = normal(5, 2, 3, H + 5, D, dtype=BF).cuda()       # queries inside a wider projection
    pos = i32([[0, 7, 9], [100000, 1, 5]])
    x = wide[:, :, :H]
    dense = binding.rope(x.contiguous(), pos, spec)
    assert torch.equal(binding.rope(x, pos, spec), dense)
    before = wide.clone()
    assert binding.rope(x, pos, spec, out=x).data_ptr() == x.data_ptr()
    assert torch.equal(wide[:, :, :H], dense) and torch.equal(wide[:, :, H:], before[:, :, H:])
    none = torch.empty(0, 3, H, D, dtype=BF, device="cuda")
    assert binding.rope(none, i32([]).view(0, 3), spec).shape == none.shape


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradient(inter):
    """The backward direction is the transpose of the forward one, and agrees with differences of the forward pass."""
    spec = Rope(48, interleaved=inter, amplitude=1.3)
    B, N, H, D = 2, 3, 2, 64
    x, g, d = (normal(s, B, N, H, D).cuda() for s in (1, 2, 3))
    pos = i32([[0, 3, 70000], [12, 9, 1 << 20]])
    dx = binding.rope(g, pos, spec, backward=True)
    loss = lambda t: float((binding.rope(t, pos, spec).double() * g.double()).sum())  # noqa: E731
    h = 2.0 ** -6      # the map is linear: the difference is exact up to float32 rounding of x +- h d
    diff = (loss(x + h * d) - loss(x - h * d)) / (2 * h)
    scale = float((g.double().abs().sum() * 4) * 1.3)
    assert abs(diff - float((dx.double() * d.double()).sum())) <= scale * 2.0 ** -24 * 8 / h


def test_rope_refusals():
    spec, x, pos = Rope(64), normal(1, 2, 3, 4, 64, dtype=BF).cuda(), i32([[0, 1, 2], [3, 4, 5]])
    for bad in (lambda: binding.rope(x[:, :, :, :32], pos, spec), lambda: binding.rope(x.half(), pos, spec),
                lambda: binding.rope(x, pos.long(), spec), lambda: binding.rope(x, pos[:1], spec),
                lambda: binding.rope(x.transpose(1, 2), pos, spec), lambda: binding.rope(x, pos.cpu(), spec),
                lambda: binding.rope(x, pos, Rope(128)), lambda: binding.rope(x, pos, spec, out=x[:1]),
                lambda: binding.rope(x[0], pos, spec), lambda: binding.rope(x[..., 1:], pos, spec)):
        with pytest.raises(AtlaskvError):
            bad()


# ---- append and read --------------------------------------------------------------

def new_cache(pool):
    return KvCache(pool.bytes().clone().cuda(), pool.H, pool.D, pool.P)


@pytest.mark.parametrize("dtype,D,H_kv,H,P,N,lens,q_len", [
    (BF, 128, 2, 8, 16, 1, [1, 16, 17, 40], None),
    (BF, 128, 8, 32, 64, 5, [5, 64, 131, 7], [5, 3, 0, 1]),
    (BF, 64, 1, 1, 16, 37, [37, 90], [37, 20]),
    (F32, 128, 3, 3, 32, 4, [4, 33, 70], None),
    (F32, 64, 2, 6, 256, 19, [300, 19, 0], [19, 2, 0]),
    (BF, 128, 1, 0, 128, 300, [300], None),
    (BF, 64, 4, 4, 16, 700, [900, 700], [700, 655]),      # many tokens: several rows a warp
])
def test_append_without_positions_stores_the_formula(dtype, D, H_kv, H, P, N, lens, q_len):
    """Without a rotation the bytes of bfloat16 input are the definition's exactly; float32 input may round a code
    the other way at a border, so its read back numbers are held to half a step (and 2^-8, their rounding)."""
    B, pages = len(lens), sum(-(-n // P) for n in lens) + 3
    pool = ref.Pool(pages, H_kv, D, P, seed=1)
    table = tables(lens, P, pages, 2)
    k, v = normal(3, B, N, H_kv, D, dtype=dtype), normal(4, B, N, H_kv, D, dtype=dtype)
    k[0, 0, 0, :32] = 2.5          # a constant group: scale 0
    v[0, 0, 0, :32] = 0.0
    q = normal(5, B, N, H, D, dtype=dtype) if H else None
    with new_cache(pool) as cache:
        q_out = cache.append(k.cuda(), v.cuda(), table.cuda(), i32(lens), None if q_len is None else i32(q_len),
                             q=None if q is None else q.cuda(), q_out=None if q is None else torch.full_like(q, 9.).cuda())
        cache.sync_status()
        got = cache.pages.cpu()
        ql = q_len or [N] * B
        for b in range(B):
            for n in range(ql[b]):
                at = lens[b] - ql[b] + n
                for h in range(H_kv):
                    pool.write(int(table[b, at // P]), at % P, h, k[b, n, h].to(F64), v[b, n, h].to(F64))
            if q is not None:
                assert torch.equal(q_out[b, :ql[b]].cpu(), q[b, :ql[b]])
                assert bool((q_out[b, ql[b]:] == 9.).all())
        if dtype == BF:
            assert torch.equal(got, pool.bytes())
        else:
            ko, vo = cache.read(N, table.cuda(), i32(lens), i32(ql))
            for x, y in ((ko, k), (vo, v)):
                for b in range(B):
                    w = y[b, :ql[b]].to(F64)
                    _, s, _ = ref.quantise(w)
                    tol = s.to(F64).repeat_interleave(32, -1) * (0.5 + 1e-5) + 2.0 ** -8 * w.abs() * 1.1
                    r = x[b, :ql[b]].cpu().to(F64)
                    assert bool(((r - w).abs() <= tol + 2.0 ** -8 * r.abs()).all())
                    assert bool((x[b, ql[b]:] == 0).all())


@pytest.mark.parametrize("dtype,inter,rot,D", [(BF, False, 128, 128), (BF, True, 64, 128), (F32, False, 32, 64)])
def test_append_rotates_by_slot_or_position(dtype, inter, rot, D):
    H_kv, H, P, N, lens = 2, 4, 32, 6, [50, 6, 33]
    pages = 10
    pool = ref.Pool(pages, H_kv, D, P, seed=1)
    table = tables(lens, P, pages, 3)
    spec = Rope(rot, interleaved=inter, factor=4.0)
    wide = normal(7, 3, N, H + 2 * H_kv, D, dtype=dtype)
    q, k, v = wide[:, :, :H], wide[:, :, H:H + H_kv], wide[:, :, H + H_kv:]
    dev = wide.cuda()
    dq, dk, dv = dev[:, :, :H], dev[:, :, H:H + H_kv], dev[:, :, H + H_kv:]
    slots = torch.tensor([[n - N + i for i in range(N)] for n in lens])
    for pos in (None, slots + 1000003):
        with new_cache(pool) as cache:
            out = cache.append(dk, dv, table.cuda(), i32(lens), rope=spec, q=dq,
                               positions=None if pos is None else i32(pos)).cpu()
            ko, vo = cache.read(N, table.cuda(), i32(lens))
            cache.sync_status()
        at = (slots if pos is None else pos).flatten()
        check_rotated(out.flatten(0, 1), q.flatten(0, 1), at, spec)
        w = ref.rotate(k.flatten(0, 1).to(F64), at, spec)
        _, s, _ = ref.quantise(w)
        tol = s.to(F64).repeat_interleave(32, -1) * (0.5 + 1e-4) + 2.0 ** -7 * w.abs() + 1e-5
        assert bool(((ko.cpu().flatten(0, 1).to(F64) - w).abs() <= tol).all())
        c, s, m = ref.quantise(v.flatten(0, 1).to(F64))
        if dtype == BF:
            assert torch.equal(vo.cpu().flatten(0, 1).to(F64), ref.value(c, s, m))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,inter,rot", [(128, False, 128), (128, True, 128), (128, False, 48), (64, False, 64),
                                         (64, True, 16), (64, False, 0)])
def test_stored_bytes_are_the_definitions(dtype, D, inter, rot):
    """Minimum, scale and codes as in exact arithmetic, whatever float32 makes of the rotation: the bytes are the
    reference's (whose float64 roundings could differ with a chance of 1e-8 a number)."""
    H_kv, P, lens = 2, 64, [700, 333]
    pages = 20
    pool = ref.Pool(pages, H_kv, D, P, seed=1)
    table = tables(lens, P, pages, 3)
    N = max(lens)
    k, v = normal(11, 2, N, H_kv, D, dtype=dtype) * 3, normal(12, 2, N, H_kv, D, dtype=dtype)
    spec = Rope(rot, base=500000.0, interleaved=inter, factor=2.0, amplitude=1.2) if rot else None
    with new_cache(pool) as cache:
        cache.append(k.cuda(), v.cuda(), table.cuda(), i32(lens), i32(lens), rope=spec)
        cache.sync_status()
        for b, n in enumerate(lens):
            w = k[b, :n].to(F64)
            w = ref.rotate(w, torch.arange(n), spec) if rot else w
            for i in range(n):
                for h in range(H_kv):
                    pool.write(int(table[b, i // P]), i % P, h, w[i, h], v[b, i, h].to(F64))
        assert torch.equal(cache.pages.cpu(), pool.bytes())


@pytest.mark.parametrize("D,H_kv,P,lens", [(128, 3, 16, [1, 15, 16, 17, 100, 0]), (64, 1, 256, [300, 256, 5]),
                                           (128, 1, 64, [2000]), (64, 5, 32, [33, 64])])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_read_whole_histories(D, H_kv, P, lens, dtype):
    pages = sum(-(-n // P) for n in lens) + 2
    pool = ref.Pool(pages, H_kv, D, P)
    table = tables(lens, P, pages, 4)
    for b, n in enumerate(lens):
        if n:
            pool.fill(table[b], n, seed=b)
    N = max(lens) + 3
    with new_cache(pool) as cache:
        k, v = cache.read(N, table.cuda(), i32(lens), i32(lens), dtype=dtype)
        cache.sync_status()
        only = torch.full_like(k, 7.)
        binding.atlaskv_cache_read(cache.handle, cache._seqs(len(lens), N, table.cuda(), i32(lens), i32(lens)),
                                   binding._dtype_code(dtype), None, only.data_ptr(),
                                   torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
    for b, n in enumerate(lens):
        wk, wv = pool.all(table[b], n)
        assert torch.equal(k[b, :n].cpu().to(F64), wk) and torch.equal(v[b, :n].cpu().to(F64), wv)
        assert bool((k[b, n:] == 0).all()) and bool((only[b, n:] == 7).all())
        assert torch.equal(only[b, :n], v[b, :n])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_read_into_tensors_on_16_byte_boundaries(dtype):
    D, H_kv, P, lens, N = 128, 2, 32, [40, 7], 9
    pool = ref.Pool(6, H_kv, D, P)
    table = tables(lens, P, 6, 4)
    for b, n in enumerate(lens):
        pool.fill(table[b], n, seed=b)
    size = 2 * N * H_kv * D
    with new_cache(pool) as cache:
        want = cache.read(N, table.cuda(), i32(lens), i32([9, 5]), dtype=dtype)
        step = 16 // dtype.itemsize
        raw = [torch.zeros(size + step, dtype=dtype, device="cuda")[step:].view(2, N, H_kv, D) for _ in range(2)]
        assert raw[0].data_ptr() % 32 == 16
        got = cache.read(N, table.cuda(), i32(lens), i32([9, 5]), k_out=raw[0], v_out=raw[1])
        cache.sync_status()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_stored_extremes():
    """Infinities and NaN are stored as 2^120 and 0 and reported; huge and tiny finite numbers are not."""
    D, P = 128, 16
    pool = ref.Pool(2, 1, D, P)
    table = i32([[1]])
    k = torch.zeros(1, 3, 1, D)
    v = normal(1, 1, 3, 1, D)
    k[0, 0, 0, :32], k[0, 0, 0, 32:64] = 3e38, -3e38
    k[0, 0, 0, 64:96] = 1e-38 * torch.arange(32)
    k[0, 1, 0, 5] = 1e20
    k = k.to(BF).cuda()
    v = v.to(BF).cuda()
    with new_cache(pool) as cache:
        cache.append(k, v, table, i32([3]))
        cache.sync_status()
        out, _ = cache.read(3, table, i32([3]))
        assert bool((out[0, 0, 0, :32] == 2.0 ** 120).all()) and bool((out[0, 0, 0, 32:64] == -2.0 ** 120).all())
        assert float(out[0, 0, 0, 64:96].abs().max()) <= 1e-36
        assert float(out[0, 1, 0, 5]) == pytest.approx(1e20, rel=2.0 ** -6)
        assert bool(torch.isfinite(out).all())
        k[0, 2, 0, 3], k[0, 2, 0, 40], v[0, 0, 0, 70] = math.inf, -math.inf, math.nan
        cache.append(k, v, table, i32([3]))
        with pytest.raises(AtlaskvError) as e:
            cache.sync_status()
        assert e.value.status == binding.ATLASKV_EDEVICE and "finite" in str(e.value)
        out, w = cache.read(3, table, i32([3]))
        assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(w).all())
        assert float(out[0, 2, 0, 3]) == 2.0 ** 120 and float(out[0, 2, 0, 40]) == -2.0 ** 120


# ---- attention over the cache --------------------------------------------------------

def check_attend(dtype, D, H_kv, H, P, N, lens, q_len=None, scale=0.0, spread=1.0, seed=0, strided=False):
    B = len(lens)
    pages = sum(-(-n // P) for n in lens) + 2
    pool = ref.Pool(pages, H_kv, D, P, seed)
    table = tables(lens, P, pages, seed + 1, width=max(1, *[-(-n // P) for n in lens]) + 2)
    for b, n in enumerate(lens):
        if n:
            pool.fill(table[b], n, seed=100 + b, spread=spread)
    q = normal(seed + 2, B, N, H, D, dtype=dtype)
    ql = q_len or [N] * B
    dq = torch.cat([q, q], 2).cuda()[:, :, H:] if strided else q.cuda()
    with new_cache(pool) as cache:
        out = torch.full((B, N, H, D), 5.0, dtype=dtype, device="cuda")
        lse = torch.full((B, N, H), 5.0, device="cuda")
        cache.attend(dq, table.cuda(), i32(lens), None if q_len is None else i32(q_len), scale=scale, out=out, lse=lse)
        cache.sync_status()
    for b in range(B):
        k, v = pool.all(table[b], lens[b])
        o, l, mag, big = ref.attend(q[b].to(F64), k, v, ql[b], scale or None)
        to, tl = ref.attend_bounds(dtype, lens[b], D, o, l, mag, big)
        go, gl = out[b, :ql[b]].cpu().to(F64), lse[b, :ql[b]].cpu().to(F64)
        assert bool(((go - o).abs() <= to).all()), (b, float(((go - o).abs() / to).max()))
        assert torch.equal(torch.isinf(gl), torch.isinf(l))
        ok = torch.isfinite(l)
        assert bool(((gl - l).abs()[ok] <= tl[ok]).all()), (b, float(((gl - l).abs() / tl)[ok].max()))
        assert bool((out[b, ql[b]:] == 5).all()) and bool((lse[b, ql[b]:] == 5).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,H_kv,H,P,N,lens,q_len", [
    (128, 2, 8, 16, 1, [1, 15, 16, 17, 31, 33, 500], None),            # one token; pages that end inside a tile
    (64, 1, 1, 16, 1, [1, 2, 129], None),
    (128, 1, 32, 128, 1, [257, 1000], None),                            # every head on one KV head
    (64, 4, 8, 32, 3, [3, 40, 2, 0, 1], [3, 2, 3, 0, 3]),               # rows that see nothing, empty sequences
    (128, 8, 8, 64, 5, [5, 700], [0, 5]),
    (128, 2, 6, 256, 7, [7, 300], [7, 6]),                              # an odd group
    (64, 2, 10, 16, 2, [65, 64, 63], None),
    (128, 1, 7, 16, 40, [40, 77], [40, 33]),
    (64, 1, 48, 32, 1, [70], None),
    (128, 2, 8, 32, 33, [33, 200, 100], [33, 33, 1]),
    (128, 1, 4, 64, 130, [130, 190], [130, 100]),
    (64, 2, 4, 16, 150, [150, 400], None),
])
def test_attend(dtype, D, H_kv, H, P, N, lens, q_len):
    check_attend(dtype, D, H_kv, H, P, N, lens, q_len, seed=D + N)


@pytest.mark.parametrize("dtype,D,H_kv,H,P,N,lens", [
    (BF, 128, 2, 8, 64, 1, [20000, 3]), (F32, 64, 1, 4, 16, 2, [9001]), (BF, 64, 1, 2, 256, 1, [70001]),
    (BF, 128, 1, 16, 32, 1, [1] * 70 + [4097]), (BF, 128, 4, 8, 16, 1, [(37 * i) % 300 for i in range(300)]),
    (BF, 128, 1, 8, 64, 64, [3000]), (BF, 128, 2, 4, 32, 300, [1300, 301]),
])
def test_attend_long_and_ragged(dtype, D, H_kv, H, P, N, lens):
    check_attend(dtype, D, H_kv, H, P, N, lens, [min(n, N) for n in lens], seed=9)


@pytest.mark.parametrize("dtype,D,B,H_kv,G,N", [
    (BF, 128, 2, 1, 4, 1), (BF, 128, 25, 8, 1, 1), (BF, 64, 50, 8, 2, 1), (BF, 128, 30, 2, 4, 3), (BF, 128, 40, 4, 4, 3),
    (BF, 64, 40, 4, 24, 1), (F32, 128, 50, 2, 3, 1), (F32, 64, 160, 1, 7, 2), (F32, 64, 3, 2, 5, 4),
])
def test_attend_with_few_and_many_items(dtype, D, B, H_kv, G, N):
    """Calls whose items get a large CTA each, share an SM by two, or fill it with small CTAs; one long sequence among them."""
    lens = [N + (53 * i + 7 * D) % 150 for i in range(B)]
    lens[-1] = 1900
    check_attend(dtype, D, H_kv, H_kv * G, 32, N, lens, seed=B)
    check_attend(dtype, D, H_kv, H_kv * G, 16, N, [N + i % 90 for i in range(B)], seed=G)


@pytest.mark.parametrize("spread,scale", [(30.0, 0.0), (1.0, 3.0), (0.01, 1e-3)])
def test_attend_sharp_and_flat(spread, scale):
    """Logits of hundreds (one key takes all), and almost equal ones."""
    check_attend(BF, 128, 2, 8, 32, 2, [300, 65], scale=scale, spread=spread, seed=4)
    check_attend(F32, 64, 1, 4, 16, 2, [300, 65], scale=scale, spread=spread, seed=5)
    check_attend(BF, 128, 1, 4, 32, 100, [300, 165], scale=scale, spread=spread, seed=6)


def test_attend_strided_queries():
    check_attend(BF, 128, 2, 8, 16, 3, [30, 50], strided=True)
    check_attend(F32, 64, 2, 8, 16, 1, [30, 50], strided=True)
    check_attend(BF, 128, 2, 8, 16, 70, [130, 250], strided=True)


def test_attend_is_repeatable_and_replays_with_other_lengths():
    """Two captured calls share one workspace; replays see the lengths of the moment."""
    D, H_kv, H, P, B = 128, 2, 8, 16, 3
    pool = ref.Pool(300, H_kv, D, P)
    table = tables([1500] * B, P, 300, 1)
    for b in range(B):
        pool.fill(table[b], 1500, seed=b)
    q = [normal(s, B, 1, H, D, dtype=BF).cuda() for s in (1, 2)]
    dt, kv = table.cuda(), i32([1500, 700, 1])
    with new_cache(pool) as cache:
        ws = torch.empty(max(256, cache.workspace_size(BF, B, 1, H)), dtype=torch.uint8, device="cuda")
        eager = [cache.attend(x, dt, kv, workspace=ws) for x in q]
        again = [cache.attend(x, dt, kv, workspace=ws) for x in q]
        assert all(torch.equal(a, b) for e, f in zip(eager, again) for a, b in zip(e, f))
        graphs, outs = [], []
        for x in q:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs.append(cache.attend(x, dt, kv, workspace=ws))
            graphs.append(g)
        for lens in ([1500, 700, 1], [3, 1499, 800]):
            kv.copy_(i32(lens))
            ws.fill_(255)
            for _ in range(2):
                for g in graphs:
                    g.replay()
            want = [cache.attend(x, dt, kv) for x in q]
            assert all(torch.equal(a, b) for e, f in zip(outs, want) for a, b in zip(e, f))
        cache.sync_status()


def test_calls_on_another_stream():
    D, H_kv, H, P = 128, 2, 8, 16
    pool = ref.Pool(60, H_kv, D, P)
    table = tables([400, 300], P, 60, 1)
    pool.fill(table[0], 400, 1)
    pool.fill(table[1], 300, 2)
    dt, kv, spec = table.cuda(), i32([400, 300]), Rope(128)
    q, k, v = (normal(s, 2, 1, h, D, dtype=BF).cuda() for s, h in ((1, H), (2, H_kv), (3, H_kv)))
    with new_cache(pool) as a, new_cache(pool) as b:
        r = a.append(k, v, dt, kv, rope=spec, q=q)
        want = a.attend(r, dt, kv) + a.read(1, dt, kv)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        r = b.append(k, v, dt, kv, rope=spec, q=q, stream=side)
        got = b.attend(r, dt, kv, stream=side) + b.read(1, dt, kv, stream=side)
        b.sync_status(side)
        assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_bad_device_data_is_reported():
    """Page ids, lengths and slots out of range are found by the kernels' own checks; other sequences are right."""
    D, H_kv, H, P = 64, 1, 2, 16
    pool = ref.Pool(8, H_kv, D, P)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    pool.fill(table[0], 32, 1)
    pool.fill(table[1], 32, 2)
    q = normal(1, 2, 2, H, D, dtype=BF).cuda()
    k, v = (normal(s, 2, 2, H_kv, D, dtype=BF).cuda() for s in (2, 3))
    good = i32([32, 20])
    with new_cache(pool) as cache:
        want, _ = cache.attend(q, table.cuda(), good)
        cache.sync_status()
    bad_table = torch.tensor([[0, 1], [8, -5]], dtype=torch.int32).cuda()
    for tab, kv, ql in ((bad_table, good, None), (table.cuda(), i32([32, 33]), None), (table.cuda(), i32([32, -1]), None),
                        (table.cuda(), good, i32([2, 3])), (table.cuda(), good, i32([2, -1]))):
        for call in ("append", "read", "attend"):
            with new_cache(pool) as cache:
                if call == "append":
                    cache.append(k[:, :2], v[:, :2], tab, kv, ql)
                elif call == "read":
                    cache.read(2, tab, kv, ql)
                else:
                    out, _ = cache.attend(q, tab, kv, ql)
                    assert torch.equal(out[0], want[0])
                with pytest.raises(AtlaskvError) as e:
                    cache.sync_status()
                assert e.value.status == binding.ATLASKV_EDEVICE
    with new_cache(pool) as cache:       # a token below slot 0
        cache.append(k, v, table.cuda(), i32([32, 1]))
        with pytest.raises(AtlaskvError):
            cache.sync_status()


def test_cache_refusals():
    D, H_kv, H, P = 64, 2, 4, 16
    pool = ref.Pool(4, H_kv, D, P)
    table, kv = i32([[0, 1], [2, 3]]), i32([20, 5])
    q = normal(1, 2, 3, H, D, dtype=BF).cuda()
    k = normal(2, 2, 3, H_kv, D, dtype=BF).cuda()
    with new_cache(pool) as c:
        for bad in (
                lambda: c.append(k, k.float(), table, kv), lambda: c.append(k, k, table[:1], kv),
                lambda: c.append(k, k, table, kv.long()), lambda: c.append(k, k, table, kv[:1]),
                lambda: c.append(k[:, :, :1], k[:, :, :1], table, kv), lambda: c.append(k.half(), k.half(), table, kv),
                lambda: c.append(k, k, table, kv, q=q.float()), lambda: c.append(k, k, table, kv, rope=Rope(128)),
                lambda: c.append(k, k, table, kv, positions=kv), lambda: c.append(k, k, table.t(), kv),
                lambda: c.append(k, k, table, kv, q=q[:, :, ::2], q_out=q[:, :, ::2]),
                lambda: c.attend(q[:, :, :3], table, kv), lambda: c.attend(q, table[:1], kv),
                lambda: c.attend(q, table, kv, scale=-1.0), lambda: c.attend(q, table, kv, scale=math.inf),
                lambda: c.attend(q.half(), table, kv), lambda: c.attend(q, table, kv, out=q.float()),
                lambda: c.attend(q, table, kv.cpu()), lambda: c.attend(q, table, kv, q_len=i32([1])),
                lambda: c.read(0, table, kv), lambda: c.read(3, table, kv, dtype=torch.float16),
                lambda: KvCache(c.pages[:, 1:], H_kv, D, P), lambda: KvCache(c.pages, H_kv, D, 2 * P),
                lambda: KvCache(c.pages.cpu(), H_kv, D, P), lambda: c.workspace_size(BF, 2, 3, 5)):
            with pytest.raises(AtlaskvError):
                bad()
        need = c.workspace_size(BF, 2, 3, H)
        if need > 0:
            with pytest.raises(AtlaskvError):
                c.attend(q, table, kv, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
        none = c.attend(q[:0], table[:0], kv[:0])
        assert none[0].shape == (0, 3, H, D)
        assert c.append(k[:0], k[:0], table[:0], kv[:0], q=q[:0]).shape == (0, 3, H, D)
        assert c.read(2, table[:0], kv[:0])[0].shape == (0, 2, H_kv, D)
        c.sync_status()


# ---- together -------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompt_then_decode(dtype):
    """Two sequences: a padded prompt is appended and attended, then tokens one by one; every output against the
    reference on the numbers that the cache holds, which stay within half a step of the rotated keys and of the values."""
    D, H_kv, H, P, N, steps = 64, 2, 6, 16, 21, 14
    spec = Rope(64, base=500000.0)
    prompt, table = [21, 13], i32([[5, 0, 7], [1, 6, 2]])
    pool = ref.Pool(8, H_kv, D, P)
    seen = [[], []]
    with new_cache(pool) as cache:
        kv = i32(prompt)
        for step in range(steps):
            n = N if step == 0 else 1
            ql = prompt if step == 0 else [1, 1]
            q, k, v = (normal(50 + 3 * step + i, 2, n, h, D, dtype=dtype) for i, h in enumerate((H, H_kv, H_kv)))
            if step:
                kv += 1
            r = cache.append(k.cuda(), v.cuda(), table, kv, i32(ql), rope=spec, q=q.cuda())
            out, lse = cache.attend(r, table, kv, i32(ql))
            lens = kv.tolist()
            T = max(lens)
            hk, hv = cache.read(T, table, kv, kv)
            for b in range(2):
                at = torch.arange(lens[b] - ql[b], lens[b])
                want = ref.rotate(k[b, :ql[b]].to(F64), at, spec)
                seen[b].append((want, v[b, :ql[b]].to(F64)))
                wk, wv = (torch.cat([s[i] for s in seen[b]]) for i in (0, 1))
                gk, gv = hk[b, :lens[b]].cpu().to(F64), hv[b, :lens[b]].cpu().to(F64)
                for w, g in ((wk, gk), (wv, gv)):
                    _, s, _ = ref.quantise(w)
                    assert bool(((g - w).abs() <= s.to(F64).repeat_interleave(32, -1) * 0.501 + 2.0 ** -7 * w.abs() + 1e-5).all())
                o, l, mag, big = ref.attend(r[b, :ql[b]].cpu().to(F64), gk, gv, ql[b])
                to, tl = ref.attend_bounds(dtype, lens[b], D, o, l, mag, big)
                assert bool(((out[b, :ql[b]].cpu().to(F64) - o).abs() <= to).all())
                assert bool(((lse[b, :ql[b]].cpu().to(F64) - l).abs() <= tl).all())
        cache.sync_status()


# ---- calls that share something ---------------------------------------------------------

@pytest.mark.parametrize("dtype,rot", [(BF, 128), (F32, 0)])
def test_nan_is_stored_as_zero_in_every_group(dtype, rot):
    """One NaN in each group of 32 numbers, so that groups which float64 has to decide hold one, too."""
    H_kv, D, P, n = 2, 128, 64, 900
    pool = ref.Pool(16, H_kv, D, P, seed=1)
    table = tables([n], P, 16, 3)
    k, v = normal(21, 1, n, H_kv, D, dtype=dtype) + 2, normal(22, 1, n, H_kv, D, dtype=dtype) - 2
    k[..., 5::32], v[..., 9::32] = math.nan, math.nan
    spec = Rope(rot, base=500000.0) if rot else None
    with new_cache(pool) as cache:
        cache.append(k.cuda(), v.cuda(), table.cuda(), i32([n]), i32([n]), rope=spec)
        with pytest.raises(AtlaskvError) as e:
            cache.sync_status()
        assert e.value.status == binding.ATLASKV_EDEVICE
        w = k[0].to(F64)
        w = (ref.rotate(w, torch.arange(n), spec) if rot else w).nan_to_num(nan=0.0)
        for i in range(n):
            for h in range(H_kv):
                pool.write(int(table[0, i // P]), i % P, h, w[i, h], v[0, i, h].to(F64).nan_to_num(nan=0.0))
        assert torch.equal(cache.pages.cpu(), pool.bytes())


def test_sequences_share_pages():
    """A common prefix, and a page twice in one table: reading and attending only look at what the table names."""
    D, H_kv, H, P = 64, 2, 6, 16
    pool = ref.Pool(8, H_kv, D, P)
    pool.fill(torch.arange(8), 8 * P, 3)
    table = torch.tensor([[1, 2, 3, 4], [1, 2, 6, 6], [5, 5, 5, 5]], dtype=torch.int32)
    lens = [64, 50, 63]
    for N in (1, 30):
        q = normal(4, 3, N, H, D, dtype=BF)
        with new_cache(pool) as cache:
            out, lse = cache.attend(q.cuda(), table.cuda(), i32(lens))
            gk, gv = cache.read(64, table.cuda(), i32(lens), i32(lens))
            cache.sync_status()
        for b, n in enumerate(lens):
            k, v = pool.all(table[b], n)
            assert torch.equal(gk[b, :n].cpu().to(F64), k) and torch.equal(gv[b, :n].cpu().to(F64), v)
            o, l, mag, big = ref.attend(q[b].to(F64), k, v, N)
            to, tl = ref.attend_bounds(BF, n, D, o, l, mag, big)
            assert bool(((out[b].cpu().to(F64) - o).abs() <= to).all())
            assert bool(((lse[b].cpu().to(F64) - l).abs() <= tl).all())


def test_pages_past_four_gigabytes():
    D, H_kv, H, P, lens = 128, 8, 16, 256, [700, 300]
    width = KvCache.page_bytes(H_kv, D, P)
    n_pages = (1 << 32) // width + 40
    with KvCache.allocate(n_pages, H_kv, D, P) as far, KvCache.allocate(8, H_kv, D, P) as near:
        far.pages[-8:].zero_()
        near.pages.zero_()
        low = torch.arange(8, dtype=torch.int32).view(2, 4)
        high = low + (n_pages - 8)
        spec, kv = Rope(128), i32(lens)
        for N in (700, 1):
            q, k, v = (normal(s + N, 2, N, h, D, dtype=BF).cuda() for s, h in ((1, H), (2, H_kv), (3, H_kv)))
            ql = i32([min(n, N) for n in lens])
            got = []
            for cache, tab in ((far, high.cuda()), (near, low.cuda())):
                r = cache.append(k, v, tab, kv, ql, rope=spec, q=q, q_out=torch.zeros_like(q))
                out, lse = (torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda"))
                cache.attend(r, tab, kv, ql, out=out, lse=lse)
                got.append((r, out, lse) + cache.read(N, tab, kv, ql))
                cache.sync_status()
            assert all(torch.equal(a, b) for a, b in zip(*got))
        assert torch.equal(far.pages[-8:][:3], near.pages[:3])


def test_two_calls_at_once():
    """One cache, two streams, a workspace each: decode steps beside a prompt, again and again."""
    D, H_kv, H, P = 128, 2, 8, 16
    pool = ref.Pool(200, H_kv, D, P)
    table = tables([900, 800, 700], P, 200, 1)
    for b, n in enumerate([900, 800, 700]):
        pool.fill(table[b], n, b)
    dt, kv = table.cuda(), i32([900, 800, 700])
    q1, q2 = normal(1, 3, 1, H, D, dtype=BF).cuda(), normal(2, 3, 300, H, D, dtype=BF).cuda()
    with new_cache(pool) as cache:
        want = [cache.attend(q, dt, kv) for q in (q1, q2)] + [cache.read(700, dt, kv)]
        torch.cuda.synchronize()
        sides = [torch.cuda.Stream() for _ in range(3)]
        for _ in range(5):
            got = []
            for q, s in zip((q1, q2), sides):
                got.append(cache.attend(q, dt, kv, stream=s))
            got.append(cache.read(700, dt, kv, stream=sides[2]))
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for e, f in zip(want, got) for a, b in zip(e, f))
        cache.sync_status()


def test_outputs_on_another_stream_wait_for_their_memory():
    """Memory that the current stream's work has not let go of yet is not written by a call on another stream first."""
    D, H_kv, H, P, N = 128, 2, 8, 16, 70
    pool = ref.Pool(60, H_kv, D, P)
    table = tables([400, 300], P, 60, 1)
    pool.fill(table[0], 400, 1)
    pool.fill(table[1], 300, 2)
    dt, kv, spec = table.cuda(), i32([400, 300]), Rope(128)
    q, k, v = (normal(s, 2, N, h, D, dtype=BF).cuda() for s, h in ((1, H), (2, H_kv), (3, H_kv)))
    pos = i32([[3] * N] * 2)
    side = torch.cuda.Stream()
    with new_cache(pool) as cache:
        calls = {
            "rope": lambda s: (binding.rope(q, pos, spec, stream=s),),
            "append": lambda s: (cache.append(k, v, dt, kv, rope=spec, q=q, stream=s),),
            "attend": lambda s: cache.attend(q, dt, kv, stream=s),
            "read": lambda s: cache.read(N, dt, kv, stream=s),
        }
        for name, call in calls.items():
            want = [x.clone() for x in call(None)]
            torch.cuda.synchronize()
            old = [torch.empty_like(x) for x in want]
            torch.cuda._sleep(20_000_000)          # about 10 ms, then the old tensors' last use
            for x in old:
                x.fill_(7.0)
            del old, x
            got = call(side)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, got)), name
        cache.sync_status()


def test_queries_rotated_in_place_and_shapes_refused():
    D, H_kv, H, P, N = 64, 1, 3, 16, 5
    spec, kv, ql, tab = Rope(32, interleaved=True), i32([9, 5]), i32([5, 2]), i32([[0], [1]])
    q, k, v = (normal(s, 2, N, h, D, dtype=F32).cuda() for s, h in ((1, H), (2, H_kv), (3, H_kv)))
    with KvCache.allocate(2, H_kv, D, P) as cache:
        want = cache.append(k, v, tab, kv, ql, rope=spec, q=q, q_out=q.clone())
        assert torch.equal(want[1, 2:], q[1, 2:])
        r = q.clone()
        assert cache.append(k, v, tab, kv, ql, rope=spec, q=r, q_out=r).data_ptr() == r.data_ptr()
        assert torch.equal(r, want)
        for bad in (lambda: cache.append(k[0], v[0], tab, kv), lambda: cache.attend(q[0], tab, kv)):
            with pytest.raises(AtlaskvError):
                bad()
        cache.sync_status()
