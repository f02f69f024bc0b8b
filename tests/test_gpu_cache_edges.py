"""Calls of the rotary-position and cache operators at the edges of what they
take: tensors that share memory, groups whose roundings are close, batches that
mix long and short work, refused calls."""
import pytest
import torch

from hierarchical_kv_pruning_b200 import binding
from hierarchical_kv_pruning_b200.binding import AtlaskvError, HikvpTree, KvCache, Rope
from tests import _cache_ref as ref
from tests.test_gpu_cache import BF, F32, F64, check_attend, i32, new_cache, normal
from tests.test_gpu_cache_tree import setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("have,want", [((1, 1), (4, 1)), ((1, 1), (4, 3)), ((1, 3), (4, 3)), ((4, 1), (4, 3)), ((1, 1), (1, 3))])
def test_expanded_tensors_are_refused_and_their_copies_taken(have, want):
    D, H_kv, H, P = 128, 2, 4, 16
    B, N = want
    x, k = normal(1, *have, H, D, dtype=BF).cuda(), normal(2, *have, H_kv, D, dtype=BF).cuda()
    spec, pos = Rope(128), i32([[5] * N] * B)
    tab, kv = i32([[b] for b in range(B)]), i32([9] * B)
    ex, ek = x.expand(B, N, H, D), k.expand(B, N, H_kv, D)
    cx, ck = ex.contiguous(), ek.contiguous()
    with KvCache.allocate(B, H_kv, D, P) as cache:
        cache.pages.zero_()
        for bad in (lambda: binding.rope(ex, pos, spec), lambda: binding.rope(cx, pos, spec, out=torch.empty_like(x).expand_as(cx)),
                    lambda: cache.append(ek, ck, tab, kv), lambda: cache.append(ck, ek, tab, kv),
                    lambda: cache.append(ck, ck, tab, kv, q=ex), lambda: cache.attend(ex, tab, kv)):
            with pytest.raises(AtlaskvError) as e:
                bad()
            assert e.value.status == binding.ATLASKV_EINVAL
        one = binding.rope(x, pos[:have[0], :have[1]].contiguous(), spec)
        assert torch.equal(binding.rope(cx, pos, spec), one.expand_as(cx))
        cache.append(ck, ck, tab, kv, q=cx)
        cache.attend(cx, tab, kv)
        cache.sync_status()


def test_many_key_tiles_again_and_again():
    """Row blocks of prompts over many key tiles, so that every buffer of the tensor-memory ring is written over many
    times by the two issuing warps: right, and the same each time."""
    check_attend(BF, 128, 1, 4, 64, 130, [2900, 700], seed=31)
    D, H_kv, H, P, n = 128, 2, 8, 64, 6000
    pool = ref.Pool(n // P + 3, H_kv, D, P)
    table = torch.arange(n // P + 1, dtype=torch.int32).repeat(2, 1)
    pool.fill(table[0], n, 3)
    dt, kv = table.cuda(), i32([n, n - 77])
    q = normal(5, 2, 400, H, D, dtype=BF).cuda()
    with new_cache(pool) as cache:
        first = cache.attend(q, dt, kv)
        for _ in range(20):
            assert all(torch.equal(a, b) for a, b in zip(first, cache.attend(q, dt, kv)))
        cache.sync_status()


def test_maxima_that_grow_along_the_sequence():
    """Keys that grow fourfold every 64 tokens: each key tile of a prompt makes the softmax store its probabilities
    again with a larger maximum."""
    D, P, n, N = 128, 64, 640, 140
    pool = ref.Pool(n // P, 1, D, P)
    table = torch.arange(n // P, dtype=torch.int32)[None]
    d = normal(41, D, dtype=BF)
    k = normal(42, 1, n, 1, D) + d.float() * (4.0 ** (torch.arange(n) // 64 - 6.0))[:, None, None]
    v = normal(43, 1, n, 1, D, dtype=BF)
    q = d + normal(44, 1, N, 4, D, dtype=BF) * 0.1
    with new_cache(pool) as cache:
        cache.append(k.to(BF).cuda(), v.cuda(), table.cuda(), i32([n]))
        out, lse = cache.attend(q.cuda(), table.cuda(), i32([n]), scale=0.3)
        cache.sync_status()
        kk, vv = (x[0].cpu().to(F64) for x in cache.read(n, table.cuda(), i32([n])))
    o, l, mag, big = ref.attend(q[0].to(F64), kk, vv, N, 0.3)
    to, tl = ref.attend_bounds(BF, n, D, o, l, mag, big)
    assert bool(((out[0].cpu().to(F64) - o).abs() <= to).all())
    assert bool(((lse[0].cpu().to(F64) - l).abs() <= tl).all())


def test_decode_rows_before_a_prompt_block():
    """One call of many single tokens over a long history and one block of 240 rows a KV head: the row tile that the single tokens
    leave empty waits for the block through all of them."""
    D, H_kv, H, P, n, B, N = 128, 2, 8, 64, 2048, 601, 60
    pool = ref.Pool(n // P, H_kv, D, P)
    table = torch.arange(n // P, dtype=torch.int32).repeat(B, 1)       # every sequence has the same history
    pool.fill(table[0], n, 3)
    one, block = normal(51, 1, 1, H, D, dtype=BF), normal(52, 1, N, H, D, dtype=BF)
    q = torch.zeros(B, N, H, D, dtype=BF)
    q[:-1, :1], q[-1:] = one, block
    ql = [1] * (B - 1) + [N]
    with new_cache(pool) as cache:
        out, lse = cache.attend(q.cuda(), table.cuda(), i32([n] * B), i32(ql))
        cache.sync_status()
    k, v = pool.all(table[0], n)
    for x, rows, m in ((one, out[:-1, :1], 1), (block, out[-1:], N)):
        o, l, mag, big = ref.attend(x[0].to(F64), k, v, m)
        to, _ = ref.attend_bounds(BF, n, D, o, l, mag, big)
        assert bool(((rows.cpu().to(F64) - o).abs() <= to).all())


# ---- stored bytes where the roundings are close ---------------------------------------

def stored_bytes(pool, table, lens, k, v):
    """Fill the pool with the definition's bytes of k, v [B][N][H_kv][D] (float64), all tokens at once."""
    kc, ks, vc, vs = ref.addresses(pool.D)
    for b, n in enumerate(lens):
        slot = torch.arange(n)
        page, blk, tok = table[b, slot // pool.P].long(), slot % pool.P // 16, slot % 16
        at = [x.view(-1, 1, 1) for x in (page, blk)]
        head = torch.arange(pool.H).view(1, -1, 1)
        for x, code, sc, dl in ((k[b, :n], kc, ks, 2), (v[b, :n], vc, vs, 4)):
            c, s, m = ref.quantise(x)
            pool.raw[at[0], head, at[1], code[tok][:, None, ::2]] = (c[..., ::2] | (c[..., 1::2] << 4)).to(torch.uint8)
            for o, w in ((0, s), (dl, m)):
                bits = w.contiguous().view(torch.int16).to(torch.int32) & 0xffff
                where = sc[tok][:, None, ::32] + o
                pool.raw[at[0], head, at[1], where] = (bits & 255).to(torch.uint8)
                pool.raw[at[0], head, at[1], where + 1] = (bits >> 8).to(torch.uint8)


def check_bytes(k, v, spec, P=64):
    """What append stores of k, v [1][n][H_kv][D] in slots 0 .. n - 1 against the definition."""
    n, H_kv, D = k.shape[1:]
    pool = ref.Pool(-(-n // P), H_kv, D, P, seed=1)
    table = torch.randperm(-(-n // P), generator=torch.Generator().manual_seed(7)).to(torch.int32)[None]
    with new_cache(pool) as cache:
        cache.append(k.cuda(), v.cuda(), table.cuda(), i32([n]), rope=spec)
        cache.sync_status()
        got = cache.pages.cpu()
    w = k.to(F64)
    w = ref.rotate(w[0], torch.arange(n), spec)[None] if spec else w
    stored_bytes(pool, table, [n], w, v.to(F64))
    assert torch.equal(got, pool.bytes()), int((got != pool.bytes()).sum())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,H_kv", [(128, 4), (64, 1)])
def test_stored_bytes_of_tiny_numbers_beside_large_ones(dtype, D, H_kv):
    """Groups in which a number is 2^-30 of the range: the difference to the minimum has more bits than a float32, and
    it decides the scale's rounding (a range just above 15 codes) or which of two codes is nearer (a tie without it)."""
    tiny = 2.0 ** -30
    base = torch.linspace(0.25, 14.0, 32).to(BF).float()

    def group(*special):
        x = base.clone()
        x[torch.tensor([5 * i + 1 for i in range(len(special))])] = torch.tensor(special)
        return x
    groups = [group(15.0, -tiny), group(15.0, tiny), group(15.0, 0.0)]                    # scale 1.0078125, 1, 1
    step = 0.99609375                                                                     # of a range of 14.9375
    for low in (-tiny, tiny, 0.0):
        groups.append(torch.cat([group(14.9375, low, step / 2, step)[:31], torch.tensor([step / 2])]))
    for h in (0.5, 1.5, 4.5, 7.5):                                                        # scale 1, minimum -h
        mid = torch.linspace(-h, 15.0 - h, 32).to(BF).float()
        for t in (tiny, -tiny, 0.0):
            x = mid.clone()
            x[0], x[31], x[7], x[20] = -h, 15.0 - h, t, -t
            groups.append(x)
    x = torch.stack(groups)
    x = torch.cat([x * s for s in (1.0, 2.0 ** 40, 2.0 ** -40, 2.0 ** 100)])
    order = torch.randperm(len(x) * 8, generator=torch.Generator().manual_seed(2))
    rows = x.repeat(8, 1)[order][: len(x) * 8 // (D // 32 * H_kv) * (D // 32 * H_kv)].view(1, -1, H_kv, D).to(dtype)
    check_bytes(rows, rows.flip(1), None)


def turned_back(target, spec, dtype):
    """Keys whose rotation by their slots is about target [n][H_kv][D]."""
    return (ref.rotate(target, torch.arange(target.shape[0]), spec, backward=True) / spec.spec.amplitude ** 2).to(dtype)[None]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,inter,rot", [(128, False, 128), (128, True, 128), (128, False, 48), (64, False, 64),
                                         (128, False, 96), (64, True, 48), (64, False, 16)])
@pytest.mark.parametrize("kind", ["small first half", "small second half", "offsets", "narrow"])
def test_stored_bytes_of_rotations_that_cancel(dtype, D, inter, rot, kind):
    """Rotated numbers far smaller than their pairs (a group's partners a thousand times as large), keys with channel
    offsets, and groups whose range is small beside their offset: float32's error is that of the pair."""
    H_kv, n = 2, 1500
    spec = Rope(rot, base=500000.0, interleaved=inter, factor=2.0, amplitude=1.2)
    g = torch.Generator().manual_seed(61)
    x = torch.randn(n, H_kv, D, generator=g, dtype=F64)
    i = torch.arange(rot // 2)
    first = 2 * i if inter else i
    second = first + (1 if inter else rot // 2)
    if kind == "small first half":
        x[..., second] *= 1000
    elif kind == "small second half":
        x[..., first] *= 1000
    elif kind == "offsets":
        x += 4 * torch.randn(H_kv, D, generator=g, dtype=F64)
    else:
        x = 100 + 0.5 * x
    k = turned_back(x, spec, dtype)
    check_bytes(k, normal(62, 1, n, H_kv, D, dtype=dtype), spec)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_stored_bytes_of_huge_and_tiny_groups(dtype):
    """Rotated groups above 2^100, where they used not to be decided in float64, and around the smallest scale."""
    spec = Rope(128, amplitude=0.9)
    x = torch.randn(800, 1, 128, generator=torch.Generator().manual_seed(63), dtype=F64)
    e = torch.arange(800) % 8
    x *= (2.0 ** torch.tensor([110.0, 117.0, 101.0, 0.0, -98.0, -99.0, -100.0, -104.0], dtype=F64))[e][:, None, None]
    k = turned_back(x, spec, dtype)
    n = k.shape[1]
    w = ref.rotate(k[0].to(F64), torch.arange(n), spec)
    assert float(w.abs().max()) < 2.0 ** 120
    pool = ref.Pool(16, 1, 128, 64, seed=1)
    table = torch.arange(16, dtype=torch.int32)[None]
    with new_cache(pool) as cache:
        cache.append(k.cuda(), k.cuda(), table.cuda(), i32([n]), rope=spec)
        cache.sync_status()
        got = cache.pages.cpu()
    want = ref.Pool(16, 1, 128, 64, seed=1)
    stored_bytes(want, table, [n], w[None], k.to(F64))
    # groups whose scale is below 2^-100 have scale 0 and codes 0
    kc, ks, vc, vs = ref.addresses(128)
    for y, code, sc in ((w, kc, ks), (k[0].to(F64), vc, vs)):
        s = ref.quantise(y)[1]
        for t, _, gr in torch.nonzero(s.to(F64) < 2.0 ** -100).tolist():
            blk = want.raw[t // 64, 0, t % 64 // 16]
            blk[code[t % 16, 32 * gr:32 * gr + 32:2]] = 0
            blk[sc[t % 16, 32 * gr]] = blk[sc[t % 16, 32 * gr] + 1] = 0
    assert torch.equal(got, want.bytes()), int((got != want.bytes()).sum())


# ---- the whole attention with a cached sequence --------------------------------------

@pytest.mark.parametrize("host", [None, 1])
def test_attend_cached_refuses_before_it_starts(host):
    """A refused call has written nothing, whatever it is refused for."""
    w, cache, table, kv = setup(BF, 4, 2, 64, 2, [30, 45], 16, 5, host)
    B, N, H, K = 2, 2, 4, w.shape.keep
    with HikvpTree.from_workload(w) as tree, cache:
        p = tree.params(K)
        size = binding.atlaskv_workspace_size_cached(tree.handle, p, cache.handle, B, N, H)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        out, kept = torch.full_like(w.q_seq, 7.0), [torch.full((B, H, k), -7, dtype=torch.int32, device="cuda") for k in K]
        io = binding.atlaskv_io(B, N, H, N, w.q_kg.data_ptr(), w.q_seq.data_ptr(), None, None, out.data_ptr(), None,
                                *[x.data_ptr() for x in kept])
        seqs = lambda **kw: binding.atlaskv_seqs(*{**dict(B=B, N=N, max_pages=table.shape[1], block_table=table.data_ptr(),  # noqa: E731
                                                          kv_len=kv.data_ptr(), q_len=None), **kw}.values())
        for bad, status in ((dict(block_table=table.data_ptr() + 2), "EINVAL"), (dict(kv_len=kv.data_ptr() + 1), "EINVAL"),
                            (dict(max_pages=1 << 27), "EUNSUPPORTED"), (dict(max_pages=0), "EINVAL"),
                            (dict(block_table=None), "EINVAL"), (dict(kv_len=None), "EINVAL")):
            with pytest.raises(AtlaskvError) as e:
                binding.atlaskv_attend_cached(tree.handle, p, io, cache.handle, seqs(**bad), ws.data_ptr(), size)
            assert e.value.status == getattr(binding, "ATLASKV_" + status)
            torch.cuda.synchronize()
            assert bool((out == 7.0).all()) and all(bool((x == -7).all()) for x in kept)
        with pytest.raises(AtlaskvError):
            binding.atlaskv_attend_cached(tree.handle, p, io, cache.handle, seqs(), ws.data_ptr(), size - 256)
        torch.cuda.synchronize()
        assert bool((out == 7.0).all()) and all(bool((x == -7).all()) for x in kept)
        binding.atlaskv_attend_cached(tree.handle, p, io, cache.handle, seqs(), ws.data_ptr(), size,
                                      torch.cuda.current_stream().cuda_stream)
        tree.sync_status()
        cache.sync_status()
        assert all(bool((x >= 0).all()) for x in kept)


@pytest.mark.parametrize("dtype,host", [(BF, None), (F32, None), (BF, 1), (F32, 1)])
def test_stage_times_hold_the_cached_sequence_part(dtype, host):
    w, cache, table, kv = setup(dtype, 4, 2, 64, 2, [300, 45], 16, 5, host)
    with HikvpTree.from_workload(w) as tree, cache:
        binding.atlaskv_set_profiling(tree.handle, binding.ATLASKV_PROFILE_TIMES)
        tree.attend_cached(w.q_kg, w.q_seq, cache, table, kv, w.shape.keep)
        ms = binding.atlaskv_stage_times(tree.handle)
        assert ms[3] > 0 and ms[4] > 0 and ms[2] == pytest.approx(ms[3] + ms[4], rel=1e-5)
        k, v = cache.read(300, table, kv, kv, dtype=dtype)
        tree.attend(w.q_kg, w.q_seq, k, v, w.shape.keep)          # an earlier call's time does not stay
        ms = binding.atlaskv_stage_times(tree.handle)
        assert (ms[3] > 0) == (dtype == BF and host is not None)


# ---- the rotation's gradient --------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("inter", [False, True])
def test_rope_records_its_gradient(dtype, inter):
    """A tensor that requires a gradient gets the transpose's, and the transpose of that the rotation's."""
    spec, pos = Rope(48, interleaved=inter, amplitude=1.3), i32([[0, 3, 70000], [12, 9, 1 << 20]])
    x, g, gg = (normal(s, 2, 3, 2, 64, dtype=dtype).cuda() for s in (1, 2, 3))
    for back in (False, True):
        leaf = x.clone().requires_grad_()
        y = binding.rope(leaf, pos, spec, backward=back)
        assert y.requires_grad and torch.equal(y, binding.rope(x, pos, spec, backward=back))
        up = g.clone().requires_grad_()
        d, = torch.autograd.grad(y, leaf, up, create_graph=True)
        assert torch.equal(d, binding.rope(g, pos, spec, backward=not back))
        dd, = torch.autograd.grad(d, up, gg)
        assert torch.equal(dd, binding.rope(gg, pos, spec, backward=back))
        with torch.no_grad():
            assert not binding.rope(leaf, pos, spec, backward=back).requires_grad
        # a gradient that is expanded, as a sum's is
        s, = torch.autograd.grad(binding.rope(leaf, pos, spec, backward=back).sum(), leaf)
        assert torch.equal(s, binding.rope(torch.ones_like(x), pos, spec, backward=not back))


def test_rope_gradient_through_a_wider_projection():
    """A slice of a projection, on another stream, in a captured step."""
    spec, pos = Rope(64), i32([[0, 3, 70000], [12, 9, 1 << 20]])
    wide = normal(4, 2, 3, 6, 128, dtype=BF).cuda().requires_grad_()
    g = normal(5, 2, 3, 4, 128, dtype=BF).cuda()
    want = torch.zeros_like(wide)
    want[:, :, 1:5] = binding.rope(g, pos, spec, backward=True)

    def step():
        return torch.autograd.grad(binding.rope(wide[:, :, 1:5], pos, spec), wide, g)[0]
    assert torch.equal(step(), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step()
        graph.replay()
    side.synchronize()
    assert torch.equal(got, want)


def test_rope_out_refuses_to_lose_a_gradient():
    spec, pos = Rope(64), i32([[0, 1, 2], [3, 4, 5]])
    x = normal(1, 2, 3, 4, 64, dtype=BF).cuda().requires_grad_()
    with pytest.raises(AtlaskvError) as e:
        binding.rope(x, pos, spec, out=torch.empty_like(x))
    assert e.value.status == binding.ATLASKV_EINVAL
    with torch.no_grad():
        assert torch.equal(binding.rope(x, pos, spec, out=torch.empty_like(x)), binding.rope(x, pos, spec))


def test_expanded_workspaces_are_refused():
    w, cache, table, kv = setup(BF, 4, 2, 64, 2, [30, 45], 16, 5)
    bad = torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 30)
    with HikvpTree.from_workload(w) as tree, cache:
        for call in (lambda: cache.attend(w.q_seq, table, kv, workspace=bad),
                     lambda: tree.attend_cached(w.q_kg, w.q_seq, cache, table, kv, w.shape.keep, workspace=bad)):
            with pytest.raises(AtlaskvError) as e:
                call()
            assert e.value.status == binding.ATLASKV_EINVAL


@pytest.mark.parametrize("D", [64, 128])
def test_float32_outputs_do_not_shrink_with_the_length(D):
    """The matrix unit cuts its sums, so a running sum over thousands of steps comes out too small.  The share by which
    the outputs are, sum (y - o) o / sum o^2, is at most 3 cut steps of a 16-token sum (2^-23 each) and 6 of a
    32-channel logit, whose shrinking moves outputs by no more than that times the logits' spread of 1.5: 12 2^-23.  The
    roundings of 16 D outputs average out below 2^-24, of which three times as much is allowed: 13.5 2^-23."""
    n, B, N, H, P = 16000, 600, 2, 8, 64
    pool = ref.Pool(n // P, 1, D, P)
    table = torch.arange(n // P, dtype=torch.int32).repeat(B, 1)       # enough equal sequences that a CTA takes whole ones
    pool.fill(table[0], n, 3)
    q = normal(71, 1, N, H, D)
    with new_cache(pool) as cache:
        out, _ = cache.attend(q.repeat(B, 1, 1, 1).cuda(), table.cuda(), i32([n] * B))
        cache.sync_status()
    k, v = pool.all(table[0], n)
    o = ref.attend(q[0].to(F64), k, v, N)[0].cuda()
    share = ((out.double() - o) * o).sum((1, 2, 3)) / (o * o).sum()
    assert float(share.abs().max()) <= 13.5 * 2.0 ** -23, (float(share.min()), float(share.max()))
