"""Calls of the rotary-position and cache operators at the edges of what they
take: tensors that share memory, groups whose roundings are close, batches that
mix long and short work, refused calls."""
import pytest
import torch

from hierarchical_kv_pruning_b200 import binding
from hierarchical_kv_pruning_b200.binding import AtlaskvError, KvCache, Rope
from tests import _cache_ref as ref
from tests.test_gpu_cache import BF, F32, F64, check_attend, i32, new_cache, normal, tables

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
