"""Knowledge-graph attention with the sequence in the 4-bit cache: against the
64-bit oracle on the numbers that the cache holds, and against atlaskv_attend
fed with the same numbers read back."""
import numpy as np
import pytest
import torch

import oracle
from hierarchical_kv_pruning_b200 import binding, synth
from hierarchical_kv_pruning_b200.binding import AtlaskvError, CsrHikvpTree, HikvpTree, KvCache, Rope
from tests._util import oracle_tree, storage

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def setup(dtype, H, H_kv, D, N, lens, P, seed, host=None, fanout=(9, 8, 7), keep=(3, 5, 20)):
    """A workload whose sequences of lens tokens are in a cache: (workload, cache, table, kv_len)."""
    T = max(max(lens), N)
    sh = synth.custom(dtype=dtype, n_heads=H, n_kv_heads=H_kv, head_dim=D, fanout=fanout, keep=keep, batch=len(lens),
                      n_tokens=N, seq_len=T, permuted=host is None)
    w = synth.make_workload(sh, "cuda", seed)
    # both lambda weights matter
    w.q_kg.mul_(0.15)
    if host:
        f = {n: getattr(w, n).cpu().pin_memory() for n in ("leaf_keys", "leaf_values") + (("mid_keys",) if host == 2 else ())}
        w = synth.Workload(sh, w.root_keys, f.get("mid_keys", w.mid_keys), f["leaf_keys"], f["leaf_values"], w.root_child,
                           w.mid_child, w.q_kg, w.q_seq, w.k_seq, w.v_seq, w.targets)
    width = -(-T // P) + 1
    g = torch.Generator().manual_seed(seed)
    table = torch.randperm(len(lens) * width + 2, generator=g)[: len(lens) * width].view(len(lens), width).to(torch.int32).cuda()
    cache = KvCache.allocate(len(lens) * width + 2, H_kv, D, P)
    cache.pages.fill_(255)      # unused slots read as NaN
    cache.append(w.k_seq[:, :T], w.v_seq[:, :T], table, i32(lens), i32(lens))
    return w, cache, table, i32(lens)


def check(w, cache, table, kv_len, r):
    sh = w.shape
    B, N, lens = sh.batch, sh.n_tokens, kv_len.tolist()
    T = max(max(lens), 1)
    k, v = cache.read(T, table, kv_len, kv_len, dtype=sh.dtype)
    cache.sync_status()
    t = oracle_tree(w)
    for b in range(B):
        q_kg, q_seq = storage(w.q_kg[b:b + 1]), storage(w.q_seq[b:b + 1])
        n = lens[b]
        assert n >= N
        ref = oracle.hikvp(t, q_kg, q_seq, storage(k[b:b + 1, :n]), storage(v[b:b + 1, :n]), sh.keep)
        for i, (_, h) in enumerate(ref["traversals"]):
            for name in ("kept_root", "kept_mid", "kept_leaf"):
                assert r[name][b, h].tolist() == ref[name][i].tolist(), (name, b, h)
            err = float(np.max(np.abs(r["out"][b, :, h].double().cpu().numpy() - ref["y"][i])))
            assert err <= (1e-5 * np.max(np.abs(ref["y"][i])) if sh.dtype == F32 else 2e-2), (b, h, err)
            lerr = float(np.max(np.abs(r["lse"][b, :, h].double().cpu().numpy() - ref["lse"][i])))
            assert lerr <= (1e-4 if sh.dtype == F32 else 2e-3), (b, h, lerr)


@pytest.mark.parametrize("dtype,H,H_kv,D,N,lens,P,host", [
    (BF, 8, 2, 128, 1, [1, 17, 300], 16, None),
    (BF, 8, 2, 128, 20, [20, 37, 150], 32, None),        # many rows: the tcgen05 kernel
    (BF, 4, 1, 64, 3, [3, 64, 65], 64, None),
    (BF, 4, 2, 64, 64, [64, 200], 16, None),
    (F32, 4, 2, 128, 2, [2, 45, 90], 16, None),
    (F32, 2, 1, 64, 5, [5, 33], 256, None),
    (BF, 8, 2, 128, 4, [4, 40, 90, 33, 64, 18, 7, 200, 31], 16, 1),      # host-resident leaves, in query chunks
    (BF, 4, 1, 128, 33, [33, 90], 32, 2),                                # host-resident mids too
    (F32, 4, 2, 64, 2, [2, 45], 16, 1),
])
def test_attend_cached(dtype, H, H_kv, D, N, lens, P, host):
    w, cache, table, kv = setup(dtype, H, H_kv, D, N, lens, P, 5, host)
    with HikvpTree.from_workload(w) as tree, cache:
        r = tree.attend_cached(w.q_kg, w.q_seq, cache, table, kv, w.shape.keep)
        tree.sync_status()
        check(w, cache, table, kv, r)
        again = tree.attend_cached(w.q_kg, w.q_seq, cache, table, kv, w.shape.keep, workspace=r["workspace"])
        assert all(torch.equal(r[n], again[n]) for n in ("out", "lse", "kept_root", "kept_mid", "kept_leaf"))


def test_same_as_attend_on_the_numbers_read_back():
    w, cache, table, kv = setup(BF, 8, 2, 128, 16, [80, 80], 16, 6)
    with HikvpTree.from_workload(w) as tree, cache:
        r = tree.attend_cached(w.q_kg, w.q_seq, cache, table, kv, w.shape.keep)
        k, v = cache.read(80, table, kv, kv)
        d = tree.attend(w.q_kg, w.q_seq, k, v, w.shape.keep)
        tree.sync_status()
        assert torch.equal(r["kept_leaf"], d["kept_leaf"])
        # two roundings of probabilities and of the result to bfloat16 on values of a few units
        assert float((r["out"].double() - d["out"].double()).abs().max()) <= 2e-2
        assert float((r["lse"] - d["lse"]).abs().max()) <= 2e-3


def test_empty_sequence_gets_the_knowledge_part():
    w, cache, table, kv = setup(BF, 4, 2, 128, 1, [1, 30], 16, 7)
    with HikvpTree.from_workload(w) as tree, cache:
        r = tree.attend_cached(w.q_kg, w.q_seq, cache, table, i32([0, 30]), w.shape.keep)
        tree.sync_status()
        cache.sync_status()
        for h in range(4):
            rows = r["kept_leaf"][0, h].long()
            k, v = (x[h // 2, rows].double() for x in (w.leaf_keys, w.leaf_values))
            logit = k @ w.q_kg[0, 0, h].double() * 128 ** -0.5
            assert float((torch.softmax(logit, 0) @ v - r["out"][0, 0, h].double()).abs().max()) <= 2e-2
            assert abs(float(torch.logsumexp(logit, 0) - r["lse"][0, 0, h])) <= 2e-3


def test_decode_steps_captured():
    """A decode step (append with the query's rotation, then attend) captured once and replayed as the sequences grow."""
    H, H_kv, D, P, B, steps = 8, 2, 128, 16, 3, 6
    w, cache, table, kv = setup(BF, H, H_kv, D, 1, [40, 15, 30], P, 8)
    spec = Rope(128)
    q, k, v = (torch.randn(B, 1, h, D, device="cuda").to(BF) for h in (H, H_kv, H_kv))
    with HikvpTree.from_workload(w) as tree, cache:
        def step():
            r = cache.append(k, v, table, kv, rope=spec, q=q)
            return tree.attend_cached(w.q_kg, r, cache, table, kv, w.shape.keep)
        kv += 1
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
        for i in range(steps):
            kv += 1
            q.copy_(torch.randn(B, 1, H, D, device="cuda"))
            k.copy_(torch.randn(B, 1, H_kv, D, device="cuda"))
            g.replay()
            snap = {n: got[n].clone() for n in ("out", "lse", "kept_root", "kept_mid", "kept_leaf")}
            want = step()
            assert all(torch.equal(snap[n], want[n]) for n in snap)
            rot = binding.rope(q, (kv - 1).view(B, 1), spec)
            wl = synth.Workload(w.shape, *[getattr(w, n) for n in (
                "root_keys", "mid_keys", "leaf_keys", "leaf_values", "root_child", "mid_child", "q_kg")], rot, w.k_seq,
                w.v_seq, w.targets)
            if i in (0, steps - 1):
                check(wl, cache, table, kv, snap)
        tree.sync_status()


def test_refusals():
    w, cache, table, kv = setup(BF, 4, 2, 64, 2, [10, 20], 16, 9)
    K = w.shape.keep
    with HikvpTree.from_workload(w) as tree, cache:
        p = tree.params(K)
        ok = tree.attend_cached(w.q_kg, w.q_seq, cache, table, kv, K)
        other = KvCache.allocate(4, 1, 64, 16)
        wide = KvCache.allocate(4, 2, 128, 16)
        for bad in (lambda: tree.attend_cached(w.q_kg, w.q_seq, other, table, kv, K),
                    lambda: tree.attend_cached(w.q_kg, w.q_seq, wide, table, kv, K),
                    lambda: tree.attend_cached(w.q_kg, w.q_seq, cache, table[:1], kv, K),
                    lambda: tree.attend_cached(w.q_kg, w.q_seq[:1], cache, table, kv, K),
                    lambda: tree.attend_cached(w.q_kg, w.q_seq.float(), cache, table, kv, K),
                    lambda: tree.attend_cached(w.q_kg, w.q_seq, cache, table, kv, (3, 5, 2000)),
                    lambda: tree.attend_cached(w.q_kg, w.q_seq, cache, table, kv, K,
                                               workspace=ok["workspace"][:ok["workspace"].numel() // 256 * 256 - 256])):
            with pytest.raises(AtlaskvError):
                bad()
        io = binding.atlaskv_io(2, 2, 4, 0, w.q_kg.data_ptr(), w.q_seq.data_ptr(), None, None, ok["out"].data_ptr())
        for seqs in (cache._seqs(2, 2, table, kv, kv), cache._seqs(2, 1, table, kv, None),
                     binding.atlaskv_seqs(2, 2, 0, table.data_ptr(), kv.data_ptr(), None),
                     binding.atlaskv_seqs(2, 2, 2, None, kv.data_ptr(), None)):
            with pytest.raises(AtlaskvError) as e:
                binding.atlaskv_attend_cached(tree.handle, p, io, cache.handle, seqs, ok["workspace"].data_ptr(),
                                              ok["workspace"].numel())
            assert e.value.status == binding.ATLASKV_EINVAL
        for args in ((None, p, cache.handle), (tree.handle, p, None)):
            with pytest.raises(AtlaskvError):
                binding.atlaskv_workspace_size_cached(*args, 2, 2, 4)
        none = tree.attend_cached(w.q_kg[:0], w.q_seq[:0], cache, table[:0], kv[:0], K)
        assert none["out"].shape[0] == 0
    cw = synth.make_csr_workload(synth.CsrShape("csr", BF, 4, 2, 64, 6, ((3, 4), (2, 3)), (2, 3, 4), 1, 2, 3), "cuda")
    with CsrHikvpTree.from_workload(cw) as csr, KvCache.allocate(4, 2, 64, 16) as c2:
        with pytest.raises(AtlaskvError) as e:
            binding.atlaskv_workspace_size_cached(csr.handle, binding.atlaskv_params(1, 1, 1, 0.0), c2.handle, 1, 1, 4)
        assert e.value.status == binding.ATLASKV_EUNSUPPORTED
