"""Rotary frequencies, and the refusals of the rotary and cache entry points
that need no GPU."""
import ctypes
import math

import pytest
import torch

from hierarchical_kv_pruning_b200 import binding, build
from tests import _cache_ref as ref


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def test_rope_frequencies(lib):
    s = binding.Rope(64, base=500000.0).spec
    for i in range(32):
        assert s.freq[i] == pytest.approx(500000.0 ** (-2 * i / 64), rel=1e-14)
    assert s.freq[32] == 0.0 and s.layout == binding.ATLASKV_ROPE_HALF and s.amplitude == 1.0
    lin = binding.Rope(64, factor=4.0).spec                       # no original length: every frequency
    assert lin.freq[3] == pytest.approx(10000.0 ** (-6 / 64) / 4, rel=1e-14)
    L, lo, hi = 8192, 1.0, 4.0
    b = binding.Rope(128, base=500000.0, interleaved=True, factor=8.0, original_len=L, low_turns=lo, high_turns=hi,
                     amplitude=1.25).spec
    seen = set()
    for i in range(64):
        f = 500000.0 ** (-2 * i / 128)
        turns = L * f / (2 * math.pi)
        if turns > hi:
            want, kind = f, "kept"
        elif turns < lo:
            want, kind = f / 8, "divided"
        else:
            w = (turns - lo) / (hi - lo)
            want, kind = w * f + (1 - w) * f / 8, "mixed"
        seen.add(kind)
        assert b.freq[i] == pytest.approx(want, rel=1e-12)
    assert seen == {"kept", "divided", "mixed"} and b.amplitude == 1.25


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=24), dict(rotary_dim=144), dict(rotary_dim=-16), dict(base=0.0),
    dict(base=math.inf), dict(base=math.nan), dict(factor=0.0), dict(factor=-1.0), dict(factor=math.nan),
    dict(original_len=-1), dict(original_len=math.inf), dict(low_turns=4.0, high_turns=4.0), dict(low_turns=-1.0),
    dict(high_turns=math.inf), dict(amplitude=math.nan), dict(amplitude=math.inf),
])
def test_rope_init_refuses(lib, kw):
    with pytest.raises(binding.AtlaskvError) as e:
        binding.Rope(**{"rotary_dim": 64, **kw})
    assert e.value.status == binding.ATLASKV_EINVAL
    assert lib.atlaskv_rope_init(None, 0, 64, 1e4, 1.0, 0.0, 1.0, 32.0, 1.0) == binding.ATLASKV_EINVAL
    spec = binding.atlaskv_rope_spec()
    assert lib.atlaskv_rope_init(ctypes.byref(spec), 2, 64, 1e4, 1.0, 0.0, 1.0, 32.0, 1.0) == binding.ATLASKV_EINVAL


def _rope_io(**kw):
    f = dict(dtype=binding.ATLASKV_BF16, H=4, head_dim=128, tokens=3, x=4096, x_stride=0, positions=4096, y=8192,
             y_stride=0, backward=0)
    f.update(kw)
    return binding.atlaskv_rope_io(*[f[n] for n, _ in binding.atlaskv_rope_io._fields_])


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), "EINVAL"), (dict(H=0), "EINVAL"), (dict(head_dim=96), "EUNSUPPORTED"), (dict(tokens=-1), "EINVAL"),
    (dict(x=None), "EINVAL"), (dict(y=None), "EINVAL"), (dict(positions=None), "EINVAL"), (dict(x=4098), "EINVAL"),
    (dict(y=8200), "EINVAL"), (dict(positions=4097), "EINVAL"), (dict(x_stride=511), "EINVAL"),
    (dict(x_stride=516), "EINVAL"), (dict(y_stride=-512), "EINVAL"), (dict(backward=2), "EINVAL"),
    (dict(y=4096, y_stride=1024), "EINVAL"), (dict(head_dim=64), "EINVAL"),     # rotary_dim 128 above the head
])
def test_rope_refuses(lib, kw, status):
    spec = binding.Rope(128).spec
    assert lib.atlaskv_rope(ctypes.byref(spec), ctypes.byref(_rope_io(**kw)), None) == \
        getattr(binding, "ATLASKV_" + status)
    assert binding.atlaskv_last_error()


def test_rope_refuses_bad_specs(lib):
    for field, bad in (("layout", 3), ("rotary_dim", 20), ("rotary_dim", 0), ("amplitude", math.nan)):
        spec = binding.Rope(64).spec
        setattr(spec, field, bad)
        assert lib.atlaskv_rope(ctypes.byref(spec), ctypes.byref(_rope_io()), None) == binding.ATLASKV_EINVAL
    spec = binding.Rope(64).spec
    spec.freq[5] = math.inf
    assert lib.atlaskv_rope(ctypes.byref(spec), ctypes.byref(_rope_io()), None) == binding.ATLASKV_EINVAL
    assert lib.atlaskv_rope(None, ctypes.byref(_rope_io()), None) == binding.ATLASKV_EINVAL
    spec = binding.Rope(64).spec
    assert lib.atlaskv_rope(ctypes.byref(spec), None, None) == binding.ATLASKV_EINVAL
    assert lib.atlaskv_rope(ctypes.byref(spec), ctypes.byref(_rope_io(tokens=0, x=None)), None) == binding.ATLASKV_OK


def test_page_bytes(lib):
    assert binding.KvCache.page_bytes(8, 128, 16) == 8 * 2560
    assert binding.KvCache.page_bytes(3, 64, 256) == 3 * 16 * 1280
    for args, status in (((0, 128, 16), "EINVAL"), ((8, 96, 16), "EUNSUPPORTED"), ((8, 128, 8), "EUNSUPPORTED"),
                         ((8, 128, 48), "EUNSUPPORTED"), ((8, 128, 512), "EUNSUPPORTED")):
        with pytest.raises(binding.AtlaskvError) as e:
            binding.KvCache.page_bytes(*args)
        assert e.value.status == getattr(binding, "ATLASKV_" + status)
    assert lib.atlaskv_cache_page_bytes(8, 128, 16, None) == binding.ATLASKV_EINVAL


@pytest.mark.parametrize("kw,status", [
    (dict(n_kv_heads=0), "EINVAL"), (dict(head_dim=32), "EUNSUPPORTED"), (dict(page_size=17), "EUNSUPPORTED"),
    (dict(n_pages=0), "EINVAL"), (dict(n_pages=1 << 31), "EINVAL"), (dict(pages=None), "EINVAL"),
    (dict(pages=4104), "EINVAL"),
])
def test_create_cache_refuses(lib, kw, status):
    f = dict(n_kv_heads=2, head_dim=64, page_size=16, n_pages=4, pages=4096)
    f.update(kw)
    d = binding.atlaskv_cache_desc(*[f[n] for n, _ in binding.atlaskv_cache_desc._fields_])
    out = ctypes.c_void_p()
    assert lib.atlaskv_create_cache(ctypes.byref(d), None, ctypes.byref(out)) == getattr(binding, "ATLASKV_" + status)
    assert out.value is None
    assert lib.atlaskv_create_cache(None, None, ctypes.byref(out)) == binding.ATLASKV_EINVAL
    assert lib.atlaskv_create_cache(ctypes.byref(d), None, None) == binding.ATLASKV_EINVAL


def test_null_caches(lib):
    sz = ctypes.c_size_t()
    seqs, a, t = binding.atlaskv_seqs(), binding.atlaskv_append_io(), binding.atlaskv_cache_attend_io()
    assert lib.atlaskv_cache_append(None, None, ctypes.byref(seqs), ctypes.byref(a), None) == binding.ATLASKV_EINVAL
    assert lib.atlaskv_cache_read(None, ctypes.byref(seqs), 1, None, None, None) == binding.ATLASKV_EINVAL
    assert lib.atlaskv_cache_attend(None, ctypes.byref(seqs), ctypes.byref(t), None, 0, None) == binding.ATLASKV_EINVAL
    assert lib.atlaskv_cache_workspace_size(None, 1, 1, 1, 1, ctypes.byref(sz)) == binding.ATLASKV_EINVAL
    assert lib.atlaskv_cache_sync_status(None, None) == binding.ATLASKV_EINVAL
    assert lib.atlaskv_destroy_cache(None) == binding.ATLASKV_OK


@pytest.mark.parametrize("D", [64, 128])
def test_reference_layout_covers_a_block_once(D):
    kc, ks, vc, vs = ref.addresses(D)
    got = torch.cat([kc[:, ::2].flatten(), vc[:, ::2].flatten()] +
                    [x[:, ::32].flatten() + i for x, o in ((ks, (0, 1, 2, 3)), (vs, (0, 1, 4, 5))) for i in o])
    assert got.sort().values.tolist() == list(range(20 * D))


def test_reference_storing_stays_within_half_a_step():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(200, 128, generator=g, dtype=ref.F64) * 3 + 2
    c, s, m = ref.quantise(x)
    v = ref.value(c, s, m)
    half = s.to(ref.F64).repeat_interleave(32, -1) / 2
    assert bool(((v - x).abs() <= half + 2.0 ** -8 * v.abs()).all())
    pool = ref.Pool(3, 2, 128, 32, seed=3)
    for i in range(40):
        pool.write([2, 0][i // 32], i % 32, i % 2, x[i], x[i + 40])
    for i in range(40):
        k, w = pool.read([2, 0][i // 32], i % 32, i % 2)
        assert torch.equal(k, v[i]) and torch.equal(w, v[i + 40])
    a, b = pool.all([2, 0], 40)
    p, q = pool.history([2, 0], 40)
    assert torch.equal(a.nan_to_num(), p.nan_to_num()) and torch.equal(b.nan_to_num(), q.nan_to_num())


def test_rope_refuses_more_heads_than_it_counts(lib):
    spec = binding.Rope(128).spec
    for H in ((1 << 20) + 1, (1 << 31) - 1):
        assert lib.atlaskv_rope(ctypes.byref(spec), ctypes.byref(_rope_io(H=H)), None) == binding.ATLASKV_EUNSUPPORTED


ROW_SHAPES = [((1, 1), (8, 1)), ((1, 1), (3, 5)), ((1, 5), (3, 5)), ((3, 1), (3, 5)), ((1, 1), (1, 5))]


@pytest.mark.parametrize("have,want", ROW_SHAPES)
def test_rows_refuses_tokens_that_share_memory(have, want):
    """The C ABI takes a token stride of 0 for a dense tensor: an expanded one would be read, or written, past its
    storage.  Its copy is dense, and one token may have any stride."""
    shape = torch.Size(want + (4, 128))
    x = torch.zeros(have + (4, 128)).expand(shape)
    with pytest.raises(binding.AtlaskvError) as e:
        binding._rows("x", x, shape, torch.float32)
    assert e.value.status == binding.ATLASKV_EINVAL
    assert binding._rows("x", x.contiguous(), shape, torch.float32) == 0
    over = torch.zeros(4096).as_strided(shape, (want[1] * 256, 256, 128, 1))      # rows of 512 elements, 256 apart
    with pytest.raises(binding.AtlaskvError):
        binding._rows("x", over, shape, torch.float32)


def test_rows_takes_slices_of_wider_rows():
    wide = torch.zeros(3, 5, 7, 128)
    assert binding._rows("x", wide[:, :, :4], torch.Size((3, 5, 4, 128)), torch.float32) == 7 * 128
    assert binding._rows("x", wide[:, :1, 2:3], torch.Size((3, 1, 1, 128)), torch.float32) == 5 * 7 * 128
    assert binding._rows("x", wide[:1, :, :4], torch.Size((1, 5, 4, 128)), torch.float32) == 7 * 128
    one = wide[:1, :1, :4].expand(1, 1, 4, 128)
    assert binding._rows("x", one, torch.Size((1, 1, 4, 128)), torch.float32) in (0, 4 * 128)
    assert binding._rows("x", wide[:0, :, :4], torch.Size((0, 5, 4, 128)), torch.float32) == 0


def test_workspaces_are_their_own_bytes():
    """A workspace whose bytes repeat or skip memory would be written past, or between, them."""
    ws = torch.empty(1024, dtype=torch.uint8)
    assert binding._space(ws) == (ws.data_ptr(), 1024) and binding._space(ws[256:])[1] == 768
    assert binding._space(ws.view(torch.float32))[1] == 1024
    for bad in (ws[:1].expand(1 << 30), ws[::2], ws.view(32, 32)[:, :16]):
        with pytest.raises(binding.AtlaskvError) as e:
            binding._space(bad)
        assert e.value.status == binding.ATLASKV_EINVAL
