"""The cache operators' refusals, on the host and without a GPU: bad arguments are reported before anything is
launched, by the C entries and by the Python wrappers."""
import ctypes

import pytest
import torch

import cache_reference as ref

ARG, DTYPE, ALIGN = 1, 2, 3
P = ctypes.c_void_p(16)


@pytest.fixture(scope="module")
def lib():
    from sampling_row_online_gb300 import binding, build
    build.build()
    return binding.library()


def cache(**kw):
    from sampling_row_online_gb300.binding import CacheStruct
    a = dict(k=16, v=16, k_scale=16, v_scale=16, pages=8, kv_heads=2, page_size=64, head_dim=128, kind=0)
    a.update(kw)
    return ctypes.byref(CacheStruct(*a.values()))


def heads(data=16):
    from sampling_row_online_gb300.binding import HeadsStruct
    return ctypes.byref(HeadsStruct(data, 1024, 256, 128))


def attention(lib, c=None, **kw):
    a = dict(table=P, per=4, ctx=P, counts=None, q=heads(), mask=None, B=2, N=3, Hq=4, dtype=1, scale=0.1, out=P, lse=None)
    a.update(kw)
    return lib.spec_cache_attention(c or cache(), *a.values(), None)


def write(lib, c=None, **kw):
    a = dict(table=P, per=4, ctx=P, counts=None, k=heads(), v=heads(), B=2, N=3, dtype=1)
    a.update(kw)
    return lib.spec_cache_write(c or cache(), *a.values(), None)


def read(lib, c=None, **kw):
    a = dict(table=P, per=4, start=None, counts=None, k=P, v=P, B=2, N=3, dtype=0)
    a.update(kw)
    return lib.spec_cache_read(c or cache(), *a.values(), None)


def commit(lib, c=None, **kw):
    a = dict(table=P, per=4, ctx=P, parent=P, each=1, tokens=P, path=P, length=P, B=2, N=5, P=3, index=P, new=P)
    a.update(kw)
    return lib.spec_cache_commit(c or cache(), *a.values(), None)


def rope(lib, **kw):
    freq = (ctypes.c_double * 64)(*([0.5] * 64))
    a = dict(q=heads(), k=heads(), oq=heads(), ok=heads(), qw=None, kw=None, base=None, offset=None, B=1, N=2, Hq=2, Hk=1, D=128,
             dtype=1, norm=1, eps=1e-6, freq=ctypes.cast(freq, ctypes.c_void_p), rot=128, pairs=0)
    a.update(kw)
    return lib.spec_qk_norm_rope(*a.values(), None)


CALLS = [attention, write, read, commit]


@pytest.mark.parametrize("call", CALLS)
def test_the_cache_is_checked(lib, call):
    assert call(lib, B=0) == 0
    assert call(lib, cache(), B=-1) == ARG
    assert call(lib, cache(), B=65536) == ARG
    assert call(lib, cache(kind=2)) == DTYPE
    for d in (0, 32, 96, 256):
        assert call(lib, cache(head_dim=d)) == ARG
    for page in (0, 8, 48, 256):
        assert call(lib, cache(page_size=page)) == ARG
    assert call(lib, cache(kv_heads=0)) == ARG
    assert call(lib, cache(pages=0)) == ARG
    assert call(lib, per=0) == ARG
    assert call(lib, per=1 << 27) == ARG
    assert call(lib, table=None) == ARG
    for name in ("k", "v", "k_scale", "v_scale"):
        assert call(lib, cache(**{name: None})) == ARG
    assert call(lib, cache(k=24)) == ALIGN
    assert call(lib, cache(v=17)) == ALIGN


def test_attention_refusals(lib):
    assert attention(lib, dtype=0) == DTYPE                 # no fp32 queries
    assert attention(lib, dtype=3) == DTYPE
    assert attention(lib, N=-1) == ARG
    assert attention(lib, N=65537) == ARG
    assert attention(lib, N=0) == 0
    assert attention(lib, Hq=3) == ARG                      # not a multiple of 2 kv heads
    assert attention(lib, Hq=0) == ARG
    for s in (float("nan"), float("inf")):
        assert attention(lib, scale=s) == ARG
    for name in ("ctx", "q", "out"):
        assert attention(lib, **{name: None}) == ARG
    assert attention(lib, q=heads(None)) == ARG
    assert attention(lib, out=ctypes.c_void_p(24)) == ALIGN


def test_write_and_read_refusals(lib):
    for call in (write, read):
        assert call(lib, dtype=3) == DTYPE
        assert call(lib, N=-1) == ARG
        assert call(lib, N=0) == 0
        assert call(lib, k=None) == ARG
        assert call(lib, v=None) == ARG
    assert write(lib, ctx=None) == ARG
    assert write(lib, k=heads(None)) == ARG
    assert read(lib, k=ctypes.c_void_p(20)) == ALIGN


def test_commit_refusals(lib):
    assert commit(lib, N=0) == ARG
    assert commit(lib, N=1025) == ARG
    assert commit(lib, P=0) == ARG
    assert commit(lib, P=6) == ARG                          # longer than the tree has nodes
    assert commit(lib, each=2) == ARG
    for name in ("ctx", "parent", "tokens", "path", "length", "index", "new"):
        assert commit(lib, **{name: None}) == ARG


def test_norm_rope_refusals(lib):
    assert rope(lib, B=0) == 0
    assert rope(lib, N=0) == 0
    assert rope(lib, Hq=0, Hk=0) == 0
    assert rope(lib, B=-1) == ARG
    assert rope(lib, dtype=3) == DTYPE
    for d in (0, 7, 514):
        assert rope(lib, D=d, rot=0) == ARG
    assert rope(lib, rot=130) == ARG
    assert rope(lib, rot=3) == ARG
    assert rope(lib, rot=-2) == ARG
    assert rope(lib, freq=None) == ARG
    assert rope(lib, eps=-1.0) == ARG
    assert rope(lib, eps=float("nan")) == ARG
    assert rope(lib, norm=2) == ARG
    assert rope(lib, pairs=2) == ARG
    assert rope(lib, norm=0, qw=P) == ARG                   # weights without the norm
    assert rope(lib, q=None) == ARG
    assert rope(lib, ok=None) == ARG
    assert rope(lib, k=heads(None)) == ARG
    bad = (ctypes.c_double * 64)(*([float("inf")] * 64))
    assert rope(lib, freq=ctypes.cast(bad, ctypes.c_void_p)) == ARG


def test_the_wrappers_check_tensors():
    from sampling_row_online_gb300 import SpecCache, binding
    k = torch.zeros((4, 2, 16, 64), dtype=torch.int8)
    s = torch.ones((4, 2))
    with pytest.raises(ValueError):
        SpecCache(k, k, s, s)                                # on the host
    with pytest.raises(ValueError):
        SpecCache(k.float(), k, s, s)
    with pytest.raises(ValueError):
        SpecCache(k, k[:, :1], s, s)
    with pytest.raises(ValueError):
        SpecCache(k, k, s[:2], s)
    with pytest.raises(TypeError):
        SpecCache(k, k, s.double(), s)
    q = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        binding.spec_cache_attention(q, None, torch.zeros((1, 4), dtype=torch.int32), None)
    with pytest.raises(TypeError):
        binding.spec_qk_norm_rope(q, None)                   # on the host
    with pytest.raises(ValueError):
        binding.spec_qk_norm_rope(None, None)
    with pytest.raises(TypeError):
        binding.spec_qk_norm_rope(q.long(), None)


def test_status_codes_have_names(lib):
    assert lib.spec_error_string(9) == b"SPEC_ERR_PAGE"
    assert lib.spec_error_string(10) == b"SPEC_ERR_NONFINITE"


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_the_reference_rounds_as_torch_does(kind):
    """The tests' own rounding against torch's conversion, and its scales against their definition."""
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(4000, generator=g) * 60, torch.randn(4000, generator=g) * 0.02, torch.tensor([0.0, -0.0, 448.0, 0.5, 1.5, 2.5])])
    x = x.clamp(-ref.QMAX[kind], ref.QMAX[kind])
    want = x.to(torch.float8_e4m3fn) if kind == "e4m3" else x.round().clamp(-127, 127).to(torch.int8)
    assert torch.equal(ref.nearest(x.double(), kind).view(torch.uint8), want.view(torch.uint8))
    q = ref.QMAX[kind]
    assert ref.scale_for(0.0, kind) == 2.0 ** -100
    assert ref.scale_for(q, kind) == 1.0 and ref.scale_for(q * 1.01, kind) == 2.0 and ref.scale_for(q / 2, kind) == 0.5
