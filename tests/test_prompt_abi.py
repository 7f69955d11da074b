"""Refusals of the operators from a prompt to a cache within a budget, on the host and without a GPU: bad arguments are
reported before anything is launched, by the C entries and by the Python wrappers."""
import ctypes

import pytest
import torch

from test_cache_abi import ALIGN, ARG, DTYPE, P, cache, heads


@pytest.fixture(scope="module")
def lib():
    from sampling_row_online_gb300 import binding, build
    build.build()
    return binding.library()


def axes(lib, **kw):
    freq, axis = (ctypes.c_double * 64)(*([0.5] * 64)), (ctypes.c_int32 * 64)(*([i % 3 for i in range(64)]))
    a = dict(q=heads(), k=heads(), oq=heads(), ok=heads(), qw=None, kw=None, base=None, positions=P, axes=3, B=1, N=2, Hq=2, Hk=1,
             D=128, dtype=1, norm=1, eps=1e-6, freq=ctypes.cast(freq, ctypes.c_void_p), axis=ctypes.cast(axis, ctypes.c_void_p),
             rot=128, pairs=0)
    a.update(kw)
    return lib.spec_qk_norm_rope_axes(*a.values(), None)


def prompt(lib, **kw):
    a = dict(q=heads(), k=heads(), v=heads(), starts=P, B=2, T=9, Hq=4, Hk=2, D=128, dtype=1, scale=0.1, out=P, lse=None)
    a.update(kw)
    return lib.spec_prompt_attention(*a.values(), None)


def weights(lib, c=None, **kw):
    a = dict(table=P, per=4, ctx=P, counts=None, q=heads(), mask=None, lse=P, B=2, N=3, Hq=4, dtype=1, scale=0.1, weights=P)
    a.update(kw)
    return lib.spec_cache_weights(c or cache(), *a.values(), None)


def evict(lib, c=None, **kw):
    a = dict(table=P, per=4, ctx=P, weights=P, B=2, keep=100, first=4, last=32, index=P, new=ctypes.c_void_p(32))
    a.update(kw)
    return lib.spec_cache_evict(c or cache(), *a.values(), None)


@pytest.mark.parametrize("call", [weights, evict])
def test_the_cache_is_checked(lib, call):
    assert call(lib, B=0) == 0
    assert call(lib, B=-1) == ARG
    assert call(lib, B=65536) == ARG
    assert call(lib, cache(kind=2)) == DTYPE
    assert call(lib, cache(head_dim=96)) == ARG
    assert call(lib, cache(page_size=48)) == ARG
    assert call(lib, cache(kv_heads=0)) == ARG
    assert call(lib, per=0) == ARG
    assert call(lib, per=1 << 27) == ARG
    assert call(lib, table=None) == ARG
    assert call(lib, cache(k=None)) == ARG
    assert call(lib, cache(v=17)) == ALIGN


def test_prompt_refusals(lib):
    assert prompt(lib, T=0) == 0
    for dtype in (0, 3, -1):
        assert prompt(lib, dtype=dtype) == DTYPE            # no fp32
    for d in (0, 32, 96, 256):
        assert prompt(lib, D=d) == ARG
    assert prompt(lib, B=-1) == ARG
    assert prompt(lib, B=65536) == ARG
    assert prompt(lib, T=-1) == ARG
    assert prompt(lib, T=(1 << 30) + 1) == ARG
    assert prompt(lib, Hq=3) == ARG                         # not a multiple of 2 kv heads
    assert prompt(lib, Hq=0) == ARG
    assert prompt(lib, Hk=0) == ARG
    for s in (float("nan"), float("inf")):
        assert prompt(lib, scale=s) == ARG
    for name in ("q", "k", "v", "starts", "out"):
        assert prompt(lib, **{name: None}) == ARG
    for name in ("q", "k", "v"):
        assert prompt(lib, **{name: heads(None)}) == ARG
    assert prompt(lib, out=ctypes.c_void_p(24)) == ALIGN


def test_weights_refusals(lib):
    assert weights(lib, N=0) == 0
    for dtype in (0, 3):
        assert weights(lib, dtype=dtype) == DTYPE
    assert weights(lib, N=-1) == ARG
    assert weights(lib, N=65537) == ARG
    assert weights(lib, Hq=3) == ARG
    assert weights(lib, scale=float("nan")) == ARG
    for name in ("ctx", "q", "lse", "weights"):
        assert weights(lib, **{name: None}) == ARG
    assert weights(lib, q=heads(None)) == ARG
    assert weights(lib, weights=ctypes.c_void_p(24)) == ALIGN


def test_evict_refusals(lib):
    for keep in (0, -1, (1 << 30) + 1):
        assert evict(lib, keep=keep, first=0, last=0) == ARG
    for first, last in ((-1, 0), (0, -1), (101, 0), (0, 101), (60, 41)):
        assert evict(lib, first=first, last=last) == ARG
    for name in ("ctx", "weights", "index", "new"):
        assert evict(lib, **{name: None}) == ARG
    assert evict(lib, new=P) == ARG                         # ctx_len's own memory
    assert evict(lib, weights=ctypes.c_void_p(24)) == ALIGN


def test_the_wrappers_check_tensors():
    from sampling_row_online_gb300 import binding
    q, k = torch.zeros((5, 4, 64), dtype=torch.bfloat16), torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    starts = torch.tensor([0, 5], dtype=torch.int32)
    with pytest.raises(TypeError):
        binding.spec_prompt_attention(q, k, k, starts)      # on the host
    with pytest.raises(ValueError):
        binding.spec_prompt_attention(q[None], k, k, starts)
    with pytest.raises(TypeError):
        binding.spec_prompt_attention(q.long(), k, k, starts)
    table = torch.zeros((1, 4), dtype=torch.int32)
    with pytest.raises(TypeError):
        binding.spec_cache_weights(q[None], None, table, None, None, None)
    with pytest.raises(TypeError):
        binding.spec_cache_evict(None, table, None, None, 4)


def test_axes_refusals(lib):
    assert axes(lib, B=0) == 0
    assert axes(lib, N=0) == 0
    for n in (0, -1, 9):
        assert axes(lib, axes=n) == ARG
    assert axes(lib, positions=None) == ARG
    assert axes(lib, axis=None) == ARG
    assert axes(lib, freq=None) == ARG
    for bad in (3, -1):
        wrong = (ctypes.c_int32 * 64)(*([0] * 63 + [bad]))
        assert axes(lib, axis=ctypes.cast(wrong, ctypes.c_void_p)) == ARG
    assert axes(lib, dtype=3) == DTYPE
    assert axes(lib, D=7, rot=0) == ARG
    assert axes(lib, rot=130) == ARG
    assert axes(lib, norm=0, qw=P) == ARG
    assert axes(lib, q=None) == ARG
    assert axes(lib, ok=None) == ARG


def test_the_axes_wrapper_checks_tensors():
    from sampling_row_online_gb300 import binding
    q = torch.zeros((1, 5, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        binding.spec_qk_norm_rope_axes(q, None, None, None, None)     # on the host
    with pytest.raises(ValueError):
        binding.spec_qk_norm_rope_axes(None, None, None, None, None)
