"""Refusals of the operators from a prompt to a cache within a budget, on the host and without a GPU: bad arguments are
reported before anything is launched, by the C entries and by the Python wrappers."""
import ctypes

import pytest
import torch

from test_cache_abi import ARG, DTYPE, P, heads


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
