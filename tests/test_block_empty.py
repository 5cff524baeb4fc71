"""Calls without rows whose gate has no row either (a gate for each token of an
empty batch), on a machine without a GPU: nothing is launched by the forward call."""

import ctypes

import pytest

A = 0x7f0000000000   # never dereferenced
G = 1 << 30


@pytest.fixture(scope="module")
def lib():
    from newton_schulz_orthogonalized_amd import _lib
    return _lib


def _fwd(lib, **kw):
    d = dict(residual=None, update=None, gate=None, post_weight=A, pre_weight=A + G, new_residual=None, normed=None, rows=0, dim=64,
             groups=0, residual_dtype=lib.MU_BF16, dtype=lib.MU_BF16, weight_dtype=lib.MU_F32, post_norm=1, residual_scale=1.0, eps=1e-6)
    return lib.MuResnorm(**{**d, **kw})


@pytest.mark.parametrize("gate", [None, A + 2 * G])
def test_no_rows_and_no_gates(lib, gate):
    assert lib.LIB.mu_residual_norm(ctypes.byref(_fwd(lib, gate=gate)), None) == lib.MU_OK
    a = lib.MuResnormGrad(fwd=_fwd(lib, gate=gate))
    need = ctypes.c_size_t(7)
    assert lib.LIB.mu_residual_norm_grad_workspace_size(ctypes.byref(a), ctypes.byref(need)) == lib.MU_OK and need.value == 0
    assert lib.LIB.mu_residual_norm_grad(ctypes.byref(a), None, 0, None) == lib.MU_OK


@pytest.mark.parametrize("kw", [dict(rows=4), dict(rows=4, gate=A + 2 * G), dict(groups=-1), dict(groups=2)])
def test_other_group_counts_stay_refused(lib, kw):
    a = _fwd(lib, **{**dict(residual=A + 3 * G, update=A + 4 * G, new_residual=A + 5 * G, normed=A + 6 * G), **kw})
    assert lib.LIB.mu_residual_norm(ctypes.byref(a), None) == lib.MU_ERR_INVALID_ARG
    need = ctypes.c_size_t(0)
    g = lib.MuResnormGrad(fwd=a)
    assert lib.LIB.mu_residual_norm_grad_workspace_size(ctypes.byref(g), ctypes.byref(need)) == lib.MU_ERR_INVALID_ARG
