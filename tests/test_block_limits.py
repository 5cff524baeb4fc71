"""Sizes of the gated product beyond one launch, on a machine without a GPU: they
are refused before anything is launched, by the workspace query too. (A call that
has launched its first kernels ends with status 5 here, no GPU.)"""

import ctypes

import pytest
import torch

A = 0x7f0000000000   # never dereferenced
T = 1 << 46

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="its addresses must not reach a kernel")


@pytest.fixture(scope="module")
def lib():
    from newton_schulz_orthogonalized_amd import _lib
    return _lib


def _both(lib, a, name):
    need = ctypes.c_size_t(0)
    query = getattr(lib.LIB, name + "_workspace_size")(ctypes.byref(a), ctypes.byref(need))
    return query, getattr(lib.LIB, name)(ctypes.byref(a), A - T, 1 << 62, None)


MANY = [(2 ** 31 - 1, 65, 4097, 1), (2 ** 31 - 1, 65, 4097, 0), (2 ** 30, 1, 1 << 14, 1), (1 << 27, 7, 1 << 20, 0)]


@pytest.mark.parametrize("tokens,dim,hidden,dtype", MANY)
def test_forward(lib, tokens, dim, hidden, dtype):
    a = lib.MuGated(x=A, w_gate=A + T, w_up=A + 2 * T, h=A - 2 * T, tokens=tokens, dim=dim, hidden=hidden, dtype=dtype, activation=0)
    assert _both(lib, a, "mu_gated_mlp") == (lib.MU_ERR_INVALID_ARG, lib.MU_ERR_INVALID_ARG)
    assert "one launch" in lib.mu_last_error()


def _grad(lib, tokens, dim, hidden, dtype, **kw):
    d = dict(grad_h=A - 2 * T, x=A, w_gate=A + T // 64, w_up=A + T // 32, tokens=tokens, dim=dim, hidden=hidden, dtype=dtype, grad_dtype=0)
    return lib.MuGatedGrad(**{**d, **kw})


@pytest.mark.parametrize("gates", [False, True])
@pytest.mark.parametrize("tokens,dim,hidden,dtype", [(2 ** 31 - 1, 4097, 65, 1), (2 ** 31 - 1, 4097, 65, 0)])
def test_gradient_of_x(lib, tokens, dim, hidden, dtype, gates):
    """The products before it (gates computed again, or their slopes) would fit."""
    kw = dict(gate=A - T, up=A - T + T // 4) if gates else {}
    assert _both(lib, _grad(lib, tokens, dim, hidden, dtype, dx=A + T, **kw), "mu_gated_mlp_grad") == (1, 1)


def test_gradients_of_the_weights(lib):
    """Behind dx, which would fit: it is not launched either."""
    a = _grad(lib, 70, 1 << 20, 1 << 20, 0, w_gate=A + T // 2, w_up=A + T // 2 + T // 8, dx=A - T, d_gate=A + T, d_up=A + T + T // 8)
    assert _both(lib, a, "mu_gated_mlp_grad") == (1, 1)


@pytest.mark.parametrize("tokens,dim,hidden", [(8192, 4096, 14336), (150001, 64, 14336), (1, 1 << 20, 1 << 20), (1 << 20, 1, 1 << 16)])
def test_sizes_within_it(lib, tokens, dim, hidden):
    need = ctypes.c_size_t(0)
    for dtype in (0, 1):
        a = lib.MuGated(x=A, w_gate=A + T, w_up=A + 2 * T, h=A - 2 * T, tokens=tokens, dim=dim, hidden=hidden, dtype=dtype, activation=0)
        assert lib.LIB.mu_gated_mlp_workspace_size(ctypes.byref(a), ctypes.byref(need)) == 0


def test_zeros_of_no_tokens(lib):
    a = _grad(lib, 0, 1 << 20, 1 << 20, 1, d_gate=A + T, d_up=A + 2 * T)
    assert _both(lib, a, "mu_gated_mlp_grad") == (1, 1)
