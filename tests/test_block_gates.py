"""Refusals of the gated product's gates by type and size, on a machine without a
GPU."""

import ctypes

import pytest
import torch

A = 0x7f0000000000   # never dereferenced
G = 1 << 30


@pytest.fixture(scope="module")
def lib():
    from newton_schulz_orthogonalized_amd import _lib
    return _lib


def _query(lib, a, name):
    need = ctypes.c_size_t(0)
    return getattr(lib.LIB, name + "_workspace_size")(ctypes.byref(a), ctypes.byref(need))


def _gated(lib, **kw):
    d = dict(x=A, w_gate=A + G, w_up=A + 2 * G, h=A + 3 * G, gate_out=A + 4 * G, up_out=A + 5 * G, tokens=20, dim=64, hidden=96,
             dtype=lib.MU_BF16, activation=0)
    return lib.MuGated(**{**d, **kw})


def _grad(lib, **kw):
    d = dict(grad_h=A, x=A + G, w_gate=A + 2 * G, w_up=A + 3 * G, gate=A + 7 * G, up=A + 8 * G, dx=A + 4 * G, d_gate=A + 5 * G,
             d_up=A + 6 * G, tokens=20, dim=64, hidden=96, dtype=lib.MU_BF16, grad_dtype=lib.MU_F32, accumulate=0, activation=0)
    return lib.MuGatedGrad(**{**d, **kw})


@pytest.mark.parametrize("act", range(4))
def test_float32_gates_need_twice_the_room(lib, act):
    """Side by side as bfloat16, on one another as float32."""
    half, flag = 20 * 96 * 2, lib.MU_GATES_F32
    for at, plain, f32 in ((half, 0, 3), (2 * half, 0, 0), (half - 2, 3, 3)):
        assert _query(lib, _gated(lib, up_out=A + 4 * G + at, activation=act), "mu_gated_mlp") == plain
        assert _query(lib, _gated(lib, up_out=A + 4 * G + at, activation=act | flag), "mu_gated_mlp") == f32
    # an input of the gradient beside one of its results
    for at, plain, f32 in ((half, 0, 3), (2 * half, 0, 0)):
        assert _query(lib, _grad(lib, gate=A + 4 * G - at, activation=act), "mu_gated_mlp_grad") == plain
        assert _query(lib, _grad(lib, gate=A + 4 * G - at, activation=act | flag), "mu_gated_mlp_grad") == f32
    assert _query(lib, _gated(lib, gate_out=A + 4 * G + 2, activation=act), "mu_gated_mlp") == 0
    assert _query(lib, _gated(lib, gate_out=A + 4 * G + 2, activation=act | flag), "mu_gated_mlp") == 3


@pytest.mark.parametrize("act", [4, 0x104, 0x200, 0x1ff, -1, -257, 0x300])
def test_unknown_activations_stay_refused(lib, act):
    assert _query(lib, _gated(lib, activation=act), "mu_gated_mlp") == 1
    assert _query(lib, _grad(lib, activation=act), "mu_gated_mlp_grad") == 1


def test_types_of_gates(lib):
    import newton_schulz_orthogonalized_amd as nso
    x, w, h = (torch.zeros(s, dtype=torch.bfloat16) for s in ((6, 8), (10, 8), (6, 10)))
    for t in (torch.bfloat16, torch.float32):
        flag = lib.MU_GATES_F32 if t == torch.float32 else 0
        gates = torch.zeros(2, 6, 10, dtype=t)
        a = lib.gated(x, w, w, h, gates, "gelu")
        assert a.activation == 1 | flag and a.up_out - a.gate_out == 60 * t.itemsize
        a = lib.gated_grad(h, x, w, w, gates, None, None, None, False, "gelu")
        assert a.activation == 1 | flag and a.up - a.gate == 60 * t.itemsize
    for bad in (torch.float16, torch.float64):
        with pytest.raises(ValueError):
            lib.gated(x, w, w, h, torch.zeros(2, 6, 10, dtype=bad), "silu")
        with pytest.raises(ValueError):
            lib.gated_grad(h, x, w, w, torch.zeros(2, 6, 10, dtype=bad), None, None, None, False, "silu")
        with pytest.raises(TypeError, match="save_gates"):
            nso.gated_mlp(x, w, w, save_gates=bad)
    f = torch.zeros(6, 8), torch.zeros(10, 8), torch.zeros(6, 10)
    with pytest.raises(ValueError):
        lib.gated(f[0], f[1], f[1], f[2], torch.zeros(2, 6, 10, dtype=torch.bfloat16), "silu")
    with pytest.raises(TypeError, match="save_gates"):
        nso.gated_mlp(f[0], f[1], f[1], save_gates=torch.bfloat16)
