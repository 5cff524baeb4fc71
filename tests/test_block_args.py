"""Refusals of the parts of a transformer block (rotary positions, the norms
around a block, the gated feed-forward product), on a machine without a GPU: the C
entry points return a status before any HIP call, the Python calls raise. And the
frequencies of rotary positions, which the host computes."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import block_oracle as B

A = 0x7f0000000000   # never dereferenced
G = 1 << 30


@pytest.fixture(scope="module")
def lib():
    from newton_schulz_orthogonalized_amd import _lib
    return _lib


# ---------------------------------------------------------------------------
# rotary
# ---------------------------------------------------------------------------

def _rotary(lib, x=None, y=None, n=1, **kw):
    t = dict(x=A, out=A + G, x_stride_b=4096, x_stride_s=128, x_stride_h=32, out_stride_b=4096, out_stride_s=128, out_stride_h=32,
             heads=4, pad0=0)
    d = dict(freqs=A + 4 * G, positions=None, offset=0, batch=2, len=32, n=n, dim=32, part=32, position_bits=0, shared_positions=0,
             interleaved=0, inverse=0, dtype=lib.MU_BF16, scale=1.0, pad0=0)
    a = lib.MuRotaryArgs(**{**d, **kw})
    a.x[0] = lib.MuRotaryTensor(**{**t, **(x or {})})
    a.x[1] = lib.MuRotaryTensor(**{**t, "x": A + 2 * G, "out": A + 3 * G, **(y or {})})
    return lib.LIB.mu_rotary(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), 2), (dict(n=0), 1), (dict(n=3), 1), (dict(batch=-1), 1), (dict(len=-1), 1), (dict(batch=1 << 20, len=1 << 20), 1),
    (dict(dim=0), 1), (dict(dim=1025), 1), (dict(part=31), 1), (dict(part=34), 1), (dict(part=0), 1), (dict(interleaved=2), 1),
    (dict(inverse=-1), 1), (dict(shared_positions=3), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(offset=(1 << 52) + 1), 1), (dict(freqs=None), 1), (dict(freqs=A + 4 * G + 4), 3),
    (dict(positions=A + 5 * G, position_bits=16), 2), (dict(positions=A + 5 * G + 4, position_bits=64), 3),
    (dict(x=dict(heads=-1)), 1), (dict(x=dict(x=None)), 1), (dict(x=dict(out=None)), 1), (dict(x=dict(x=A + 1)), 3),
    (dict(x=dict(x_stride_s=-1)), 1), (dict(x=dict(x_stride_b=1 << 60)), 1),
    (dict(x=dict(out=A + 64)), 3),                                # overlaps the input, and is not it
    (dict(x=dict(out=A, out_stride_h=64)), 3),                    # the same address with other strides
    (dict(x=dict(out_stride_h=0)), 3), (dict(x=dict(out_stride_s=64)), 3),   # rows of the output on one another
    (dict(freqs=A + G + 64), 3), (dict(positions=A + G, position_bits=32), 3),
    (dict(n=2, y=dict(out=A + G + 8)), 3), (dict(n=2, y=dict(out=A)), 3),
])
def test_bad_rotary_rejected(lib, kw, code):
    assert _rotary(lib, **kw) == code
    assert lib.mu_last_error() != ""


def test_null_rotary_rejected(lib):
    assert lib.LIB.mu_rotary(None, None) == lib.MU_ERR_INVALID_ARG


def test_empty_rotary_is_nothing(lib):
    for kw in (dict(batch=0), dict(len=0), dict(x=dict(heads=0))):
        assert _rotary(lib, **kw) == lib.MU_OK
    assert _rotary(lib, batch=0, x=dict(x=None, out=None)) == lib.MU_OK


def _cpu(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def test_python_rotary_refusals(lib):
    import newton_schulz_orthogonalized_amd as nso
    f = nso.rotary_frequencies(16, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        nso.rotary(_cpu(1, 2, 3, 16), freqs=f)

    def args(xs, outs=None, freqs=f, positions=None):
        return lib.rotary_args(xs, outs or [torch.empty_like(x) for x in xs], freqs, positions, 0, False, False, 1.0)
    q = _cpu(2, 5, 4, 16)
    a = args((q, _cpu(2, 5, 1, 16)))
    assert (a.n, a.batch, a.len, a.dim, a.part, a.x[0].heads, a.x[1].heads) == (2, 2, 5, 16, 16, 4, 1)
    assert args((_cpu(7, 4, 16),)).batch == 1 and args((q,), positions=torch.zeros(5, dtype=torch.int32)).shared_positions == 1
    assert args((q,), positions=torch.zeros(2, 5, dtype=torch.int64)).shared_positions == 0
    for xs in ((_cpu(2, 16),), (_cpu(1, 2, 3, 4, 16),), (q, _cpu(2, 6, 4, 16)), (q, _cpu(2, 5, 4, 8)), (q.transpose(2, 3),)):
        with pytest.raises(ValueError):
            args(xs)
    with pytest.raises(TypeError):
        args((q, _cpu(2, 5, 4, 16, dtype=torch.bfloat16)))
    with pytest.raises(TypeError):
        args((q.half(),))
    with pytest.raises(TypeError, match="float64"):
        args((q,), freqs=f.float())
    with pytest.raises(ValueError):
        args((q,), outs=[_cpu(2, 5, 4, 8)])
    for p in (torch.zeros(2, dtype=torch.int32), torch.zeros(5, 2, dtype=torch.int32)):
        with pytest.raises(ValueError):
            args((q,), positions=p)
    with pytest.raises(TypeError):
        args((q,), positions=torch.zeros(5))
    with pytest.raises(ValueError, match="out"):
        nso.rotary(q, q, freqs=f, out=q)
    with pytest.raises(ValueError, match="no_grad"):
        nso.rotary(q.clone().requires_grad_(), freqs=f, out=q)


def test_frequencies():
    import newton_schulz_orthogonalized_amd as nso
    for kw in (dict(), dict(base=500000.0, factor=8.0), dict(factor=8.0, original_length=8192, high=4.0),
               dict(factor=40.0, original_length=4096, low=1.0, high=32.0)):
        for part in (2, 64, 130):
            got = nso.rotary_frequencies(part, device="cpu", **kw)
            assert got.dtype == torch.float64 and np.allclose(got.numpy(), B.frequencies_ref(part, **kw), rtol=1e-13, atol=0)
    f = nso.rotary_frequencies(128, device="cpu", factor=8.0, original_length=8192, high=4.0)
    plain = nso.rotary_frequencies(128, device="cpu")
    assert f[0] == plain[0] and abs(f[-1] * 8 / plain[-1] - 1) < 1e-15      # many turns: kept; few: slowed down
    for kw in (dict(part=3), dict(part=0), dict(part=4, base=0.0), dict(part=4, factor=-1.0), dict(part=4, factor=math.inf),
               dict(part=4, original_length=0), dict(part=4, original_length=10, low=4.0, high=4.0)):
        with pytest.raises(ValueError):
            nso.rotary_frequencies(device="cpu", **kw)


# ---------------------------------------------------------------------------
# residual_norm
# ---------------------------------------------------------------------------

def _resnorm(lib, **kw):
    d = dict(residual=A, update=A + G, gate=None, post_weight=None, pre_weight=A + 4 * G, new_residual=A + 2 * G, normed=A + 3 * G,
             rows=12, dim=64, groups=1, residual_dtype=lib.MU_BF16, dtype=lib.MU_BF16, weight_dtype=lib.MU_F32, post_norm=0,
             residual_scale=1.0, eps=1e-6)
    return lib.MuResnorm(**{**d, **kw})


BAD_NORMS = [
    (dict(residual_dtype=5), 2), (dict(dtype=5), 2), (dict(weight_dtype=5), 2), (dict(dtype=0), 2), (dict(dim=0), 1), (dict(dim=16385), 1),
    (dict(rows=-1), 1), (dict(groups=0, gate=A + 5 * G), 1), (dict(groups=5, gate=A + 5 * G), 1), (dict(groups=2), 1), (dict(post_norm=2), 1),
    (dict(residual_scale=float("inf")), 1), (dict(eps=0.0), 1), (dict(eps=float("nan")), 1), (dict(eps=-1.0), 1),
    (dict(post_weight=A + 5 * G), 1),
]


@pytest.mark.parametrize("kw,code", BAD_NORMS + [
    (dict(residual=None), 1), (dict(normed=None), 1), (dict(new_residual=None), 1), (dict(update=None), 1),
    (dict(update=None, new_residual=None, post_norm=1), 1), (dict(update=None, new_residual=None, gate=A + 5 * G), 1),
    (dict(residual=A + 1), 3), (dict(pre_weight=A + 4 * G + 2), 3), (dict(normed=A + 3 * G + 1), 3),
    (dict(new_residual=A + 2), 3), (dict(normed=A + G + 4), 3), (dict(normed=A + 2 * G), 3), (dict(normed=A + 4 * G), 3),
    (dict(residual_dtype=0, normed=A), 3),                        # the residual's buffer as another type
])
def test_bad_residual_norm_rejected(lib, kw, code):
    assert lib.LIB.mu_residual_norm(ctypes.byref(_resnorm(lib, **kw)), None) == code
    assert lib.mu_last_error() != ""


def test_empty_residual_norm_is_nothing(lib):
    a = _resnorm(lib, rows=0, residual=None, update=None, new_residual=None, normed=None, gate=A, groups=3)
    assert lib.LIB.mu_residual_norm(ctypes.byref(a), None) == lib.MU_OK
    assert lib.LIB.mu_residual_norm(None, None) == lib.MU_ERR_INVALID_ARG


def _resnorm_grad(lib, fwd=None, **kw):
    d = dict(grad_residual=A + 6 * G, grad_normed=A + 7 * G, d_residual=A + 8 * G, d_update=A + 9 * G, d_gate=None, d_post=None,
             d_pre=A + 10 * G)
    f = _resnorm(lib, residual=None, normed=None, **(fwd or {}))
    return lib.MuResnormGrad(fwd=f, **{**d, **kw})


@pytest.mark.parametrize("kw,code", [(dict(fwd=f), c) for f, c in BAD_NORMS] + [
    (dict(d_gate=A + 11 * G), 1), (dict(d_post=A + 11 * G), 1), (dict(fwd=dict(pre_weight=None)), 1),
    (dict(fwd=dict(new_residual=None)), 1), (dict(fwd=dict(update=None)), 1),
    (dict(grad_normed=A + 7 * G + 1), 3), (dict(d_residual=A + 8 * G + 1), 3), (dict(d_pre=A + 10 * G + 2), 3),
    (dict(d_residual=A + 6 * G), 3), (dict(d_update=A + 8 * G), 3), (dict(d_pre=A + 4 * G), 3), (dict(d_residual=A + 2 * G), 3),
])
def test_bad_residual_norm_gradient_rejected(lib, kw, code):
    a = _resnorm_grad(lib, **kw)
    need = ctypes.c_size_t(0)
    assert lib.LIB.mu_residual_norm_grad(ctypes.byref(a), A + 20 * G, 1 << 30, None) == code
    assert lib.LIB.mu_residual_norm_grad_workspace_size(ctypes.byref(a), ctypes.byref(need)) == code


def test_residual_norm_gradient_workspace(lib):
    a, need = _resnorm_grad(lib), ctypes.c_size_t(0)
    fn = lib.LIB.mu_residual_norm_grad
    assert lib.LIB.mu_residual_norm_grad_workspace_size(ctypes.byref(a), ctypes.byref(need)) == 0 and need.value > 0
    assert lib.LIB.mu_residual_norm_grad_workspace_size(ctypes.byref(a), None) == lib.MU_ERR_INVALID_ARG
    for ws, nb in ((None, need.value), (A + 20 * G + 8, need.value), (A + 20 * G, need.value - 1)):
        assert fn(ctypes.byref(a), ws, nb, None) == lib.MU_ERR_WORKSPACE
    assert fn(None, None, 0, None) == lib.MU_ERR_INVALID_ARG


def test_python_residual_norm_refusals(lib):
    import newton_schulz_orthogonalized_amd as nso
    r, w = _cpu(6, 8), _cpu(8)
    with pytest.raises(ValueError, match="GPU"):
        nso.residual_norm(r, r)
    with pytest.raises(TypeError, match="rms_norm"):
        nso.residual_norm(r, None)

    def args(r=r, y=r, gate=None, post=None, pre=None, new=r, n=r):
        return lib.resnorm(r, y, gate, post, pre, new, n, False, 1.0, 1e-6)
    assert args(gate=_cpu(3, 8)).groups == 3 and args(gate=w).groups == 1
    for kw in (dict(y=_cpu(5, 8)), dict(pre=_cpu(7)), dict(post=_cpu(1, 8)), dict(gate=_cpu(3, 7)), dict(gate=_cpu(1, 3, 8)),
               dict(r=_cpu(8, 6).t()), dict(n=_cpu(6, 9))):
        with pytest.raises(ValueError):
            args(**kw)
    for kw in (dict(pre=w, post=w.bfloat16()), dict(n=r.bfloat16()), dict(new=r.bfloat16()), dict(pre=w.double()), dict(r=r.half(), new=None)):
        with pytest.raises(TypeError):
            args(**kw)
    with pytest.raises(ValueError, match="no_grad"):
        nso.residual_norm(r.clone().requires_grad_(), r, out=r)
    with pytest.raises(TypeError, match="dtype"):
        nso.rms_norm(r, out=r, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        lib.resnorm_grad(r.bfloat16(), r, r, r, None, None, None, False, 1.0, 1e-6, (None,) * 5)
    with pytest.raises(ValueError):
        lib.resnorm_grad(r, r[:5], r, r, None, None, None, False, 1.0, 1e-6, (None,) * 5)


# ---------------------------------------------------------------------------
# gated_mlp
# ---------------------------------------------------------------------------

def _gated(lib, **kw):
    d = dict(x=A, w_gate=A + G, w_up=A + 2 * G, h=A + 3 * G, gate_out=None, up_out=None, tokens=20, dim=64, hidden=96,
             dtype=lib.MU_BF16, activation=0)
    return lib.MuGated(**{**d, **kw})


BAD_SIZES = [(dict(dtype=9), 2), (dict(tokens=-1), 1), (dict(tokens=1 << 31), 1), (dict(dim=0), 1), (dict(hidden=0), 1),
             (dict(dim=(1 << 20) + 1), 1), (dict(hidden=(1 << 20) + 1), 1), (dict(activation=4), 1), (dict(activation=-1), 1)]


@pytest.mark.parametrize("kw,code", BAD_SIZES + [
    (dict(x=None), 1), (dict(w_gate=None), 1), (dict(w_up=None), 1), (dict(h=None), 1), (dict(gate_out=A + 4 * G), 1), (dict(up_out=A + 4 * G), 1),
    (dict(x=A + 1), 3), (dict(h=A + 3 * G + 1), 3), (dict(h=A + 64), 3), (dict(gate_out=A + 3 * G + 64, up_out=A + 5 * G), 3),
    (dict(gate_out=A + 4 * G, up_out=A + 4 * G), 3),
])
def test_bad_gated_rejected(lib, kw, code):
    a, need = _gated(lib, **kw), ctypes.c_size_t(0)
    assert lib.LIB.mu_gated_mlp(ctypes.byref(a), A + 20 * G, 1 << 30, None) == code
    assert lib.LIB.mu_gated_mlp_workspace_size(ctypes.byref(a), ctypes.byref(need)) == code


def test_gated_workspace(lib):
    need = ctypes.c_size_t(0)
    odd = _gated(lib, dim=63)
    assert lib.LIB.mu_gated_mlp_workspace_size(ctypes.byref(odd), ctypes.byref(need)) == 0 and need.value >= (20 + 2 * 96) * 64 * 2
    assert lib.LIB.mu_gated_mlp_workspace_size(ctypes.byref(odd), None) == lib.MU_ERR_INVALID_ARG
    for ws, nb in ((None, need.value), (A + 20 * G + 8, need.value), (A + 20 * G, need.value - 1)):
        assert lib.LIB.mu_gated_mlp(ctypes.byref(odd), ws, nb, None) == lib.MU_ERR_WORKSPACE
    assert lib.LIB.mu_gated_mlp(None, None, 0, None) == lib.MU_ERR_INVALID_ARG
    empty = _gated(lib, tokens=0, x=None, h=None)
    assert lib.LIB.mu_gated_mlp(ctypes.byref(empty), None, 0, None) == lib.MU_OK


def _gated_grad(lib, **kw):
    d = dict(grad_h=A, x=A + G, w_gate=A + 2 * G, w_up=A + 3 * G, gate=None, up=None, dx=A + 4 * G, d_gate=A + 5 * G, d_up=A + 6 * G,
             tokens=20, dim=64, hidden=96, dtype=lib.MU_BF16, grad_dtype=lib.MU_F32, accumulate=0, activation=0)
    return lib.MuGatedGrad(**{**d, **kw})


@pytest.mark.parametrize("kw,code", BAD_SIZES + [
    (dict(grad_dtype=5), 2), (dict(dtype=0, grad_dtype=1), 2), (dict(accumulate=2), 1), (dict(d_up=None), 1), (dict(d_gate=None), 1),
    (dict(gate=A + 7 * G), 1), (dict(grad_h=None), 1), (dict(x=None), 1), (dict(w_up=None), 1), (dict(d_gate=A + 5 * G + 2), 3),
    (dict(dx=A + 64), 3), (dict(d_up=A + 5 * G + 64), 3), (dict(dx=A + G), 3), (dict(gate=A + 7 * G, up=A + 4 * G), 3),
])
def test_bad_gated_gradient_rejected(lib, kw, code):
    a, need = _gated_grad(lib, **kw), ctypes.c_size_t(0)
    assert lib.LIB.mu_gated_mlp_grad(ctypes.byref(a), A + 20 * G, 1 << 30, None) == code
    assert lib.LIB.mu_gated_mlp_grad_workspace_size(ctypes.byref(a), ctypes.byref(need)) == code


def test_gated_gradient_workspace(lib):
    a, need = _gated_grad(lib), ctypes.c_size_t(0)
    assert lib.LIB.mu_gated_mlp_grad_workspace_size(ctypes.byref(a), ctypes.byref(need)) == 0 and need.value >= 2 * 20 * 96 * 2
    for ws, nb in ((None, need.value), (A + 20 * G + 8, need.value), (A + 20 * G, need.value - 1)):
        assert lib.LIB.mu_gated_mlp_grad(ctypes.byref(a), ws, nb, None) == lib.MU_ERR_WORKSPACE
    nothing = _gated_grad(lib, dx=None, d_gate=None, d_up=None)
    assert lib.LIB.mu_gated_mlp_grad(ctypes.byref(nothing), None, 0, None) == lib.MU_OK


def test_python_gated_refusals(lib):
    import newton_schulz_orthogonalized_amd as nso
    x, w = _cpu(3, 4, 8), _cpu(10, 8)
    with pytest.raises(ValueError, match="GPU"):
        nso.gated_mlp(x, w, w)

    def args(x=x, wg=w, wu=w, h=_cpu(3, 4, 10), gates=None, act="silu"):
        return lib.gated(x, wg, wu, h, gates, act)
    assert (args().tokens, args().dim, args().hidden) == (12, 8, 10)
    for kw in (dict(x=_cpu(3, 7)), dict(wu=_cpu(9, 8)), dict(wg=_cpu(8)), dict(wg=_cpu(8, 10).t()), dict(h=_cpu(3, 4, 9)),
               dict(gates=_cpu(3, 4, 10)), dict(act="swish"), dict(h=_cpu(12, 10)), dict(h=_cpu(3, 4, 10, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            args(**kw)
    with pytest.raises(TypeError):
        args(wu=w.bfloat16())
    with pytest.raises(TypeError):
        lib.gated(x.half(), w.half(), w.half(), _cpu(3, 4, 10).half(), None, "silu")
    with pytest.raises(ValueError, match="no_grad"):
        nso.gated_mlp(x.clone().requires_grad_(), w, w, out=_cpu(3, 4, 10))
    g = _cpu(3, 4, 10)
    for kw in (dict(d_gate=w), dict(accumulate=True), dict(d_gate=w, d_up=w, need_weights=False)):
        with pytest.raises(ValueError):
            nso.gated_mlp_grad(g, x, w, w, **kw)
    with pytest.raises(TypeError):
        nso.gated_mlp_grad(g, x, w, w, d_gate=w, d_up=w, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lib.gated_grad(_cpu(3, 4, 9), x, w, w, None, None, None, None, False, "silu")
    with pytest.raises(TypeError):
        lib.gated_grad(g, x, w, w, None, None, w, w.bfloat16(), False, "silu")


def test_forward_mode_is_refused():
    import newton_schulz_orthogonalized_amd as nso
    x = _cpu(2, 2, 1, 8)
    with torch.autograd.forward_ad.dual_level():
        d = torch.autograd.forward_ad.make_dual(x, x)
        flat = torch.autograd.forward_ad.make_dual(_cpu(2, 8), _cpu(2, 8))
        for call in (lambda: nso.rotary(d, freqs=nso.rotary_frequencies(8, device="cpu")), lambda: nso.residual_norm(flat, _cpu(2, 8)),
                     lambda: nso.rms_norm(flat), lambda: nso.gated_mlp(flat, _cpu(3, 8), _cpu(3, 8))):
            with pytest.raises(NotImplementedError):
                call()


# ---------------------------------------------------------------------------
# the reference itself
# ---------------------------------------------------------------------------

def test_reference_gradients_against_differences():
    """The reference's formulas against central differences of its own forward
    functions, in float64 (step 1e-6: 1e-9 of the terms)."""
    rng = np.random.default_rng(7)
    r, y, gate, post, pre = (rng.normal(size=s) for s in ((6, 9), (6, 9), (3, 9), (9,), (9,)))
    dr, dn = rng.normal(size=(6, 9)), rng.normal(size=(6, 9))

    def loss(ts, post_norm=True):
        new, n, _ = B.residual_norm_ref(ts[0], ts[1], ts[2], post_norm, ts[3] if post_norm else None, ts[4], 0.7, 1e-3)
        return (new * dr + n * dn).sum()
    for post_norm in (True, False):
        ts = [r, y, gate, post, pre]
        new, _, _ = B.residual_norm_ref(r, y, gate, post_norm, post if post_norm else None, pre, 0.7, 1e-3)
        g = B.residual_norm_grad_ref(dr, dn, new, y, gate, post_norm, post if post_norm else None, pre, 0.7, 1e-3)
        for i, name in enumerate(("r", "y", "gate", "post", "pre")):
            if name == "post" and not post_norm:
                continue
            e = rng.normal(size=ts[i].shape)
            up, dn_ = ([t + s * 1e-6 * e if j == i else t for j, t in enumerate(ts)] for s in (1, -1))
            num = (loss(up, post_norm) - loss(dn_, post_norm)) / 2e-6
            assert abs(num - (g[name][0] * e).sum()) < 1e-6, name
    x, wg, wu, dh = (rng.normal(size=s) for s in ((5, 7), (4, 7), (4, 7), (5, 4)))
    for act in ("silu", "gelu", "gelu_tanh", "relu"):
        _, g, u, _, _ = B.gated_mlp_ref(x, wg, wu, act)
        grads = B.gated_mlp_grad_ref(dh, x, wg, wu, g, u, act)[:3]
        for i in range(3):
            e = rng.normal(size=(x, wg, wu)[i].shape)
            vals = [(B.gated_mlp_ref(*[t + s * 1e-6 * e if j == i else t for j, t in enumerate((x, wg, wu))], act)[0] * dh).sum() for s in (1, -1)]
            assert abs((vals[0] - vals[1]) / 2e-6 - (grads[i] * e).sum()) < 1e-6, act


def test_reference_rotary_is_a_rotation():
    """Turning back undoes a turn; norms of pairs stay; dot products depend on the
    difference of positions; a quarter turn by hand."""
    rng = np.random.default_rng(8)
    x, y = rng.normal(size=(1, 1, 1, 10)), rng.normal(size=(1, 1, 1, 10))
    f = B.frequencies_ref(8)
    for inter in (False, True):
        def at(v, p):
            return B.rotary_ref(v, np.array([[p]]), f, inter)[0]
        back = B.rotary_ref(at(x, 5), np.array([[5]]), f, inter, inverse=True)[0]
        assert np.allclose(back, x, atol=1e-14)
        assert abs((at(x, 9) * at(y, 4)).sum() - (at(x, 1005) * at(y, 1000)).sum()) < 1e-12
    quarter = B.rotary_ref(np.array([[[[1.0, 2.0, 3.0]]]]), np.array([[1]]), np.array([math.pi / 2]))[0]
    assert np.allclose(quarter, [-2.0, 1.0, 3.0])
