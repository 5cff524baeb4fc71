"""What the gated product keeps for its gradient: both products unrounded (float32)
unless the caller chooses otherwise.

Tolerances as in test_gpu_gated_tiles.py, whose helpers these are: with unrounded
gates the gradients differ from the formula by the products' float32 sums, the
rounding of dg and du to the type and that of the results alone.
"""

import pytest
import torch

from gpu_util import need_gpu
from test_gpu_gated_tiles import BF, FP, ULP, _activation, _few, _half, _inputs, _normal, _within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    import newton_schulz_orthogonalized_amd  # noqa: F401  (fails loudly without the library)
    yield
    torch.cuda.empty_cache()


# tiles of 64, of 128 and of 256; whole and ragged
SHAPES = [(BF, 70, 96, 130), (BF, 64, 64, 128), (BF, 1000, 768, 2048), (BF, 1001, 200, 2050), (BF, 4096, 128, 2048), (BF, 4100, 64, 1999),
          (FP, 130, 70, 100)]


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("dtype,t,d,f", SHAPES)
def test_gradients_through_autograd(dtype, t, d, f, act):
    """No gate is rounded on its way to the gradient."""
    import newton_schulz_orthogonalized_amd as nso
    x, wg, wu = (v.requires_grad_() for v in _inputs(dtype, t, d, f))
    X, G, U = x.detach().double(), wg.detach().double(), wu.detach().double()
    ax, ag, au = X.abs(), G.abs(), U.abs()
    g, u = X @ G.t(), X @ U.t()
    eg, eu = 2 * d * ULP * (ax @ ag.t()), 2 * d * ULP * (ax @ au.t())
    a, slope, z = _activation(g, act)
    jump = (g.abs() <= eg).double() if act == "relu" else 1.2 * eg      # a step at 0, or a bounded second derivative
    h = nso.gated_mlp(x, wg, wu, activation=act)
    half = _half(dtype)
    dense = _normal((t, f), 99000, dtype, 0.1)
    for dh in (_few(dense, 99001), dense):
        D = dh.double()
        dg, du = D * u * slope, D * a
        edg = D.abs() * ((4 * (z + 8) * ULP * (1 + g.abs()) + jump) * (u.abs() + eu) + slope.abs() * eu) + (half + 3 * ULP) * dg.abs()
        edu = D.abs() * (1.13 * eg + 4 * (z + 8) * ULP * (a.abs() + ULP)) + (half + 2 * ULP) * du.abs()
        dx, d_gate, d_up = torch.autograd.grad(h, (x, wg, wu), dh, retain_graph=True)
        mdx = dg.abs() @ ag + du.abs() @ au
        _within(dx, dg @ G + du @ U, 1.02 * (edg @ ag + edu @ au) + 4 * f * ULP * mdx, dtype, "dx")
        _within(d_gate, dg.t() @ X, 1.02 * edg.t() @ ax + 2 * t * ULP * dg.abs().t() @ ax, dtype, "d_gate")
        _within(d_up, du.t() @ X, 1.02 * edu.t() @ ax + 2 * t * ULP * du.abs().t() @ ax, dtype, "d_up")


@pytest.mark.parametrize("t,d,f", [(1, 1, 1), (3, 72, 65), (70, 96, 130), (200, 64, 257), (1000, 768, 2048), (1001, 200, 2050), (4096, 128, 2048),
                                   (4100, 64, 1999), (8193, 264, 2056), (700, 1032, 16385)])
def test_float32_gates_are_the_products(t, d, f):
    """Integers: sums far past what bfloat16 holds, each exact; the result as without
    gates; and with small sums the gradients of bfloat16 gates."""
    import newton_schulz_orthogonalized_amd as nso

    def ints(shape, seed, top, keep=1.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        v = torch.randint(-top, top + 1, shape, generator=g, device="cuda").double()
        return (v * (torch.rand(shape, generator=g, device="cuda") < keep)).to(BF)
    x, wg, wu = ints((t, d), 99100, 100), ints((f, d), 99101, 100), ints((f, d), 99102, 100)
    gates = torch.full((2, t, f), 7.0, device="cuda")
    h = nso.gated_mlp(x, wg, wu, activation="relu", gates_out=gates)
    assert torch.equal(gates[0].double(), x.double() @ wg.double().t()) and torch.equal(gates[1].double(), x.double() @ wu.double().t())
    assert torch.equal(h, nso.gated_mlp(x, wg, wu, activation="relu"))
    keep = min(1.0, 10 / d)
    x, wg, wu, dh = ints((t, d), 99103, 2), ints((f, d), 99104, 2, keep), ints((f, d), 99105, 2, keep), ints((t, f), 99106, 1, 0.2)
    small = torch.full((2, t, f), 7.0, dtype=BF, device="cuda")
    nso.gated_mlp(x, wg, wu, activation="relu", gates_out=gates)
    nso.gated_mlp(x, wg, wu, activation="relu", gates_out=small)
    assert torch.equal(gates, small.float())
    for dtype in (BF, FP):
        got, want = (nso.gated_mlp_grad(dh, x, wg, wu, v, activation="relu", dtype=dtype) for v in (gates, small))
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("lead", [16, 3])
@pytest.mark.parametrize("t,d,f", [(1, 40, 33), (130, 136, 70), (1000, 768, 2048), (4100, 64, 1999), (4096, 128, 2048)])
def test_nothing_beside_the_gates_is_written(t, d, f, lead):
    """And nothing beside them is read: they are surrounded by NaN for the gradient."""
    import newton_schulz_orthogonalized_amd as nso
    x, wg, wu = _inputs(BF, t, d, f)
    dh = _normal((t, f), 99200, BF)
    want = torch.empty((2, t, f), device="cuda")
    nso.gated_mlp(x, wg, wu, gates_out=want)
    buf = torch.full((2 * t * f + lead + 40,), 7.0, device="cuda")
    gates = buf[lead:lead + 2 * t * f].view(2, t, f)
    h = nso.gated_mlp(x, wg, wu, gates_out=gates)
    assert torch.equal(gates, want) and torch.equal(h, nso.gated_mlp(x, wg, wu))
    assert bool((buf[:lead] == 7).all()) and bool((buf[lead + 2 * t * f:] == 7).all())
    buf[:lead] = float("nan")
    buf[lead + 2 * t * f:] = float("nan")
    got, dense = nso.gated_mlp_grad(dh, x, wg, wu, gates), nso.gated_mlp_grad(dh, x, wg, wu, want)
    assert all(torch.equal(a, b) and bool(a.isfinite().all()) for a, b in zip(got, dense))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("t,d,f", [(42, 48, 80), (1000, 768, 2048), (2500, 128, 4099)])
def test_what_autograd_keeps(t, d, f, dtype):
    """float32 gates unless asked for others; the functional calls give the same bits."""
    import newton_schulz_orthogonalized_amd as nso
    leaves = [v.requires_grad_() for v in _inputs(dtype, t, d, f)]
    dh = _normal((t, f), 99300, dtype)
    for kw, kept in (({}, FP), (dict(save_gates=FP), FP), (dict(save_gates=True), dtype), (dict(save_gates=dtype), dtype), (dict(save_gates=False), None)):
        saved = []
        with torch.autograd.graph.saved_tensors_hooks(lambda v: saved.append((v.dtype, v.numel())) or v, lambda v: v):
            h = nso.gated_mlp(*leaves, activation="gelu", **kw)
        assert [s for s in saved if s[1] == 2 * t * f] == ([] if kept is None else [(kept, 2 * t * f)])
        got = torch.autograd.grad(h, leaves, dh)
        with torch.no_grad():
            gates = None if kept is None else torch.empty((2, t, f), dtype=kept, device="cuda")
            assert torch.equal(nso.gated_mlp(*leaves, activation="gelu", gates_out=gates), h)
            want = nso.gated_mlp_grad(dh, *leaves, gates, activation="gelu")
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gates_of_more_than_2_31_elements():
    """Integers that bfloat16 holds: both types of gates hold the same values, at both
    ends and around the places where 31- and 32-bit offsets would turn over, and give
    the same gradients."""
    import newton_schulz_orthogonalized_amd as nso
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    t, d, f = 150001, 64, 14336
    g = torch.Generator(device="cuda")
    g.manual_seed(99400)

    def ints(shape, top, keep):
        v = torch.randint(-top, top + 1, shape, generator=g, device="cuda", dtype=torch.int8)
        return (v * (torch.rand(shape, generator=g, device="cuda") < keep)).to(BF)
    x, wg, wu, dh = ints((t, d), 2, 1.0), ints((f, d), 2, 0.15), ints((f, d), 2, 0.15), ints((t, f), 1, 0.05)
    gates = torch.empty((2, t, f), device="cuda")
    nso.gated_mlp(x, wg, wu, activation="relu", gates_out=gates)
    rows = torch.tensor(sorted({0, 1, t - 2, t - 1} | {e // f + i for e in (1 << 29, 1 << 30, 1 << 31) for i in (-1, 0, 1) if e // f + i < t}),
                        device="cuda")
    for v, w in zip(gates, (wg, wu)):
        assert torch.equal(v[rows].double(), x[rows].double() @ w.double().t())
    got = nso.gated_mlp_grad(dh, x, wg, wu, gates, activation="relu", dtype=FP)
    small = gates.to(BF)
    assert float(gates.abs().max()) <= 256
    del gates
    want = nso.gated_mlp_grad(dh, x, wg, wu, small, activation="relu", dtype=FP)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
