"""The activations behind the gated product's large tiles (256 and 128), forward,
gradients from saved gates and from gates computed again, against float64 products
on the GPU; and rows of NaN there.

Inputs, formulas and tolerances are those of test_gpu_gated.py's normal inputs: U =
2^-24, a product over K off by 2 K U of the product of magnitudes, an activation by
its argument's error and 4 (Z + 8) U of itself or, the slope, of 1 + |g|, dg and du
rounded to the type before their products, every result once. With a gradient of h
that has a few entries in each row and column, each sum has a few terms and shows
each of them.
"""

import math

import pytest
import torch

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32
ULP = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    import newton_schulz_orthogonalized_amd  # noqa: F401  (fails loudly without the library)
    yield
    torch.cuda.empty_cache()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, seed, dtype, std=1.0):
    return torch.randn(shape, generator=_gen(seed), device="cuda", dtype=torch.float64).mul_(std).to(dtype)


def _half(dtype):
    return 2.0 ** -8 if dtype == BF else ULP


def _within(got, ref, tol, dtype, what):
    bad = ~((got.double() - ref).abs() <= tol + _half(dtype) * (ref.abs() + tol))
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), ref[bad][:4].tolist())


def _activation(g, kind):
    """(act(g), act'(g), argument of the exponential in it), float64."""
    if kind == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s + g * s * (1 - s), g.abs()
    if kind == "gelu":
        phi = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi), g * g
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        z = c * (g + 0.044715 * g ** 3)
        t = torch.tanh(z)
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g), 8 * z.abs()
    return g.clamp(min=0), (g > 0).double(), torch.zeros_like(g)


# type, tokens, dim, hidden. Tiles of 256: results of whole and of ragged runs, a last row by itself; of 128: the same;
# float32 (tiles of 128), whole and ragged
SHAPES = [(BF, 4096, 128, 2048), (BF, 4100, 64, 1999), (BF, 8193, 264, 2056), (BF, 1030, 130, 4100),
          (BF, 1000, 768, 2048), (BF, 1001, 200, 2050), (FP, 1024, 96, 2048), (FP, 1027, 101, 2053)]


def _inputs(dtype, t, d, f):
    return (_normal((t, d), 98000 + t, dtype), _normal((f, d), 98001, dtype, 2 * d ** -0.5), _normal((f, d), 98002, dtype, d ** -0.5))


def _few(dh, seed):
    """dh with two entries of each row and two of each column kept, or more by chance."""
    t, f = dh.shape
    keep = torch.zeros_like(dh, dtype=torch.bool)
    rows, cols = torch.arange(t, device="cuda"), torch.arange(f, device="cuda")
    for i in range(2):
        keep[rows, torch.randint(f, (t,), generator=_gen(seed + i), device="cuda")] = True
        keep[torch.randint(t, (f,), generator=_gen(seed + 2 + i), device="cuda"), cols] = True
    return torch.where(keep, dh, torch.zeros_like(dh))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("dtype,t,d,f", SHAPES)
def test_activations(dtype, t, d, f, act):
    import newton_schulz_orthogonalized_amd as nso
    x, wg, wu = _inputs(dtype, t, d, f)
    X, G, U = x.double(), wg.double(), wu.double()
    ax, ag, au = X.abs(), G.abs(), U.abs()
    g, u = X @ G.t(), X @ U.t()
    eg, eu = 2 * d * ULP * (ax @ ag.t()), 2 * d * ULP * (ax @ au.t())
    a, slope, z = _activation(g, act)

    gates = torch.full((2, t, f), 7.0, dtype=dtype, device="cuda")
    h = nso.gated_mlp(x, wg, wu, activation=act, gates_out=gates)
    _within(gates[0], g, eg, dtype, "g")
    _within(gates[1], u, eu, dtype, "u")
    ea = 1.13 * eg + 4 * (z + 8) * ULP * (a.abs() + ULP)
    _within(h, a * u, ea * (u.abs() + eu) + a.abs() * eu + 2 * ULP * (a * u).abs(), dtype, "h")
    assert torch.equal(nso.gated_mlp(x, wg, wu, activation=act), h)

    half = _half(dtype)
    sg, su = gates[0].double(), gates[1].double()
    sa, ss, sz = _activation(sg, act)
    jump = (g.abs() <= eg).double() if act == "relu" else 1.2 * eg      # a step at 0, or a bounded second derivative
    dense = _normal((t, f), 98003, dtype, 0.1)
    for few in (True, False):
        dh = _few(dense, 98010) if few else dense
        D = dh.double()
        # the formula's dg and du, and how far off they are: from the saved gates, and from unrounded ones
        forms = [(gates, D * su * ss, D * sa,
                  (D * su).abs() * (4 * (sz + 8) * ULP * (1 + sg.abs())), D.abs() * 4 * (sz + 8) * ULP * (sa.abs() + ULP)),
                 (None, D * u * slope, D * a,
                  D.abs() * ((4 * (z + 8) * ULP * (1 + g.abs()) + jump) * (u.abs() + eu) + slope.abs() * eu),
                  D.abs() * (1.13 * eg + 4 * (z + 8) * ULP * (a.abs() + ULP)))]
        for saved, dg, du, edg, edu in forms:
            edg, edu = edg + (half + 3 * ULP) * dg.abs(), edu + (half + 2 * ULP) * du.abs()
            res = nso.gated_mlp_grad(dh, x, wg, wu, saved, activation=act, dtype=FP)
            what = ("few" if few else "all", "saved" if saved is not None else "again")
            mdx = dg.abs() @ ag + du.abs() @ au
            _within(res[0], dg @ G + du @ U, 1.02 * (edg @ ag + edu @ au) + 4 * f * ULP * mdx, dtype, ("dx", what))
            _within(res[1], dg.t() @ X, 1.02 * edg.t() @ ax + 2 * t * ULP * dg.abs().t() @ ax, FP, ("d_gate", what))
            _within(res[2], du.t() @ X, 1.02 * edu.t() @ ax + 2 * t * ULP * du.abs().t() @ ax, FP, ("d_up", what))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("dtype,t,d,f", [SHAPES[1], SHAPES[2], SHAPES[4], SHAPES[7]])
def test_nan_and_infinity_stay_in_their_rows(dtype, t, d, f, act):
    """Of x, in the first, an inner and the last row; of the weights, in one hidden column."""
    import newton_schulz_orthogonalized_amd as nso
    x, wg, wu = _inputs(dtype, t, d, f)
    dh = _normal((t, f), 98020, dtype, 0.1)
    clean = nso.gated_mlp(x, wg, wu, activation=act)
    clean_dx = nso.gated_mlp_grad(dh, x, wg, wu, activation=act, need_weights=False)[0]
    assert bool(clean.isfinite().all()) and bool(clean_dx.isfinite().all())
    y = x.clone()
    y[0, 3], y[t // 2, d - 1], y[t - 1, 0] = float("nan"), float("inf"), float("nan")
    rows = torch.ones(t, dtype=torch.bool, device="cuda")
    rows[[0, t // 2, t - 1]] = False
    gates = torch.empty((2, t, f), dtype=dtype, device="cuda")
    h = nso.gated_mlp(y, wg, wu, activation=act, gates_out=gates)
    assert torch.equal(h[rows], clean[rows])
    assert bool(h[0].isnan().all()) and bool(h[t - 1].isnan().all()) and not bool(h[t // 2].isfinite().any())
    saved_dx = None
    for saved in (gates, None):
        dx = nso.gated_mlp_grad(dh, y, wg, wu, saved, activation=act, need_weights=False)[0]
        if saved is None:
            assert torch.equal(dx[rows], clean_dx[rows])
        else:
            saved_dx = dx
        assert bool(dx[rows].isfinite().all()) and bool(dx[0].isnan().all()) and bool(dx[t - 1].isnan().all())
    nso.gated_mlp(x, wg, wu, activation=act, gates_out=gates)
    assert torch.equal(nso.gated_mlp_grad(dh, x, wg, wu, gates, activation=act, need_weights=False)[0][rows], saved_dx[rows])
    v = wu.clone()
    v[f - 1, 2] = float("nan")
    h = nso.gated_mlp(x, wg, v, activation=act)
    assert torch.equal(h[:, :f - 1], clean[:, :f - 1]) and bool(h[:, f - 1].isnan().all())
