"""GPU parity of the gated feed-forward product and its gradients against a
float64 reference.

Two kinds of inputs. Small integers with the relu: every product, sum and factor
is exact in both types, so results must be equal (a float32 result) or the exact
value rounded once. Normal inputs, with tolerances in U = 2^-24: a matrix
product over K is off by at most 2 K U of the product of magnitudes; an activation
by its argument's error (slopes stay below 1.13, their own below 1.2) and by 4 (Z + 8) U of
itself or, the slope, of 1 + |g|, Z being its exponential's argument (hardware
exponential and reciprocal: 4 U each, the argument's rounding Z U). dg and du are
rounded to the type (half a step, 2^-8 of bfloat16) before their products, and
every result once.
"""

import numpy as np
import pytest
import torch

from gpu_util import need_gpu, to_np
from oracle import block_oracle as B
from oracle import muon_oracle as O
from workloads import as_dtype, host_normal

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32
ULP = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    import newton_schulz_orthogonalized_amd  # noqa: F401  (fails loudly without the library)
    yield


def _half(dtype):
    return 2.0 ** -8 if dtype == BF else ULP


def _normal(shape, seed, dtype, std=1.0):
    return as_dtype(host_normal(shape, seed, std), dtype).cuda()


def _ints(shape, seed, dtype, top, density=1.0):
    r = np.random.default_rng(seed)
    v = r.integers(-top, top + 1, shape) * (r.random(shape) < density)
    return torch.from_numpy(v.astype(np.float32)).to(dtype).cuda()


def _rounded(ref, dtype):
    return O.bf16_round(ref) if dtype == BF else ref


def _within(got, ref, tol, dtype, what):
    bad = ~(np.abs(to_np(got) - ref) <= tol + _half(dtype) * (np.abs(ref) + tol))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4], to_np(got)[bad][:4], ref[bad][:4])


# tokens, dim, hidden: single tokens, both sides of tiles and of slices of k, odd rows
SHAPES = [(1, 1, 1), (1, 64, 64), (1, 100, 513), (2, 8, 5), (3, 513, 130), (7, 72, 65), (16, 256, 128), (17, 128, 64), (33, 64, 200),
          (64, 1000, 96), (65, 96, 129), (100, 24, 1), (128, 128, 64), (129, 66, 300), (200, 320, 257), (257, 192, 100),
          (300, 130, 260), (515, 264, 520)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("t,d,f", SHAPES)
def test_integers_are_exact(t, d, f, dtype):
    import newton_schulz_orthogonalized_amd as nso
    keep = min(1.0, 12 / d)    # g and u stay below 256, sums below 2^24
    x, wg, wu = _ints((t, d), 94000 + t, dtype, 2), _ints((f, d), 94001 + d, dtype, 2, keep), _ints((f, d), 94002 + f, dtype, 2, keep)
    dh = _ints((t, f), 94003, dtype, 1)
    h, g, u, mg, mu = B.gated_mlp_ref(to_np(x), to_np(wg), to_np(wu), "relu")
    assert max(mg.max(), mu.max()) <= 256 and np.abs(h).max() < 2 ** 24
    gates = torch.full((2, t, f), 7.0, dtype=dtype, device="cuda")
    got = nso.gated_mlp(x, wg, wu, activation="relu", gates_out=gates)
    torch.cuda.synchronize()
    assert np.array_equal(to_np(gates[0]), g) and np.array_equal(to_np(gates[1]), u)
    assert np.array_equal(to_np(got), _rounded(h, dtype))
    assert torch.equal(nso.gated_mlp(x, wg, wu, activation="relu"), got)
    dx, d_gate, d_up, dg, du = B.gated_mlp_grad_ref(to_np(dh), to_np(x), to_np(wg), to_np(wu), g, u, "relu")
    assert max(np.abs(v).max() for v in (dx, d_gate, d_up)) < 2 ** 24
    for saved in (gates, None):
        for wt in {dtype, FP}:
            a, b, c = nso.gated_mlp_grad(dh, x, wg, wu, saved, activation="relu", dtype=wt)
            torch.cuda.synchronize()
            assert np.array_equal(to_np(a), _rounded(dx, dtype))
            assert np.array_equal(to_np(b), _rounded(d_gate, wt)) and np.array_equal(to_np(c), _rounded(d_up, wt))
            # added to what is there
            nso.gated_mlp_grad(dh, x, wg, wu, saved, activation="relu", d_gate=b, d_up=c, accumulate=True, need_x=False)
            torch.cuda.synchronize()
            assert np.array_equal(to_np(b), _rounded(d_gate + _rounded(d_gate, wt), wt))
            assert np.array_equal(to_np(c), _rounded(d_up + _rounded(d_up, wt), wt))


# many tiles of each edge: whole and ragged, even and odd numbers of slices of k, several tiles for a workgroup; and few
# tiles over many tokens, whose weights' gradients are split
LARGE = [(4096, 192, 2048), (3900, 264, 2100), (4100, 64, 1999), (2050, 1000, 3500), (1030, 4096, 7000), (520, 2056, 14000),
         (1000, 768, 2048), (2050, 257, 1500), (90, 2048, 1000),
         (4100, 24, 16), (3000, 130, 70), (9000, 64, 128), (2049, 513, 200)]

# tiles of 256 whose last strip is a single row and whose last columns are half a tile or less: of the forward
# product and the gradient of x, of results narrower than half a tile, and of the weights' gradients
LARGE += [(8193, 264, 2056), (32769, 8, 24), (700, 1032, 16385)]


@pytest.mark.parametrize("dtype,wt", [(BF, BF), (BF, FP), (FP, FP)])
@pytest.mark.parametrize("t,d,f", LARGE)
def test_integers_are_exact_over_many_tiles(t, d, f, dtype, wt):
    """As above, against float64 products on the GPU, every element."""
    import newton_schulz_orthogonalized_amd as nso
    keep = min(1.0, 10 / d)
    x, wg, wu = _ints((t, d), 94050 + t, dtype, 2), _ints((f, d), 94051 + d, dtype, 2, keep), _ints((f, d), 94052 + f, dtype, 2, keep)
    dh = _ints((t, f), 94053, dtype, 1, 0.2)
    X, G, U, DH = (v.double() for v in (x, wg, wu, dh))
    g, u = X @ G.t(), X @ U.t()
    assert max(float((X.abs() @ W.abs().t()).max()) for W in (G, U)) <= 256
    gates = torch.full((2, t, f), 7.0, dtype=dtype, device="cuda")
    h = nso.gated_mlp(x, wg, wu, activation="relu", gates_out=gates)
    assert torch.equal(gates[0].double(), g) and torch.equal(gates[1].double(), u)
    assert torch.equal(h, (g.clamp(min=0) * u).to(dtype))
    assert torch.equal(nso.gated_mlp(x, wg, wu, activation="relu"), h)
    dg, du = DH * u * (g > 0), DH * g.clamp(min=0)
    want = [dg @ G + du @ U, dg.t() @ X, du.t() @ X]
    assert max(float(v.abs().max()) for v in want) < 2 ** 24
    for saved in (gates, None):
        got = nso.gated_mlp_grad(dh, x, wg, wu, saved, activation="relu", dtype=wt)
        assert torch.equal(got[0], want[0].to(dtype))
        assert torch.equal(got[1], want[1].to(wt)) and torch.equal(got[2], want[2].to(wt))
        nso.gated_mlp_grad(dh, x, wg, wu, saved, activation="relu", d_gate=got[1], d_up=got[2], accumulate=True, need_x=False)
        assert torch.equal(got[1], (want[1] + want[1].to(wt).double()).to(wt))
        assert torch.equal(got[2], (want[2] + want[2].to(wt).double()).to(wt))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("t,d,f", [(1, 96, 77), (5, 64, 64), (40, 130, 100), (150, 200, 190), (260, 64, 300)])
def test_normal_inputs(t, d, f, act, dtype):
    import newton_schulz_orthogonalized_amd as nso
    x, wg, wu = _normal((t, d), 94100 + t, dtype), _normal((f, d), 94101, dtype, 2 * d ** -0.5), _normal((f, d), 94102, dtype, d ** -0.5)
    dh = _normal((t, f), 94103, dtype, 0.1)
    gates = torch.empty(2, t, f, dtype=dtype, device="cuda")
    got = nso.gated_mlp(x, wg, wu, activation=act, gates_out=gates)
    torch.cuda.synchronize()
    h, g, u, mg, mu = B.gated_mlp_ref(to_np(x), to_np(wg), to_np(wu), act)
    eg, eu = 2 * d * ULP * mg, 2 * d * ULP * mu
    _within(gates[0], g, eg, dtype, "g")
    _within(gates[1], u, eu, dtype, "u")
    a, s, z = B.activation_ref(g, act)
    ea = 1.13 * eg + 4 * (z + 8) * ULP * (np.abs(a) + ULP)
    _within(got, h, (ea * (np.abs(u) + eu) + np.abs(a) * eu) + 2 * ULP * np.abs(h), dtype, "h")

    # the gradients, from the gates that were saved
    sg, su = to_np(gates[0]), to_np(gates[1])
    res = nso.gated_mlp_grad(dh, x, wg, wu, gates, activation=act, dtype=FP)
    torch.cuda.synchronize()
    dx, d_gate, d_up, dg, du = B.gated_mlp_grad_ref(to_np(dh), to_np(x), to_np(wg), to_np(wu), sg, su, act)
    a, s, z = B.activation_ref(sg, act)
    es = 4 * (z + 8) * ULP * (1 + np.abs(sg))
    half = _half(dtype)
    edg = np.abs(to_np(dh) * su) * es + (half + 3 * ULP) * np.abs(dg)
    edu = np.abs(to_np(dh)) * 4 * (z + 8) * ULP * (np.abs(a) + ULP) + (half + 2 * ULP) * np.abs(du)
    ax, ag, au = np.abs(to_np(x)), np.abs(to_np(wg)), np.abs(to_np(wu))
    mdx = np.abs(dg) @ ag + np.abs(du) @ au
    _within(res[0], dx, 1.01 * (edg @ ag + edu @ au) + 4 * f * ULP * mdx, dtype, "dx")
    _within(res[1], d_gate, 1.01 * edg.T @ ax + 2 * t * ULP * np.abs(dg).T @ ax, FP, "d_gate")
    _within(res[2], d_up, 1.01 * edu.T @ ax + 2 * t * ULP * np.abs(du).T @ ax, FP, "d_up")
    again = nso.gated_mlp_grad(dh, x, wg, wu, gates, activation=act, dtype=FP)
    assert all(torch.equal(p, q) for p, q in zip(res, again))

    # and from products computed again: the gates unrounded, so nearer the formula than their rounding
    res = nso.gated_mlp_grad(dh, x, wg, wu, None, activation=act, dtype=FP)
    torch.cuda.synchronize()
    dx, d_gate, d_up, dg, du = B.gated_mlp_grad_ref(to_np(dh), to_np(x), to_np(wg), to_np(wu), g, u, act)
    a, s, z = B.activation_ref(g, act)
    jump = (np.abs(g) <= eg).astype(float) if act == "relu" else 1.2 * eg      # a step at 0, or a bounded second derivative
    es = 4 * (z + 8) * ULP * (1 + np.abs(g)) + jump
    edg = np.abs(to_np(dh)) * (es * (np.abs(u) + eu) + np.abs(s) * eu) + (half + 3 * ULP) * np.abs(dg)
    edu = np.abs(to_np(dh)) * (1.13 * eg + 4 * (z + 8) * ULP * (np.abs(a) + ULP)) + (half + 2 * ULP) * np.abs(du)
    _within(res[0], dx, 1.02 * (edg @ ag + edu @ au) + 4 * f * ULP * mdx, dtype, "dx again")
    _within(res[1], d_gate, 1.02 * edg.T @ ax + 2 * t * ULP * np.abs(dg).T @ ax, FP, "d_gate again")
    _within(res[2], d_up, 1.02 * edu.T @ ax + 2 * t * ULP * np.abs(du).T @ ax, FP, "d_up again")


def _place(t, lead, fill=float("nan")):
    """t inside a buffer of `fill`, `lead` elements from its start."""
    buf = torch.full((t.numel() + lead + 40,), fill, dtype=t.dtype, device="cuda")
    v = buf[lead:lead + t.numel()].view(t.shape)
    v.copy_(t)
    return buf, v


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lead", [16, 3])
@pytest.mark.parametrize("t,d,f", [(1, 40, 33), (19, 72, 50), (130, 136, 70), (70, 50, 129)])
def test_nothing_beside_the_buffers_is_read_or_written(t, d, f, lead, dtype):
    """Operands surrounded by NaN, aligned and not; results surrounded by a mark."""
    import newton_schulz_orthogonalized_amd as nso
    ts = [_ints((t, d), 94200, dtype, 2), _ints((f, d), 94201, dtype, 1), _ints((f, d), 94202, dtype, 1)]
    dh = _ints((t, f), 94203, dtype, 1)
    want = nso.gated_mlp(*ts, activation="relu")
    want_g = nso.gated_mlp_grad(dh, *ts, activation="relu")
    x, wg, wu = (_place(v, lead)[1] for v in ts)
    _, vdh = _place(dh, lead)
    bh, vh = _place(torch.zeros(t, f, dtype=dtype), lead, 7.0)
    bg, vg = _place(torch.zeros(2, t, f, dtype=dtype), lead, 7.0)
    nso.gated_mlp(x, wg, wu, activation="relu", out=vh, gates_out=vg)
    assert torch.equal(vh, want)
    b1, v1 = _place(torch.zeros(f, d, dtype=dtype), lead, 7.0)
    b2, v2 = _place(torch.zeros(f, d, dtype=dtype), lead, 7.0)
    for gates in (vg, None):
        dx, _, _ = nso.gated_mlp_grad(vdh, x, wg, wu, gates, activation="relu", d_gate=v1, d_up=v2)
        assert torch.equal(dx, want_g[0]) and torch.equal(v1, want_g[1]) and torch.equal(v2, want_g[2])
    for b, n in ((bh, t * f), (bg, 2 * t * f), (b1, f * d), (b2, f * d)):
        assert bool((b[:lead] == 7).all()) and bool((b[lead + n:] == 7).all())


def test_nan_and_infinity_stay_in_their_rows():
    import newton_schulz_orthogonalized_amd as nso
    t, d, f = 140, 64, 90
    x, wg, wu, dh = _ints((t, d), 94300, BF, 2), _ints((f, d), 94301, BF, 1), _ints((f, d), 94302, BF, 1), _ints((t, f), 94303, BF, 1)
    clean = nso.gated_mlp(x, wg, wu, activation="relu")
    clean_dx = nso.gated_mlp_grad(dh, x, wg, wu, activation="relu")[0]
    x[37, 5] = float("nan")
    h = nso.gated_mlp(x, wg, wu)
    assert bool(h[37].isnan().all()) and int(h.isnan().any(1).sum()) == 1
    rows = torch.arange(t, device="cuda") != 37
    assert torch.equal(nso.gated_mlp(x, wg, wu, activation="relu")[rows], clean[rows])
    assert torch.equal(nso.gated_mlp_grad(dh, x, wg, wu, activation="relu")[0][rows], clean_dx[rows])
    x[37, 5] = 0
    wu[11, 3] = float("inf")
    h = nso.gated_mlp(x, wg, wu, activation="relu")
    cols = torch.arange(f, device="cuda") != 11
    x2 = nso.gated_mlp(x, wg, torch.where(wu.isinf(), 0, wu), activation="relu")
    assert torch.equal(h[:, cols], x2[:, cols])


def test_saturated_activations():
    """Gates far from zero: act(g) is g or 0 and its slope 1 or 0, without NaN."""
    import newton_schulz_orthogonalized_amd as nso
    for dtype in (BF, FP):
        x = torch.tensor([[200.0], [-200.0], [1e4], [-1e4]], dtype=dtype, device="cuda")
        one = torch.ones(1, 1, dtype=dtype, device="cuda")
        for act in ("silu", "gelu", "gelu_tanh", "relu"):
            h = nso.gated_mlp(x, one, one, activation=act)
            assert torch.equal(h, torch.where(x > 0, (x.float() * x.float()).to(dtype), torch.zeros_like(x))), act
            dx, dg, du = nso.gated_mlp_grad(torch.ones_like(x), x, one, one, activation=act)
            assert torch.equal(dx, torch.where(x > 0, 2 * x, torch.zeros_like(x))), act
            assert bool(dg.isfinite().all()) and bool(du.isfinite().all())


@pytest.mark.parametrize("save_gates", [True, False])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_autograd(dtype, save_gates):
    import newton_schulz_orthogonalized_amd as nso
    b, s, d, f = 2, 21, 48, 80
    x = _normal((b, s, d), 94400, dtype).requires_grad_()
    wg, wu = _normal((f, d), 94401, dtype, 0.2).requires_grad_(), _normal((f, d), 94402, dtype, 0.2).requires_grad_()
    g = _normal((s, b, f), 94403, dtype).transpose(0, 1)
    h = nso.gated_mlp(x, wg, wu, activation="gelu", save_gates=save_gates)
    with torch.no_grad():
        gates = torch.empty(2, b, s, f, dtype=dtype, device="cuda")
        assert torch.equal(nso.gated_mlp(x, wg, wu, activation="gelu", gates_out=gates), h)
        want = nso.gated_mlp_grad(g.contiguous(), x, wg, wu, gates if save_gates else None, activation="gelu")
    got = torch.autograd.grad(h, (x, wg, wu), g, retain_graph=True)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    for i, leaf in enumerate((x, wg, wu)):
        only, = torch.autograd.grad(h, leaf, g, retain_graph=True)
        assert torch.equal(only, want[i])
    shared = nso.gated_mlp(x, wg, wg, activation="relu", save_gates=save_gates)    # one weight in both places
    both, = torch.autograd.grad(shared, wg, g)
    with torch.no_grad():
        nso.gated_mlp(x, wg, wg, activation="relu", gates_out=gates)
        _, p, q = nso.gated_mlp_grad(g.contiguous(), x, wg, wg, gates if save_gates else None, activation="relu")
    assert torch.equal(both, p + q)


def test_gradients_against_differences():
    """Central differences with a step of 2^-7 (its square leaves 2^-14 of the
    loss's terms, the float32 results, off by 2 K U = 2^-18 of theirs, 2^-12 over
    the step)."""
    import newton_schulz_orthogonalized_amd as nso
    t, d, f = 6, 30, 25
    x, wg, wu = (_normal(s, 94500 + i, FP, 0.3).requires_grad_() for i, s in enumerate(((t, d), (f, d), (f, d))))
    g = _normal((t, f), 94510, FP)
    for act in ("silu", "gelu", "gelu_tanh"):
        got = torch.autograd.grad(nso.gated_mlp(x, wg, wu, activation=act), (x, wg, wu), g)
        for i in range(3):
            e = _normal(tuple((x, wg, wu)[i].shape), 94520 + i, FP)
            vals = []
            with torch.no_grad():
                for sign in (1, -1):
                    ts = [v + sign * 2.0 ** -7 * e if j == i else v for j, v in enumerate((x, wg, wu))]
                    vals.append((to_np(nso.gated_mlp(*ts, activation=act)) * to_np(g)).sum())
            num, ana = (vals[0] - vals[1]) * 64, (to_np(got[i]) * to_np(e)).sum()
            size = np.abs(to_np(g)).sum() * 8
            assert abs(num - ana) <= size * 2.0 ** -11, (act, i, num, ana)


def test_empty_calls():
    import newton_schulz_orthogonalized_amd as nso
    x, w = torch.empty(0, 24, device="cuda", dtype=BF), _normal((10, 24), 94600, BF)
    assert nso.gated_mlp(x, w, w.clone()).shape == (0, 10)
    dx, a, b = nso.gated_mlp_grad(torch.empty(0, 10, device="cuda", dtype=BF), x, w, w.clone(), dtype=FP)
    assert dx.shape == (0, 24) and bool((a == 0).all()) and bool((b == 0).all()) and a.dtype == FP
    a.fill_(3)
    nso.gated_mlp_grad(torch.empty(0, 10, device="cuda", dtype=BF), x, w, w.clone(), d_gate=a, d_up=b, accumulate=True)
    assert bool((a == 3).all())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("t,d,f", [(3, 24, 9), (40, 130, 100), (129, 64, 70)])
def test_a_workspace_of_nan(t, d, f, dtype):
    """What a workspace holds before the call does not matter, behind rows that
    are padded in it either."""
    import newton_schulz_orthogonalized_amd as nso
    x, wg, wu, dh = (_ints(s, 94650 + i, dtype, 2) for i, s in enumerate(((t, d), (f, d), (f, d), (t, f))))
    for gates in (None, _ints((2, t, f), 94660, dtype, 2)):
        want = nso.gated_mlp_grad(dh, x, wg, wu, gates, activation="relu", workspace=torch.zeros(1 << 22, dtype=torch.uint8, device="cuda"))
        got = nso.gated_mlp_grad(dh, x, wg, wu, gates, activation="relu",
                                 workspace=torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda"))
        assert all(bool(a.isfinite().all()) and torch.equal(a, b) for a, b in zip(got, want))


def test_streams_workspaces_and_captured_calls():
    """On a stream of its own, with a workspace of the caller's, and two graphs
    captured and replayed in turn, each replay against the eager calls."""
    import newton_schulz_orthogonalized_amd as nso
    t, d, f = 150, 100, 130     # odd rows: operands are copied into the workspace
    x, wg, wu = _normal((t, d), 94700, BF), _normal((f, d), 94701, BF, 0.1), _normal((f, d), 94702, BF, 0.1)
    dh = _normal((t, f), 94703, BF)

    def both(**more):
        gates = torch.empty(2, t, f, dtype=BF, device="cuda")
        h = nso.gated_mlp(x, wg, wu, gates_out=gates, **more)
        return (h, gates, *nso.gated_mlp_grad(dh, x, wg, wu, gates, dtype=FP, **more))
    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    h = nso.gated_mlp(x, wg, wu, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(h, want[0])
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
    got = both(workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        c1 = both()
    with torch.cuda.graph(g2):
        c2 = both()
    for _ in range(3):
        x.mul_(0.75)
        wg.mul_(-1)
        g1.replay()
        g2.replay()
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(c1, want)) and all(torch.equal(a, b) for a, b in zip(c2, want))
