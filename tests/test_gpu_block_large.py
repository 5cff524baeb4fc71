"""The block's calls on buffers of more than 2^31 elements: rows at both ends and
around the places where 31- and 32-bit offsets would turn over.

The norms and the rotation give a row the bits that a call on that row alone
gives. The gated product runs on small integers with the relu, where every
product and sum is exact, against float64 products of rows and columns."""

import pytest
import torch

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    import newton_schulz_orthogonalized_amd  # noqa: F401  (fails loudly without the library)
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    yield
    torch.cuda.empty_cache()


def _places(rows, row):
    """Rows of `row` elements at the ends and around element 2^30 and 2^31 (2^31 and 2^32 bytes)."""
    at = {0, 1, rows - 2, rows - 1}
    for e in (1 << 30, 1 << 31):
        at |= {e // row + d for d in (-1, 0, 1) if 0 <= e // row + d < rows}
    return torch.tensor(sorted(at), device="cuda")


def _noise(shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(shape, dtype=BF, device="cuda").normal_(generator=g)


def test_norms():
    import newton_schulz_orthogonalized_amd as nso
    rows, dim = (1 << 20) + 1029, 2048
    r, y, dn = (_noise((rows, dim), 95000 + i) for i in range(3))
    post, pre = _noise((dim,), 95003), _noise((dim,), 95004)
    kw = dict(post_weight=post, pre_weight=pre, residual_scale=0.8)
    at = _places(rows, dim)
    out, normed = nso.residual_norm(r, y, **kw)
    want = nso.residual_norm(r[at], y[at], **kw)
    assert torch.equal(out[at], want[0]) and torch.equal(normed[at], want[1])
    dr, dy = nso.residual_norm_grad(r, dn, out, y, **kw)[:2]
    want = nso.residual_norm_grad(r[at], dn[at], out[at], y[at], **kw)
    assert torch.equal(dr[at], want[0]) and torch.equal(dy[at], want[1])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary(interleaved):
    import newton_schulz_orthogonalized_amd as nso
    rows, heads, dim = 420001, 40, 128
    x = _noise((rows, heads, dim), 95010)
    freqs = nso.rotary_frequencies(dim)
    got = nso.rotary(x, freqs=freqs, interleaved=interleaved)
    at = _places(rows, heads * dim)
    assert torch.equal(got[at], nso.rotary(x[at], freqs=freqs, positions=at, interleaved=interleaved))
    nso.rotary(x, freqs=freqs, interleaved=interleaved, out=x)
    assert torch.equal(x[at], got[at])


def test_gated_product():
    import newton_schulz_orthogonalized_amd as nso
    t, d, f = 150001, 64, 14336
    g = torch.Generator(device="cuda")
    g.manual_seed(95020)

    def ints(shape, top, keep):
        v = torch.randint(-top, top + 1, shape, generator=g, device="cuda", dtype=torch.int8)
        return (v * (torch.rand(shape, generator=g, device="cuda") < keep)).to(BF)

    x, wg, wu = ints((t, d), 2, 1.0), ints((f, d), 2, 0.15), ints((f, d), 2, 0.15)
    dh = ints((t, f), 1, 0.05)
    rows = _places(t, f)
    cols = torch.cat([torch.arange(16, device="cuda"), torch.arange(f - 16, f, device="cuda")])
    X, G, U, DH = x[rows].double(), wg.double(), wu.double(), dh[rows].double()
    gg, uu = X @ G.t(), X @ U.t()
    assert max(float((X.abs() @ W.abs().t()).max()) for W in (G, U)) <= 256
    gates = torch.empty((2, t, f), dtype=BF, device="cuda")
    h = nso.gated_mlp(x, wg, wu, activation="relu", gates_out=gates)
    assert torch.equal(gates[0, rows].double(), gg) and torch.equal(gates[1, rows].double(), uu)
    assert torch.equal(h[rows], (gg.clamp(min=0) * uu).to(BF))
    want_x = (DH * uu * (gg > 0)) @ G + (DH * gg.clamp(min=0)) @ U
    X, DH = x.double(), dh[:, cols].double()
    gg, uu = X @ G[cols].t(), X @ U[cols].t()
    want_g, want_u = (DH * uu * (gg > 0)).t() @ X, (DH * gg.clamp(min=0)).t() @ X
    assert max(float(v.abs().max()) for v in (want_x, want_g, want_u)) < 2 ** 24
    for saved in (gates, None):
        dx, dg, du = nso.gated_mlp_grad(dh, x, wg, wu, saved, activation="relu", dtype=torch.float32)
        assert torch.equal(dx[rows], want_x.to(BF))
        assert torch.equal(dg[cols].double(), want_g) and torch.equal(du[cols].double(), want_u)
