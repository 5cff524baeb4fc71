"""How far the gated product's float32 sums over long k are off.

Norm of the error over the norm, for independent normal terms. A chain of n additions
rounds each partial sum s by at most U |s| / sqrt(3) in the root mean square (U =
2^-24), and s over j terms has the square j: U^2 n^2 / 6 of a sum whose square is n.
In pieces of C = 512 terms that are added up behind each other, the pieces leave
U^2 n C / 6 and their sum U^2 n^2 / (6 C): relative U sqrt((C + n / C) / 6). A sum cut
into parts has shorter ones of both. Factors before and roundings behind the sum add
their U^2 each; tolerance 1.2 of that, for a hundred thousand results.
"""

import math

import pytest
import torch

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

ULP, C = 2.0 ** -24, 512


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    import newton_schulz_orthogonalized_amd  # noqa: F401  (fails loudly without the library)
    yield


def _normal(shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


def _check(got, want, n, more, what):
    err = float((got.double() - want).norm() / want.norm())
    assert err <= 1.2 * ULP * math.sqrt((C + n / C) / 6 + more), (what, err / ULP)


# tokens, dim, hidden; tiles of 64 and of 128, k split and not, whole and ragged
@pytest.mark.parametrize("t,d,f", [(200, 4096, 600), (1100, 4096, 2100), (1000, 8200, 1999), (64, 16384, 1024)])
def test_forward(t, d, f):
    import newton_schulz_orthogonalized_amd as nso
    x, wg, wu = _normal((t, d), 99400), _normal((f, d), 99401), _normal((f, d), 99402)
    gates = torch.empty((2, t, f), device="cuda")
    nso.gated_mlp(x, wg, wu, activation="relu", gates_out=gates)
    for v, w in zip(gates, (wg, wu)):
        _check(v, x.double() @ w.double().t(), d, 0, "forward")


@pytest.mark.parametrize("t,d,f", [(200, 600, 4096), (2200, 2100, 4096), (1999, 2200, 5000), (8192, 130, 1000), (16384, 520, 2050)])
def test_gradients(t, d, f):
    """The slopes' two products round dg, the activation's one du."""
    import newton_schulz_orthogonalized_amd as nso
    x, wg, wu, dh, gates = _normal((t, d), 99410), _normal((f, d), 99411), _normal((f, d), 99412), _normal((t, f), 99413), _normal((2, t, f), 99414)
    dx, d_gate, d_up = nso.gated_mlp_grad(dh, x, wg, wu, gates, activation="relu")
    g, u = gates.double()
    dg, du = dh.double() * u * (g > 0), dh.double() * g.clamp(min=0)
    _check(dx, dg @ wg.double() + du @ wu.double(), 2 * f, 1, "dx")
    _check(d_gate, dg.t() @ x.double(), t, 1, "d_gate")
    _check(d_up, du.t() @ x.double(), t, 1, "d_up")
