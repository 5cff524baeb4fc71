"""Gates so far from zero that their square or cube leaves float32: act(g) is g or
0 and its slope 1 or 0, in the forward product and both forms of the gradient."""

import pytest
import torch

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    import newton_schulz_orthogonalized_amd  # noqa: F401  (fails loudly without the library)
    yield


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("power", [30, 45, 63, 66, 100, 120])
def test_slopes(power, act, dtype):
    """Gates of 2^power and -2^power beside up projections of 1 and -1: powers of
    two throughout, every value exact."""
    import newton_schulz_orthogonalized_amd as nso
    x = torch.tensor([[1.0], [-1.0]], dtype=dtype, device="cuda") * 2.0 ** power
    wg, wu = torch.ones(1, 1, dtype=dtype, device="cuda"), torch.full((1, 1), 2.0 ** -power, dtype=dtype, device="cuda")
    dh = torch.full_like(x, 2.0 ** -power)
    gates = torch.empty(2, 2, 1, dtype=dtype, device="cuda")
    h = nso.gated_mlp(x, wg, wu, activation=act, gates_out=gates)
    assert h.tolist() == [[2.0 ** power], [0.0]]
    for saved in (gates, None):
        dx, dg, du = nso.gated_mlp_grad(dh, x, wg, wu, saved, activation=act)
        assert dx.tolist() == [[2.0 ** (1 - power)], [0.0]]
        assert dg.tolist() == [[1.0]] and du.tolist() == [[2.0 ** power]]
