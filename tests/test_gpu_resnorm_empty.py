"""Empty batches through residual_norm with a gate for each token or sequence: the
gate then has no row either."""

import pytest
import torch

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    import newton_schulz_orthogonalized_amd  # noqa: F401  (fails loudly without the library)
    yield


@pytest.mark.parametrize("post_norm", [False, True])
def test_a_gate_without_rows(post_norm):
    import newton_schulz_orthogonalized_amd as nso
    r, gate, w = torch.empty(0, 7, 32, device="cuda"), torch.empty(0, 32, device="cuda"), torch.ones(32, device="cuda")
    kw = dict(gate=gate, pre_weight=w, post_norm=post_norm, post_weight=w if post_norm else None)
    new, n = nso.residual_norm(r, r.clone(), **kw)
    assert new.shape == n.shape == r.shape
    res = nso.residual_norm_grad(r, r, new, r, **kw)
    assert res[2].shape == (0, 32) and bool((res[4] == 0).all()) and (res[3] is None or bool((res[3] == 0).all()))
    leaves = [t.clone().requires_grad_() for t in (r, r, gate, w)]
    out = nso.residual_norm(leaves[0], leaves[1], gate=leaves[2], pre_weight=leaves[3], post_norm=post_norm)
    torch.autograd.backward(out, (r, r))
    assert [t.grad.shape for t in leaves] == [t.shape for t in leaves] and bool((leaves[3].grad == 0).all())
