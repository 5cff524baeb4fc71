"""Norms of rows at the end of the documented range: 16384 elements of 1e17, whose
squares sum to 1.6e38, against the reference with test_gpu_resnorm.py's
tolerances."""

import pytest
import torch

from gpu_util import need_gpu
from test_gpu_resnorm import _check_forward, _check_grads, _normal

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    import newton_schulz_orthogonalized_amd  # noqa: F401  (fails loudly without the library)
    yield


@pytest.mark.parametrize("rt,yt", [(BF, BF), (FP, FP), (FP, BF)])
@pytest.mark.parametrize("dim", [64, 2050, 16384])
def test_elements_of_1e17(dim, rt, yt):
    import newton_schulz_orthogonalized_amd as nso
    rows = 3
    signs = _normal((rows, dim), 97200, FP).sign()
    r, y = (signs * 0.5e17).to(rt), (signs * 1e17).to(yt)     # r' = 0.5e17 of the residual and N(y)
    pre, post = _normal((dim,), 97201, yt, 0.2, 1.0), _normal((dim,), 97202, yt, 0.2, 0.6)
    for post_norm in (True, False):     # without the norm of y: r' = 1e17, 0.5e17 from either side
        ya = y if post_norm else (y.float() * 0.5).to(yt)
        kw = dict(post_norm=post_norm, post_weight=post if post_norm else None, pre_weight=pre, residual_scale=1.0)
        new, n = nso.residual_norm(r, ya, **kw)
        _check_forward(r, ya, None, post_norm, kw["post_weight"], pre, 1.0, 1e-6, new, n)
        assert bool((n.float().abs() > 0).any(1).all())
        dr, dn = _normal((rows, dim), 97203, rt), _normal((rows, dim), 97204, yt)
        res = nso.residual_norm_grad(dr, dn, new, ya, **kw)
        assert all(x is None or bool(x.isfinite().all()) for x in res)
        _check_grads(res, dr, dn, new, ya, None, post_norm, kw["post_weight"], pre, 1.0, 1e-6)
