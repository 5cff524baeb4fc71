"""Gradients of tens of megabytes that autograd hands to the block's calls
transposed or expanded. Their dense copies come from one large free block of the
allocator, and so does what is allocated behind them: a copy that nobody held over
the launch would share its memory with the call's workspace. The functional calls
on dense gradients give the same bits."""

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
    torch.cuda.empty_cache()


def _noise(shape, seed, dtype, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0, std, generator=g)


def _one_free_block(nbytes):
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    block = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    del block


def _like(kind, shape, seed, dtype):
    if kind == "transposed":
        return _noise(shape[::-1], seed, dtype).t()
    return _noise((1, 1), seed, dtype).expand(shape)


@pytest.mark.parametrize("kind", ["transposed", "expanded"])
@pytest.mark.parametrize("rt,yt", [(BF, BF), (FP, BF), (FP, FP)])
def test_norms(kind, rt, yt):
    import newton_schulz_orthogonalized_amd as nso
    rows, dim = 6000, 2048
    r, y, w = _noise((rows, dim), 96000, rt), _noise((rows, dim), 96001, yt), _noise((dim,), 96002, yt)
    kw = dict(post_weight=w, pre_weight=w, residual_scale=0.5)
    dr, dn = _like(kind, (rows, dim), 96003, rt), _like(kind, (rows, dim), 96004, yt)
    new, n = nso.residual_norm(r, y, **kw)
    want = nso.residual_norm_grad(dr.contiguous(), dn.contiguous(), new, y, **kw)
    leaves = [t.clone().requires_grad_() for t in (r, y)]
    ws = [w.clone().requires_grad_() for _ in range(2)]
    res = nso.residual_norm(*leaves, post_weight=ws[0], pre_weight=ws[1], residual_scale=0.5)
    _one_free_block(12 * rows * dim * 4)
    got = torch.autograd.grad(res, [*leaves, *ws], (dr, dn))
    assert all(torch.equal(a, b) for a, b in zip(got, (want[0], want[1], want[3], want[4])))
    want = nso.residual_norm_grad(None, dn.contiguous(), y, None, pre_weight=w)
    n = nso.rms_norm(leaves[1], ws[1])
    _one_free_block(12 * rows * dim * 4)
    got = torch.autograd.grad(n, (leaves[1], ws[1]), dn)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[4])


@pytest.mark.parametrize("kind", ["transposed", "expanded"])
@pytest.mark.parametrize("save_gates", [True, False])
@pytest.mark.parametrize("dtype,t,d,f", [(BF, 2048, 512, 4096), (BF, 3000, 500, 3001), (FP, 2500, 250, 1111)])
def test_gated_product(dtype, t, d, f, save_gates, kind):
    import newton_schulz_orthogonalized_amd as nso
    x, wg, wu = _noise((t, d), 96010, dtype), _noise((f, d), 96011, dtype, d ** -0.5), _noise((f, d), 96012, dtype, d ** -0.5)
    g = _like(kind, (t, f), 96013, dtype)
    gates = torch.empty((2, t, f), dtype=dtype, device="cuda") if save_gates else None
    h = nso.gated_mlp(x, wg, wu, gates_out=gates)
    want = nso.gated_mlp_grad(g.contiguous(), x, wg, wu, gates)
    leaves = [v.clone().requires_grad_() for v in (x, wg, wu)]
    out = nso.gated_mlp(*leaves, save_gates=save_gates)
    assert torch.equal(out, h)
    _one_free_block(16 * t * f * dtype.itemsize)
    got = torch.autograd.grad(out, leaves, g)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_sum_of_the_results():
    """backward() of a plain sum: every gradient is an expanded one."""
    import newton_schulz_orthogonalized_amd as nso
    t, d, f = 4000, 512, 2048
    x, wg, wu = _noise((t, d), 96020, BF), _noise((f, d), 96021, BF, d ** -0.5), _noise((f, d), 96022, BF, d ** -0.5)
    ones = torch.ones((t, f), dtype=BF, device="cuda")
    want = nso.gated_mlp_grad(ones, x, wg, wu)
    leaves = [v.clone().requires_grad_() for v in (x, wg, wu)]
    out = nso.gated_mlp(*leaves, save_gates=False).sum()
    _one_free_block(16 * t * f * 2)
    out.backward()
    assert all(torch.equal(a.grad, b) for a, b in zip(leaves, want))
