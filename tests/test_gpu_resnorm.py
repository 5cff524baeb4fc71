"""GPU parity of the norms around a block (residual_norm, rms_norm) and their
gradients against a float64 reference.

Tolerances, in U = 2^-24. A float32 sum of squares passes at most 16 additions in
a lane, 6 between lanes and 16 between waves: 40 U of it with the squares'
rounding; mean, eps, root and quotient leave its norm factor within 24 U. Products
and the residual sum add fewer than 8: new_residual is within 32 U of |a r| +
|update's share|, and the second norm of those errors (times their root mean square
over new_residual's) and 28 U of itself. The gradients' terms are within 128 U of
the sums of magnitudes that the reference gives (factors of 24 U, to the third
power in the projection, whose sum is 42 U of its magnitudes), the update's within
272 U; a sum over n rows adds n + 48 U of its magnitudes. Each result is rounded
by at most half a step of its type (bfloat16 2^-8).
"""

import numpy as np
import pytest
import torch

from gpu_util import need_gpu, to_np
from oracle import block_oracle as B
from workloads import as_dtype, host_normal

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32
ULP = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    import newton_schulz_orthogonalized_amd  # noqa: F401  (fails loudly without the library)
    yield


def _normal(shape, seed, dtype, std=1.0, mean=0.0):
    return as_dtype(host_normal(shape, seed, std) + mean, dtype).cuda()


def _np(t):
    return None if t is None else to_np(t)


def _half(dtype):
    return 2.0 ** -8 if dtype == BF else ULP


def _within(got, ref, tol, dtype, what):
    bad = ~(np.abs(to_np(got) - ref) <= tol + _half(dtype) * (np.abs(ref) + tol))
    assert not bad.any(), (what, np.argwhere(bad)[:4], to_np(got)[bad][:4], ref[bad][:4])


def _make(rows, dim, groups, rt, yt, wt, weights, seed):
    r, y = _normal((rows, dim), seed, rt, 2.0), _normal((rows, dim), seed + 1, yt, 0.5)
    gate = _normal((groups, dim), seed + 2, wt, 0.5) if groups else None
    post = _normal((dim,), seed + 3, wt, 0.2, 0.6) if weights else None
    pre = _normal((dim,), seed + 4, wt, 0.2, 1.0) if weights else None
    return r, y, gate, post, pre


def _check_forward(r, y, gate, post_norm, post, pre, a, eps, new, n):
    ref_new, ref_n, mag = B.residual_norm_ref(to_np(r), _np(y), _np(gate), post_norm, _np(post), _np(pre), a, eps)
    if new is not None:
        _within(new, ref_new, 32 * ULP * mag, r.dtype, "new_residual")
    w = np.ones(r.shape[1]) if pre is None else np.abs(to_np(pre))
    f = 1.0 / np.sqrt(np.mean(ref_new ** 2, 1, keepdims=True) + eps)
    grown = np.sqrt(np.mean(mag ** 2, 1, keepdims=True)) * f
    _within(n, ref_n, 32 * ULP * mag * f * w + np.abs(ref_n) * (32 * grown + 28) * ULP, n.dtype, "normed")


def _check_grads(res, dr, dn, new, y, gate, post_norm, post, pre, a, eps):
    ref = B.residual_norm_grad_ref(_np(dr), _np(dn), to_np(new), _np(y), _np(gate), post_norm, _np(post), _np(pre), a, eps)
    rows = new.shape[0]
    for got, name, k in zip(res, ("r", "y", "gate", "post", "pre"), (128, 272, 176 + rows, 176 + rows, 80 + rows)):
        if got is not None:
            g, mag = ref[name]
            _within(got, g.reshape(got.shape), k * ULP * mag.reshape(got.shape), got.dtype, name)


TYPES = [(BF, BF, BF), (FP, FP, FP), (FP, BF, BF), (BF, BF, FP), (FP, BF, FP)]
# rows, dim, groups (0: no gate)
SHAPES = [(1, 1, 0), (1, 7, 1), (3, 64, 0), (6, 513, 3), (9, 512, 9), (5, 1000, 0), (33, 1024, 1), (4, 1025, 2), (8, 2048, 4),
          (7, 2050, 0), (6, 4096, 2), (3, 4097, 0), (4, 8192, 1), (2, 9001, 2), (2, 16384, 0), (130, 96, 2), (700, 24, 700),
          (37, 64, 1), (1000, 65, 2), (257, 128, 0), (70, 129, 7), (300, 200, 1), (100, 256, 4), (41, 257, 0)]


@pytest.mark.parametrize("rt,yt,wt", TYPES)
@pytest.mark.parametrize("rows,dim,groups", SHAPES)
def test_forward_and_gradients(rows, dim, groups, rt, yt, wt):
    import newton_schulz_orthogonalized_amd as nso
    for i, (weights, post_norm, a, eps) in enumerate([(True, True, 0.75, 1e-6), (False, False, 1.0, 1e-5), (False, True, -0.5, 1e-3)]):
        r, y, gate, post, pre = _make(rows, dim, groups, rt, yt, wt, weights, 92000 + rows + dim)
        kw = dict(gate=gate, post_norm=post_norm, post_weight=post, pre_weight=pre, residual_scale=a, eps=eps)
        new, n = nso.residual_norm(r, y, **kw)
        torch.cuda.synchronize()
        assert new.dtype == rt and n.dtype == yt
        _check_forward(r, y, gate, post_norm, post, pre, a, eps, new, n)
        dr, dn = _normal((rows, dim), 92500 + i, rt), _normal((rows, dim), 92600 + i, yt)
        for gr, gn in ((dr, dn), (None, dn), (dr, None)):
            res = nso.residual_norm_grad(gr, gn, new, y, **kw)
            torch.cuda.synchronize()
            assert [x is None for x in res] == [False, False, gate is None, post is None, pre is None]
            _check_grads(res, gr, gn, new, y, gate, post_norm, post, pre, a, eps)
        if gate is not None and groups == 1:
            flat = nso.residual_norm(r, y, **{**kw, "gate": gate[0]})
            assert torch.equal(flat[0], new) and torch.equal(flat[1], n)


@pytest.mark.parametrize("xt,nt,wt", [(BF, BF, FP), (FP, FP, FP), (FP, BF, BF)])
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 64), (70, 257), (5, 2048), (9, 5000)])
def test_rms_norm(rows, dim, xt, nt, wt):
    import newton_schulz_orthogonalized_amd as nso
    x, w, dn = _normal((rows, dim), 93000, xt, 3.0), _normal((dim,), 93001, wt, 0.2, 1.0), _normal((rows, dim), 93002, nt)
    x.requires_grad_()
    w.requires_grad_()
    n = nso.rms_norm(x, w, dtype=nt, eps=1e-5)
    _check_forward(x, None, None, False, None, w, 1.0, 1e-5, None, n)
    n.backward(dn)
    _check_grads((x.grad, None, None, None, w.grad), None, dn, x, None, None, False, None, w, 1.0, 1e-5)
    with torch.no_grad():
        assert torch.equal(nso.rms_norm(x, dtype=nt), nso.rms_norm(x, torch.ones_like(w), dtype=nt))
        if xt == nt:
            y = x.detach().clone()
            nso.rms_norm(y, w, eps=1e-5, out=y)
            assert torch.equal(y, n)


@pytest.mark.parametrize("rows,dim,groups", [(3000, 512, 2), (2048, 300, 1), (20000, 64, 1), (9000, 128, 3), (7000, 250, 100), (5000, 100, 5000), (1500, 2048, 3), (600, 6000, 600)])
def test_sums_over_many_rows(rows, dim, groups):
    """Column sums of more rows than workgroups, and more gates than workgroups;
    the same call gives the same bits."""
    import newton_schulz_orthogonalized_amd as nso
    r, y, gate, post, pre = _make(rows, dim, groups, FP, BF, FP, True, 93100)
    kw = dict(gate=gate, post_weight=post, pre_weight=pre, residual_scale=0.5)
    new, n = nso.residual_norm(r, y, **kw)
    dr, dn = _normal((rows, dim), 93110, FP), _normal((rows, dim), 93111, BF)
    res = nso.residual_norm_grad(dr, dn, new, y, **kw)
    _check_grads(res, dr, dn, new, y, gate, True, post, pre, 0.5, 1e-6)
    again = nso.residual_norm_grad(dr, dn, new, y, **kw)
    assert all(torch.equal(a, b) for a, b in zip(res, again))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim", [9, 130, 2050])
def test_odd_addresses_guards_and_places(dim, dtype):
    """Rows that start at odd elements; nothing is written beside the results;
    the residual and the update in place."""
    import newton_schulz_orthogonalized_amd as nso
    rows = 5

    def place(t):
        buf = torch.full((t.numel() + 11,), 7.0, dtype=t.dtype, device="cuda")
        v = buf[3:3 + t.numel()].view(t.shape)
        v.copy_(t)
        return buf, v
    r, y, gate, post, pre = _make(rows, dim, 1, dtype, dtype, dtype, True, 93200 + dim)
    kw = dict(gate=gate, post_weight=post, pre_weight=pre)
    want = nso.residual_norm(r, y, **kw)
    (br, vr), (by, vy) = place(r), place(y)
    (bo, vo), (bn, vn) = place(torch.zeros_like(r)), place(torch.zeros_like(y))
    nso.residual_norm(vr, vy, out=vo, normed_out=vn, **kw)
    assert torch.equal(vo, want[0]) and torch.equal(vn, want[1]) and torch.equal(vr, r) and torch.equal(vy, y)
    res = nso.residual_norm(vr, vy, out=vr, normed_out=vy, **kw)
    assert res[0] is vr and torch.equal(vr, want[0]) and torch.equal(vy, want[1])
    for b in (br, by, bo, bn):
        assert bool((b[:3] == 7).all()) and bool((b[-8:] == 7).all())


def test_extremes():
    """Rows of zeros, tiny and large values, NaN and infinity: each row by itself."""
    import newton_schulz_orthogonalized_amd as nso
    dim = 600
    r, y = _normal((7, dim), 93300, FP), _normal((7, dim), 93301, FP)
    r[1], y[1] = 0.0, 0.0
    r[2] *= 1e-15
    y[2] *= 1e-15
    r[3] *= 1e17
    y[4, 5], y[5, 7] = float("nan"), float("inf")
    new, n = nso.residual_norm(r, y, post_norm=True)
    good = [0, 1, 2, 3, 6]
    _check_forward(r[good], y[good], None, True, None, None, 1.0, 1e-6, new[good], n[good])
    assert bool((new[1] == 0).all()) and bool((n[1] == 0).all())
    assert bool(new[4].isnan().all()) and bool(n[4].isnan().all()) and bool(new[5, 7].isnan()) and bool(n[5].isnan().all())
    dr, dn = torch.ones_like(r), _normal((7, dim), 93302, FP)
    d_r, d_y, *_ = nso.residual_norm_grad(dr, dn, new, y, post_norm=True)
    assert bool(d_r[good].isfinite().all()) and bool(d_y[good].isfinite().all())
    assert bool(d_r[4].isnan().all())
    tiny = nso.rms_norm(r[1:2], eps=1e-30)
    d_tiny = nso.residual_norm_grad(None, dn[1:2], r[1:2], None, eps=1e-30)[0]
    assert bool((tiny == 0).all()) and bool(d_tiny.isfinite().all())


@pytest.mark.parametrize("rt,yt", [(BF, BF), (FP, FP), (FP, BF)])
def test_autograd(rt, yt):
    """Through autograd: the functional call's gradients, batches of any shape,
    shared and broadcast tensors, parts of the gradients."""
    import newton_schulz_orthogonalized_amd as nso
    b, s, dim = 3, 5, 72
    wt = yt
    r, y = _normal((b, s, dim), 93400, rt).requires_grad_(), _normal((b, s, dim), 93401, yt).requires_grad_()
    gate, w = _normal((b, dim), 93402, wt).requires_grad_(), _normal((dim,), 93403, wt, 0.1, 1.0).requires_grad_()
    dr, dn = _normal((b, s, dim), 93404, rt), _normal((s, b, dim), 93405, yt).transpose(0, 1)
    kw = dict(gate=gate, post_weight=w, pre_weight=w, residual_scale=0.5)    # one weight in both places
    new, n = nso.residual_norm(r, y, **kw)
    with torch.no_grad():
        plain = nso.residual_norm(r, y, **kw)
        want = nso.residual_norm_grad(dr, dn.contiguous(), plain[0], y, **kw)
    assert torch.equal(plain[0], new) and torch.equal(plain[1], n)
    got = torch.autograd.grad((new, n), (r, y, gate, w), (dr, dn), retain_graph=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    assert torch.equal(got[3], want[3] + want[4])
    only, = torch.autograd.grad(n, y, dn, retain_graph=True)
    with torch.no_grad():
        assert torch.equal(only, nso.residual_norm_grad(None, dn.contiguous(), new, y, **kw)[1])
    only, = torch.autograd.grad(new, r, dr)
    assert torch.equal(only, (dr.float() * 0.5).to(rt))
    # a gate shared by the batch and expanded to it gets the sum
    row = _normal((1, dim), 93406, wt).requires_grad_()
    new, n = nso.residual_norm(r, y, gate=row.expand(b, dim).contiguous())
    n.backward(dn)
    assert row.grad.shape == row.shape


def test_gradients_against_differences():
    """Central differences with a step of 2^-7: its square leaves 2^-14 of the
    loss's terms, and the float32 results (off by 64 U of them) over the step
    2^-12; together less than 2^-11."""
    import newton_schulz_orthogonalized_amd as nso
    rows, dim = 4, 40
    r, y, gate, post, pre = _make(rows, dim, 2, FP, FP, FP, True, 93500)
    dr, dn = _normal((rows, dim), 93510, FP), _normal((rows, dim), 93511, FP)
    leaves = [t.requires_grad_() for t in (r, y, gate, post, pre)]
    kw = dict(residual_scale=0.75)

    def loss(ts):
        new, n = nso.residual_norm(ts[0], ts[1], gate=ts[2], post_weight=ts[3], pre_weight=ts[4], **kw)
        return new, n
    got = torch.autograd.grad(loss(leaves), leaves, (dr, dn))
    step = 2.0 ** -7
    for i, t in enumerate(leaves):
        e = _normal(tuple(t.shape), 93520 + i, FP)
        with torch.no_grad():
            vals = []
            for sign in (1, -1):
                new, n = loss([x + sign * step * e if j == i else x for j, x in enumerate(leaves)])
                vals.append((to_np(new) * to_np(dr) + to_np(n) * to_np(dn)).sum())
        num, ana = (vals[0] - vals[1]) / (2 * step), (to_np(got[i]) * to_np(e)).sum()
        size = (np.abs(to_np(dr)).sum() + np.abs(to_np(dn)).sum()) * 4
        assert abs(num - ana) <= size * 2.0 ** -11, (i, num, ana, size)


def test_empty_calls():
    import newton_schulz_orthogonalized_amd as nso
    r = torch.empty(0, 32, device="cuda")
    w, gate = torch.ones(32, device="cuda"), torch.ones(3, 32, device="cuda")
    new, n = nso.residual_norm(r, r.clone(), gate=gate, post_weight=w, pre_weight=w)
    assert new.shape == n.shape == (0, 32)
    res = nso.residual_norm_grad(r, r, new, r, gate=gate, post_weight=w, pre_weight=w)
    assert all(bool((x == 0).all()) for x in res) and res[2].shape == (3, 32)


def test_a_stream_of_its_own_and_a_captured_call():
    import newton_schulz_orthogonalized_amd as nso
    rows, dim = 90, 768
    r, y, gate, post, pre = _make(rows, dim, 3, FP, BF, BF, True, 93600)
    kw = dict(gate=gate, post_weight=post, pre_weight=pre)
    dr, dn = _normal((rows, dim), 93610, FP), _normal((rows, dim), 93611, BF)

    def both(**more):
        new, n = nso.residual_norm(r, y, **kw, **more)
        return (new, n, *nso.residual_norm_grad(dr, dn, new, y, **kw, **more))
    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g, h = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = both()
    with torch.cuda.graph(h):
        cap2 = both()
    for _ in range(3):
        r.mul_(0.5)
        dn.mul_(-0.75)
        g.replay()
        h.replay()
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(cap, want)) and all(torch.equal(a, b) for a, b in zip(cap2, want))
