"""GPU parity of rotary positions against a float64 reference.

Tolerance: the angle's last float32 is half a turn's fraction, off by 2^-25 of
half a turn (pi 2^-25 radians); sine and cosine by 2 units of 2^-23 at most; their
product with scale, two products and a sum by 2^-24 each: together less than
8 * 2^-24 of scale (|a| + |b|), and half a step of the result's type (2^-8 of
bfloat16). The float64 angle is off by 2^-52 of it, 2^-29 at a million turns.
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


def _normal(shape, seed, dtype):
    return as_dtype(host_normal(shape, seed), dtype).cuda()


def _close(got, ref, mag, dtype):
    half = 2.0 ** -8 if dtype == BF else ULP
    tol = 8 * ULP * mag
    bad = ~(np.abs(to_np(got) - ref) <= tol + half * (np.abs(ref) + tol) * (mag > 0))
    assert not bad.any(), (np.argwhere(bad)[:4], to_np(got)[bad][:4], ref[bad][:4])


# batch, length, heads, k heads, dim, part
SHAPES = [(1, 1, 1, 1, 2, 2), (2, 3, 4, 2, 8, 4), (1, 70, 3, 1, 64, 64), (3, 17, 5, 5, 90, 70), (64, 1, 32, 8, 128, 64),
          (2, 33, 2, 1, 100, 2), (1, 5, 1, 1, 1024, 1024), (1, 9, 40, 1, 250, 250), (2, 129, 8, 2, 128, 128), (1, 300, 1, 1, 33, 32)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("b,s,hq,hk,d,part", SHAPES)
def test_both_tensors(b, s, hq, hk, d, part, dtype, interleaved):
    import newton_schulz_orthogonalized_amd as nso
    q, k = _normal((b, s, hq, d), 91000 + s, dtype), _normal((b, s, hk, d), 91001 + s, dtype)
    freqs = nso.rotary_frequencies(part)
    ref_f = B.frequencies_ref(part)
    assert np.allclose(to_np(freqs), ref_f, rtol=1e-14, atol=0)
    pos = np.broadcast_to(np.arange(s), (b, s))
    for inverse, scale in ((False, 1.0), (True, 1.25)):
        oq, ok = nso.rotary(q, k, freqs=freqs, interleaved=interleaved, scale=scale, inverse=inverse)
        torch.cuda.synchronize()
        for x, o in ((q, oq), (k, ok)):
            assert o.shape == x.shape and o.is_contiguous()
            ref, mag = B.rotary_ref(to_np(x), pos, ref_f, interleaved, scale, inverse)
            _close(o, ref, mag, dtype)
            assert torch.equal(o[..., part:], x[..., part:])
    assert torch.equal(nso.rotary(k, freqs=freqs, interleaved=interleaved, scale=scale, inverse=True), ok)


@pytest.mark.parametrize("bits", [torch.int32, torch.int64])
@pytest.mark.parametrize("shared", [False, True])
def test_positions(bits, shared):
    """Positions of their own, negative ones and ones of millions among them, an
    offset, and one row of positions for all sequences."""
    import newton_schulz_orthogonalized_amd as nso
    b, s, h, d = 3, 11, 2, 64
    x = _normal((b, s, h, d), 91100, FP)
    freqs = nso.rotary_frequencies(d, base=500000.0, factor=8.0, original_length=8192, high=4.0)
    rng = np.random.default_rng(91101)
    pos = rng.integers(-1000, 3_000_000, (s,) if shared else (b, s))
    t = torch.from_numpy(pos).to(bits).cuda()
    for offset in (0, 7, -100_000):
        o = nso.rotary(x, freqs=freqs, positions=t, offset=offset)
        ref, mag = B.rotary_ref(to_np(x), np.broadcast_to(pos + offset, (b, s)), to_np(freqs))
        _close(o, ref, mag, FP)


@pytest.mark.parametrize("kw", [dict(), dict(factor=4.0), dict(factor=8.0, original_length=8192, low=1.0, high=4.0),
                                dict(base=500000.0, factor=32.0, original_length=4096.0)])
def test_scaled_frequencies(kw):
    import newton_schulz_orthogonalized_amd as nso
    for part in (2, 70, 128):
        assert np.allclose(to_np(nso.rotary_frequencies(part, **kw)), B.frequencies_ref(part, **kw), rtol=1e-13, atol=0)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d,part,lead", [(64, 64, 0), (64, 32, 1), (90, 70, 1), (128, 128, 3)])
def test_views_of_a_fused_projection(d, part, lead, dtype):
    """Strided inputs at odd addresses, in place and into another buffer; what
    lies beside them is left as it was."""
    import newton_schulz_orthogonalized_amd as nso
    b, s, hq, hk = 2, 13, 4, 2
    flat = _normal((b * s * (hq + 2 * hk) * d + lead,), 91200, dtype)
    qkv = flat[lead:].view(b, s, hq + 2 * hk, d)
    before = qkv.clone()
    freqs = nso.rotary_frequencies(part)
    q, k = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
    oq, ok = nso.rotary(q, k, freqs=freqs)
    assert torch.equal(qkv, before)
    res = nso.rotary(q, k, freqs=freqs, out=(q, k))
    assert res[0].data_ptr() == q.data_ptr() and torch.equal(q, oq) and torch.equal(k, ok)
    assert torch.equal(qkv[:, :, hq + hk:], before[:, :, hq + hk:])
    wide = torch.full((b, hq, s, 2 * d), 7.0, dtype=dtype, device="cuda")   # heads first, rows apart
    out = wide[..., :d].permute(0, 2, 1, 3)
    nso.rotary(before[:, :, :hq], freqs=freqs, out=out)
    assert torch.equal(out, oq) and bool((wide[..., d:] == 7).all())


def test_packed_rows_and_one_token_of_a_batch():
    import newton_schulz_orthogonalized_amd as nso
    x = _normal((50, 3, 64), 91300, BF)
    pos = torch.cat([torch.arange(20), torch.arange(30)]).cuda()   # two sequences
    freqs = nso.rotary_frequencies(64)
    o = nso.rotary(x, freqs=freqs, positions=pos)
    assert torch.equal(o[:20], nso.rotary(x[:20], freqs=freqs)) and torch.equal(o[20:], nso.rotary(x[20:], freqs=freqs))
    one = nso.rotary(x[:, None], freqs=freqs, positions=pos[:, None])
    assert torch.equal(one[:, 0], o)
    assert torch.equal(nso.rotary(x[7:8], freqs=freqs, offset=7), o[7:8])


def test_many_rows_past_the_first_workgroups():
    import newton_schulz_orthogonalized_amd as nso
    x = _normal((1, 40000, 1, 4), 91400, FP)
    freqs = nso.rotary_frequencies(4, base=3.0)
    ref, mag = B.rotary_ref(to_np(x), np.arange(40000)[None], to_np(freqs))
    _close(nso.rotary(x, freqs=freqs), ref, mag, FP)


def test_empty_calls():
    import newton_schulz_orthogonalized_amd as nso
    freqs = nso.rotary_frequencies(4)
    for shape in ((0, 3, 2, 4), (2, 0, 2, 4), (2, 3, 0, 4), (0, 2, 4)):
        assert nso.rotary(torch.empty(shape, device="cuda"), freqs=freqs).shape == shape
    q = _normal((1, 3, 2, 4), 91500, FP)
    o, e = nso.rotary(q, q[:, :, :0], freqs=freqs)
    assert torch.equal(o, nso.rotary(q, freqs=freqs)) and e.numel() == 0


def test_nan_and_infinity_stay_in_their_pair():
    import newton_schulz_orthogonalized_amd as nso
    x = _normal((1, 6, 2, 16), 91600, FP)
    clean = nso.rotary(x, freqs=nso.rotary_frequencies(12))
    x[0, 2, 1, 3], x[0, 4, 0, 14] = float("nan"), float("inf")
    o = nso.rotary(x, freqs=nso.rotary_frequencies(12))
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit[0, 2, 1, 3] = hit[0, 2, 1, 9] = hit[0, 4, 0, 14] = True
    assert torch.equal(o[~hit], clean[~hit]) and bool(o[0, 2, 1, [3, 9]].isnan().all()) and bool(o[0, 4, 0, 14].isinf())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_gradients(dtype, interleaved):
    """Through autograd: the inverse turn of the results' gradients, whose layout
    may be any (heads first, expanded); broadcast queries get the sum."""
    import newton_schulz_orthogonalized_amd as nso
    b, s, hq, hk, d, part = 2, 9, 4, 2, 32, 20
    freqs = nso.rotary_frequencies(part)
    base = _normal((b, s, 1, d), 91700, dtype).requires_grad_()
    q, k = base.expand(b, s, hq, d), _normal((b, s, hk, d), 91701, dtype).requires_grad_()
    oq, ok = nso.rotary(q, k, freqs=freqs, interleaved=interleaved, scale=1.5, offset=3)
    gq = _normal((b, hq, s, d), 91702, dtype).transpose(1, 2)
    gk = _normal((1, 1, 1, d), 91703, dtype).expand(b, s, hk, d)
    torch.autograd.backward((oq, ok), (gq, gk))
    pos = np.broadcast_to(np.arange(s) + 3, (b, s))
    ref, mag = B.rotary_ref(to_np(gk), pos, to_np(freqs), interleaved, 1.5, True)
    _close(k.grad, ref, mag, dtype)
    per_head = nso.rotary(gq, freqs=freqs, interleaved=interleaved, scale=1.5, offset=3, inverse=True)
    assert torch.equal(base.grad, per_head.sum(2, keepdim=True))
    only, = torch.autograd.grad(nso.rotary(q, k, freqs=freqs)[1], k, gk)     # q's gradient is not asked for
    assert torch.equal(only, nso.rotary(gk, freqs=freqs, inverse=True))


def test_gradient_against_differences():
    """The call is linear: <g, R(x + e) - R(x)> = <R'g, e>, in float64 sums of
    float32 results (each off by 8 * 2^-24 of its pair)."""
    import newton_schulz_orthogonalized_amd as nso
    x, e, g = (_normal((1, 7, 2, 24), 91800 + i, FP) for i in range(3))
    freqs = nso.rotary_frequencies(24)
    x.requires_grad_()
    o = nso.rotary(x, freqs=freqs, scale=0.7)
    dx, = torch.autograd.grad(o, x, g)
    with torch.no_grad():
        moved = to_np(nso.rotary(x + e, freqs=freqs, scale=0.7)) - to_np(o)
    lhs, rhs = (moved * to_np(g)).sum(), (to_np(dx) * to_np(e)).sum()
    size = 2 * (np.abs(to_np(g)).sum() * (np.abs(to_np(x)).max() + np.abs(to_np(e)).max()))
    assert abs(lhs - rhs) <= 64 * ULP * size


def test_a_stream_of_its_own_and_a_captured_call():
    import newton_schulz_orthogonalized_amd as nso
    q, k = _normal((2, 65, 4, 64), 91900, BF), _normal((2, 65, 2, 64), 91901, BF)
    freqs = nso.rotary_frequencies(64)
    want = nso.rotary(q, k, freqs=freqs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = nso.rotary(q, k, freqs=freqs, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    pos = torch.arange(65, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = nso.rotary(q, k, freqs=freqs, positions=pos)
    for step in range(4):
        pos.copy_(torch.arange(65, device="cuda") + step)
        q.mul_(0.5)
        g.replay()
        want = nso.rotary(q, k, freqs=freqs, offset=step)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(cap, want))
