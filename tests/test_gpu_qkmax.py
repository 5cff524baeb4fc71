"""GPU parity of the attention max logits against a float64 reference.

Tolerance: a logit is a float32 sum of D products (those of bfloat16 are
exact). Each partial sum is off by at most one step of the sum of magnitudes
(2^-23: a matrix instruction may truncate where it aligns its terms), a float32
product by half a step, and the scale by half a step: (D + 2) * 2^-23 of
|scale| sum |q_d k_d|, of which the reference gives the largest. A maximum
moves by no more than its terms do.
"""

import numpy as np
import pytest
import torch

from gpu_util import need_gpu, to_np
from oracle import feed_oracle as F
from oracle import muon_oracle as O
from workloads import as_dtype, host_normal

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    import newton_schulz_orthogonalized_amd  # noqa: F401  (fails loudly without the library)
    yield


def _qk(b, nq, nk, hq, hk, d, dtype, seed):
    q = as_dtype(host_normal((b, nq, hq, d), seed), dtype).cuda()
    k = as_dtype(host_normal((b, nk, hk, d), seed + 1), dtype).cuda()
    return q, k


def _agree(got, seqs, group, scale, causal, d):
    best, mag = F.qk_max_logits_ref(seqs, group, scale, causal)
    got = to_np(got)
    assert np.all(np.abs(got - best) <= (d + 2) * 2.0 ** -23 * mag), (got, best)
    assert np.all(got[mag == 0] == 0)


def _dense(q, k, lq=None, lk=None):
    q, k = to_np(q), to_np(k)
    return [(q[b, :None if lq is None else lq[b]], k[b, :None if lk is None else lk[b]]) for b in range(q.shape[0])]


LENGTHS = [(1, 1), (2, 1), (1, 70), (31, 33), (64, 64), (65, 127), (128, 300), (300, 129), (257, 257), (520, 520)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,nk", LENGTHS)
def test_lengths(nq, nk, d, dtype, causal):
    import newton_schulz_orthogonalized_amd as nso
    q, k = _qk(2, nq, nk, 4, 2, d, dtype, 80000 + nq)
    got = nso.qk_max_logits(q, k, causal=causal)
    torch.cuda.synchronize()
    _agree(got, _dense(q, k), 2, d ** -0.5, causal, d)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [1, 3, 8, 16, 31, 32, 40, 72, 80, 96, 100, 120, 160, 192, 200, 255, 256])
def test_head_dimensions(d, dtype):
    """Every kind of head width; widths off a multiple of 8 put rows at odd
    addresses."""
    import newton_schulz_orthogonalized_amd as nso
    print(f"[qkmax] d {d} {dtype}", flush=True)
    q, k = _qk(1, 150, 170, 3, 1, d, dtype, 81000 + d)
    for causal in (True, False):
        got = nso.qk_max_logits(q, k, causal=causal, scale=-0.7)
        torch.cuda.synchronize()
        _agree(got, _dense(q, k), 3, -0.7, causal, d)


@pytest.mark.parametrize("hq,hk", [(1, 1), (5, 5), (8, 1), (12, 4), (32, 8), (33, 11), (64, 64)])
def test_head_groups(hq, hk):
    import newton_schulz_orthogonalized_amd as nso
    q, k = _qk(2, 140, 140, hq, hk, 64, BF, 82000 + hq)
    got = nso.qk_max_logits(q, k)
    torch.cuda.synchronize()
    _agree(got, _dense(q, k), hq // hk, 0.125, True, 64)


def test_every_pair_counts():
    """One large logit at a time, at corners of tiles and of the causal border:
    the head that holds it, and no other, reports it; one place above the border
    none does."""
    import newton_schulz_orthogonalized_amd as nso
    n, d = 600, 64
    for i, j in [(0, 0), (599, 599), (599, 0), (31, 31), (32, 31), (63, 32), (127, 127), (128, 127), (255, 255), (256, 255),
                 (300, 299), (511, 64), (512, 511), (400, 399)]:
        q = torch.zeros(1, n, 4, d, dtype=BF, device="cuda")
        k = torch.zeros(1, n, 2, d, dtype=BF, device="cuda")
        q[0, i, 2, 11] = -3.0
        k[0, j, 1, 11] = 5.0
        got = nso.qk_max_logits(q, k, scale=1.0)
        assert got.tolist() == [0.0, 0.0, 15.0, 0.0], (i, j)
        if j + 1 <= n - 1 and j + 1 > i:
            k[0, j, 1, 11] = 0.0
            k[0, j + 1, 1, 11] = 5.0
            assert nso.qk_max_logits(q, k, scale=1.0).tolist() == [0.0] * 4, (i, j + 1)
            assert nso.qk_max_logits(q, k, scale=1.0, causal=False).tolist() == [0.0, 0.0, 15.0, 0.0]


@pytest.mark.parametrize("dtype", [BF, FP])
def test_padded_batches(dtype):
    """Lengths per batch row, 0 and out-of-range ones among them; what lies
    behind them, NaN included, does not matter."""
    import newton_schulz_orthogonalized_amd as nso
    b, s, d = 6, 200, 80
    q, k = _qk(b, s, s, 4, 2, d, dtype, 83000)
    raw = [200, 1, 0, 77, 128, 999]
    lens = [min(max(x, 0), s) for x in raw]
    for i, n in enumerate(lens):
        q[i, n:], k[i, n:] = float("nan"), float("inf")
    t = torch.tensor(raw, dtype=torch.int32, device="cuda")
    for causal in (True, False):
        got = nso.qk_max_logits(q, k, causal=causal, lengths=t)
        torch.cuda.synchronize()
        _agree(got, _dense(q, k, lens, lens), 2, d ** -0.5, causal, d)
    lk = [150, 20, 5, 0, 200, 64]
    q, k = _qk(b, s, s, 4, 2, d, dtype, 83100)
    tk = torch.tensor(lk, dtype=torch.int32, device="cuda")
    for causal in (True, False):   # more queries than keys: the first queries see nothing
        got = nso.qk_max_logits(q, k, causal=causal, lengths=t, k_lengths=tk)
        torch.cuda.synchronize()
        _agree(got, _dense(q, k, lens, lk), 2, d ** -0.5, causal, d)
    none = torch.full((b,), -3, dtype=torch.int32, device="cuda")
    assert nso.qk_max_logits(q, k, lengths=none).tolist() == [0.0] * 4


@pytest.mark.parametrize("d", [64, 100, 128])
@pytest.mark.parametrize("docs", [[1], [300], [1, 1, 1], [0, 5, 0, 130, 64, 1, 0], [257, 3, 128, 400, 65, 31, 1, 99]])
def test_packed_sequences(docs, d):
    import newton_schulz_orthogonalized_amd as nso
    n = sum(docs)
    q, k = _qk(1, n + 5, n + 5, 6, 2, d, BF, 84000 + n)
    q, k = q[0], k[0]
    q[n:], k[n:] = float("nan"), float("nan")    # rows behind the last sequence
    edges = np.concatenate([[0], np.cumsum(docs)])
    cu = torch.tensor(edges, dtype=torch.int32, device="cuda")
    for causal in (True, False):
        got = nso.qk_max_logits(q, k, causal=causal, cu_seqlens=cu)
        torch.cuda.synchronize()
        _agree(got, [(to_np(q[a:b]), to_np(k[a:b])) for a, b in zip(edges[:-1], edges[1:])], 3, d ** -0.5, causal, d)


def test_packed_keys_of_their_own_and_entries_out_of_range():
    import newton_schulz_orthogonalized_amd as nso
    q, k = _qk(1, 100, 333, 2, 2, 64, BF, 85000)
    q, k = q[0], k[0]
    eq, ek = [0, 10, 10, 64, 100], [0, 200, 203, 203, 333]
    cq, ck = (torch.tensor(e, dtype=torch.int32, device="cuda") for e in (eq, ek))
    got = nso.qk_max_logits(q, k, cu_seqlens=cq, cu_seqlens_k=ck)
    torch.cuda.synchronize()
    seqs = [(to_np(q[eq[i]:eq[i + 1]]), to_np(k[ek[i]:ek[i + 1]])) for i in range(4)]
    _agree(got, seqs, 1, 0.125, True, 64)
    # entries beyond the buffers are cut to them, falling ones are empty sequences
    cq = torch.tensor([-7, 50, 20, 100000], dtype=torch.int32, device="cuda")
    got = nso.qk_max_logits(q, q, cu_seqlens=cq)
    torch.cuda.synchronize()
    _agree(got, [(to_np(q[0:50]),) * 2, (to_np(q[20:100]),) * 2], 1, 0.125, True, 64)


def test_strided_views_of_a_fused_projection():
    """q and k as column ranges of one projection, heads-first tensors
    transposed into place, an expanded batch, and a view at an odd offset."""
    import newton_schulz_orthogonalized_amd as nso
    for d in (64, 72, 128):
        qkv = as_dtype(host_normal((2, 190, 10, d), 86000 + d), BF).cuda()
        q, k = qkv[:, :, :6], qkv[:, :, 6:8]
        _agree(nso.qk_max_logits(q, k), _dense(q, k), 3, d ** -0.5, True, d)
        ht = as_dtype(host_normal((2, 4, 190, d), 86100 + d), BF).cuda()
        q, k = ht.transpose(1, 2), ht[:, :2].transpose(1, 2)
        _agree(nso.qk_max_logits(q, k), _dense(q, k), 2, d ** -0.5, True, d)
        q, k = _qk(1, 50, 60, 2, 1, d, BF, 86200)
        q, k = q.expand(3, -1, -1, -1), k.expand(3, -1, -1, -1)
        _agree(nso.qk_max_logits(q, k), _dense(q, k), 2, d ** -0.5, True, d)
        flat = as_dtype(host_normal(200 * 2 * d + 3, 86300), BF).cuda()
        q = flat[3:].view(1, 200, 2, d)
        _agree(nso.qk_max_logits(q, q), _dense(q, q), 1, d ** -0.5, True, d)
        every = as_dtype(host_normal((1, 150, 4, d), 86400), BF).cuda()[:, ::3]     # every third row
        _agree(nso.qk_max_logits(every, every), _dense(every, every), 1, d ** -0.5, True, d)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_nan_and_infinity_where_they_are_seen(dtype):
    import newton_schulz_orthogonalized_amd as nso
    q, k = _qk(1, 140, 140, 3, 3, 64, dtype, 87000)
    k[0, 100, 0, 5] = float("nan")     # head 0: seen by queries 100 .. 139
    q[0, 3, 1, 5] = float("inf")       # head 1
    got = nso.qk_max_logits(q, k)
    torch.cuda.synchronize()
    assert bool(got[0].isnan()) and bool(got[1].isinf()) and bool(got[2].isfinite())
    # the last key of a causal block whose queries end before it
    q2, k2 = q[:, :100].clone(), k.clone()
    q2[0, 3, 1, 5] = 1.0
    got = nso.qk_max_logits(q2, k2[:, :100])
    torch.cuda.synchronize()
    assert bool(got.isfinite().all())
    k3 = k[:, :100].clone()
    k3[0, 99] = float("nan")           # seen by the last query only
    assert bool(nso.qk_max_logits(q2, k3).isnan().all())
    assert bool(nso.qk_max_logits(q2[:, :99], k3[:, :99]).isfinite().all())
    q2[0, 0] = float("nan")
    q4 = torch.cat([q2[:, :1], q2], 1)   # 101 queries, 100 keys: the first sees nothing
    q4[0, 1] = 0.0
    k4 = k[:, :100].clone()
    assert bool(nso.qk_max_logits(q4, k4).isfinite().all())


def test_accumulates_over_micro_batches_and_feeds_qk_clip():
    """Two micro-batches' logits kept in one buffer, then QK-Clip with them: the
    clipped heads and weights are the reference's."""
    import newton_schulz_orthogonalized_amd as nso
    hq, hk, d, dm, s = 4, 2, 64, 96, 130
    wq = as_dtype(host_normal((hq * d, dm), 88000), BF).cuda()
    wk = as_dtype(host_normal((hk * d, dm), 88001), BF).cuda()
    out = torch.zeros(hq, device="cuda")
    best = np.zeros(hq)
    for mb in range(2):
        x = as_dtype(host_normal((2 * s, dm), 88010 + mb), FP).cuda()
        q = (x @ wq.float().t()).to(BF).view(2, s, hq, d)
        k = (x @ wk.float().t()).to(BF).view(2, s, hk, d)
        nso.qk_max_logits(q, k, out=out, accumulate=True)
        torch.cuda.synchronize()
        one, mag = F.qk_max_logits_ref(_dense(q, k), 2, d ** -0.5, True)
        best = np.maximum(best, one)
        assert np.all(np.abs(to_np(out) - best) <= (d + 2) * 2.0 ** -23 * np.maximum(mag, best) * 2)
    tau = float(np.sort(best)[1:3].mean())       # clips two heads
    ml = to_np(out).astype(np.float32)
    q_ref, k_ref, gamma = O.qk_clip_ref(to_np(wq), to_np(wk), ml, q_heads=hq, k_heads=hk, tau=tau)
    assert int((np.asarray(gamma) < 1).sum()) == 2
    nso.qk_clip([wq], [wk], [out], q_heads=hq, k_heads=hk, tau=tau)
    torch.cuda.synchronize()
    assert np.array_equal(to_np(wq), O.bf16_round(q_ref)) and np.array_equal(to_np(wk), O.bf16_round(k_ref))


def test_empty_calls():
    import newton_schulz_orthogonalized_amd as nso
    for shape in ((0, 5), (2, 0)):
        q = torch.zeros(*shape, 3, 64, device="cuda", dtype=BF)
        assert nso.qk_max_logits(q, q).tolist() == [0.0] * 3
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.zeros(7, 3, 64, device="cuda", dtype=BF)
    assert nso.qk_max_logits(q, q, cu_seqlens=cu).tolist() == [0.0] * 3


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 72), (BF, 50), (BF, 256), (FP, 64), (FP, 33)])
def test_heads_of_few_keys(dtype, d):
    """Calls so short that a workgroup takes a whole head: sequences of lengths 0
    and 1 among them, first, last and all empty, into fresh and kept maxima, and
    captured with lengths that change."""
    import newton_schulz_orthogonalized_amd as nso
    q, k = _qk(4, 30, 32, 6, 3, d, dtype, 89400 + d)
    print(f"[qkmax] few keys {dtype} {d}", flush=True)
    first = torch.full((6,), 0.25, device="cuda")
    out = torch.zeros(6, device="cuda")
    lens = torch.zeros(4, dtype=torch.int32, device="cuda")
    nso.qk_max_logits(q, k, lengths=lens, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nso.qk_max_logits(q, k, lengths=lens, out=out)
    for lq in ([0, 0, 0, 0], [0, 30, 0, 0], [1, 0, 0, 30], [0, 0, 0, 1], [30, 1, 17, 30]):
        lens.copy_(torch.tensor(lq, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for causal in (True, False):
            seqs = _dense(q, k, lq, lq)
            got = nso.qk_max_logits(q, k, causal=causal, lengths=lens)
            torch.cuda.synchronize()
            _agree(got, seqs, 2, d ** -0.5, causal, d)
            if causal:
                assert torch.equal(got, out)
            kept = nso.qk_max_logits(q, k, causal=causal, lengths=lens, out=first.clone(), accumulate=True)
            assert torch.equal(kept, torch.maximum(first, got))
    cu = torch.tensor([0, 0, 7, 7, 24], dtype=torch.int32, device="cuda")
    got = nso.qk_max_logits(q[0], k[0, :30], cu_seqlens=cu)
    torch.cuda.synchronize()
    _agree(got, [(to_np(q[0, a:b]), to_np(k[0, a:b])) for a, b in ((0, 7), (7, 24))], 2, d ** -0.5, True, d)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [50, 100, 190])
def test_rows_at_odd_addresses(d, dtype):
    """Rows that do not begin at 16-byte pieces, over many query and key tiles."""
    import newton_schulz_orthogonalized_amd as nso
    q, k = _qk(2, 700, 650, 4, 2, d, dtype, 89500 + d)
    for causal in (True, False):
        got = nso.qk_max_logits(q, k, causal=causal)
        torch.cuda.synchronize()
        _agree(got, _dense(q, k), 2, d ** -0.5, causal, d)


@pytest.mark.parametrize("batch", [1, 2, 63, 64, 65, 130, 4097])
def test_numbers_of_sequences(batch):
    """Padded and packed sequences of unlike lengths, empty ones among them, in
    fresh and kept maxima."""
    import newton_schulz_orthogonalized_amd as nso
    d, most = 32, 300 if batch < 200 else 5
    lens = np.clip(np.abs(host_normal((batch,), 89700 + batch)) * most / 2, 0, most).astype(int).tolist()
    lens[-1] = most - 1
    kept = torch.full((4,), 3.0, device="cuda")
    edges = np.concatenate([[0], np.cumsum(lens)])
    cu = torch.tensor(edges, dtype=torch.int32, device="cuda")
    q, k = _qk(1, int(edges[-1]), int(edges[-1]), 4, 2, d, BF, 89800)
    q, k = q[0], k[0]
    got = nso.qk_max_logits(q, k, cu_seqlens=cu)
    both = nso.qk_max_logits(q, k, cu_seqlens=cu, out=kept.clone(), accumulate=True)
    torch.cuda.synchronize()
    _agree(got, [(to_np(q[a:b]), to_np(k[a:b])) for a, b in zip(edges[:-1], edges[1:])], 2, d ** -0.5, True, d)
    assert torch.equal(both, torch.maximum(kept, got))
    q, k = _qk(batch, most, most, 4, 2, d, BF, 89900)
    t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = nso.qk_max_logits(q, k, lengths=t)
    both = nso.qk_max_logits(q, k, lengths=t, out=kept.clone(), accumulate=True)
    torch.cuda.synchronize()
    _agree(got, _dense(q, k, lens, lens), 2, d ** -0.5, True, d)
    assert torch.equal(both, torch.maximum(kept, got))
    got = nso.qk_max_logits(q, k, causal=False)
    both = nso.qk_max_logits(q, k, causal=False, out=kept.clone(), accumulate=True)
    torch.cuda.synchronize()
    _agree(got, _dense(q, k), 2, d ** -0.5, False, d)
    assert torch.equal(both, torch.maximum(kept, got))


def test_more_workgroups_than_tiles():
    """Runs of the work that end before, in and behind a head's first tile."""
    import newton_schulz_orthogonalized_amd as nso
    for n, hq in ((33, 511), (65, 97), (200, 65), (257, 40), (300, 13)):
        q, k = _qk(1, n, n, hq, 1, 64, BF, 89600 + n)
        got = nso.qk_max_logits(q, k)
        torch.cuda.synchronize()
        _agree(got, _dense(q, k), hq, 0.125, True, 64)


def test_long_sequence_against_blocks():
    """A long sequence with many key blocks for each query block."""
    import newton_schulz_orthogonalized_amd as nso
    q, k = _qk(1, 3000, 3000, 2, 1, 128, BF, 89000)
    got = nso.qk_max_logits(q, k)
    torch.cuda.synchronize()
    _agree(got, _dense(q, k), 2, 128 ** -0.5, True, 128)


def test_many_short_sequences_and_streams():
    import newton_schulz_orthogonalized_amd as nso
    q, k = _qk(700, 3, 3, 2, 2, 32, BF, 89100)
    a = nso.qk_max_logits(q, k)
    _agree(a, _dense(q, k), 1, 32 ** -0.5, True, 32)
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i in range(4):
        st[i % 2].wait_stream(torch.cuda.current_stream())
        got.append(nso.qk_max_logits(q, k, stream=st[i % 2]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, g) for g in got)


def test_captured_and_replayed():
    import newton_schulz_orthogonalized_amd as nso
    q, k = _qk(2, 333, 333, 4, 2, 64, BF, 89200)
    lens = torch.tensor([333, 100], dtype=torch.int32, device="cuda")
    out = torch.zeros(4, device="cuda")
    nso.qk_max_logits(q, k, lengths=lens, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nso.qk_max_logits(q, k, lengths=lens, out=out)
    for r in range(4):
        q.mul_(0.75)
        lens.copy_(torch.tensor([50 * r + 1, 333 - r], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, nso.qk_max_logits(q, k, lengths=lens)), r


def test_refusals_on_the_gpu():
    import newton_schulz_orthogonalized_amd as nso
    from newton_schulz_orthogonalized_amd import _lib
    q, k = _qk(1, 8, 8, 3, 2, 16, BF, 89300)
    with pytest.raises(_lib.MuonError):
        nso.qk_max_logits(q, k)                        # 2 does not divide 3
    with pytest.raises(_lib.MuonError):
        nso.qk_max_logits(q, q, scale=float("inf"))
    with pytest.raises(ValueError):
        nso.qk_max_logits(q, q.cpu())
    with pytest.raises(ValueError):
        nso.qk_max_logits(q.transpose(2, 3), q.transpose(2, 3))
    with pytest.raises(TypeError):
        nso.qk_max_logits(q.half(), q.half())


def _profiled(call):
    from newton_schulz_orthogonalized_amd import _lib
    _lib.mu_profile_enable(True)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        _lib.mu_profile_enable(False)
    return _lib.mu_profile_read(_lib.MU_K_QKMAX)


def test_profiled_operations_are_those_of_visible_pairs():
    """Dense calls report 2 dim operations a visible pair and query head; with
    lengths on the device the pairs are unknown and none are reported."""
    import newton_schulz_orthogonalized_amd as nso
    for nq, nk in ((300, 300), (200, 333), (333, 200), (1, 70)):
        q, k = _qk(3, nq, nk, 4, 2, 64, BF, 90100)
        for causal in (True, False):
            seen = np.ones((nq, nk)) if not causal else np.arange(nk)[None, :] <= np.arange(nq)[:, None] + nk - nq
            p = _profiled(lambda: nso.qk_max_logits(q, k, causal=causal))
            assert p["flops"] == 2.0 * 3 * 4 * 64 * seen.sum() and p["ms"] > 0, (nq, nk, causal)
            assert p["bytes"] == 2.0 * 64 * 3 * (nq * 4 + nk * 2)
    q, k = _qk(1, 500, 500, 4, 2, 64, BF, 90200)
    cu = torch.tensor([0, 100, 500], dtype=torch.int32, device="cuda")
    for call in (lambda: nso.qk_max_logits(q[0], k[0], cu_seqlens=cu), lambda: nso.qk_max_logits(q, k, lengths=cu[1:2])):
        p = _profiled(call)
        assert p["flops"] == 0.0 and p["bytes"] == 2.0 * 64 * 500 * 6


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [16, 32, 40, 64, 80, 96, 128, 160, 192, 256])
def test_long_runs_of_every_width(d, dtype):
    """So many tiles for each workgroup that every slot of the ring is filled
    again and read: against float64 products (on the GPU, a head at a time), and
    single large logits, each at its own key and column, nothing else in sight."""
    import newton_schulz_orthogonalized_amd as nso
    print(f"[qkmax] long runs {dtype} {d}", flush=True)
    n, hq, hk = 2050, 8, 2
    q, k = _qk(1, n, n, hq, hk, d, dtype, 90300 + d)
    for causal in (True, False):
        got = nso.qk_max_logits(q, k, causal=causal)
        torch.cuda.synchronize()
        for h in range(hq):
            a, b = q[0, :, h].double(), k[0, :, h * hk // hq].double().t().contiguous()
            s, mag = (a @ b).abs(), a.abs() @ b.abs()
            if causal:
                s, mag = s.tril(), mag.tril()
            off = abs(float(got[h]) - float(s.max()) * d ** -0.5)
            assert off <= (d + 2) * 2.0 ** -23 * float(mag.max()) * d ** -0.5, (causal, h)
    q.zero_(), k.zero_()
    for step in range(24):
        j, h = 85 * step + step % 31, step % hq          # keys all along, at every place of a tile
        i, c = min(n - 1, j + (step * 37) % 500), (step * 29) % d
        q[0, i, h, c], k[0, j, h * hk // hq, c] = -3.0, 5.0
        for causal in (True, False):
            got = nso.qk_max_logits(q, k, causal=causal, scale=1.0).tolist()
            assert got == [15.0 if x == h else 0.0 for x in range(hq)], (causal, i, j, c)
        q[0, i, h, c], k[0, j, h * hk // hq, c] = 0.0, 0.0
