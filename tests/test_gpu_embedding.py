"""GPU parity of the embedding lookup and its gradient against a float64
reference.

Tolerances: a lookup is one float32 product rounded to its type, compared bit
for bit. A gradient row is a float32 sum of n rows in some order, off by at
most (n - 1) * 2^-24 of the sum of magnitudes (to first order), one more product
(scale) and, accumulating, one more sum, and a rounding to its type (bfloat16 2^-8).
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
ULP = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    import newton_schulz_orthogonalized_amd  # noqa: F401  (fails loudly without the library)
    yield


def _tokens(kind, n, vocab, seed):
    r = np.random.default_rng(seed)
    if kind == "uniform":
        return r.integers(0, vocab, n)
    if kind == "skewed":   # frequency about 1 / rank
        return np.minimum((np.exp(r.random(n) * np.log(vocab + 1)) - 1).astype(np.int64), vocab - 1)
    if kind == "one":
        return np.full(n, vocab - 1)
    if kind == "outside":
        t = r.integers(0, vocab, n)
        t[::3] = r.choice([-1, -100, vocab, vocab + 5, 2 ** 31 - 1], t[::3].size)
        return t
    if kind == "sorted":
        return np.sort(r.integers(0, vocab, n))
    raise ValueError(kind)


def _check_grad(tok, vocab, dim, row_t, grad_t, seed, scale=1.0, padding=None, accumulate=False, bits=64, shape=None):
    import newton_schulz_orthogonalized_amd as nso
    rows = as_dtype(host_normal((tok.size, dim), seed), row_t).cuda()
    t = torch.from_numpy(np.asarray(tok, np.int64)).to(torch.int64 if bits == 64 else torch.int32).cuda()
    if shape is not None:
        t, rows = t.view(shape), rows.view(*shape, dim)
    base = None
    if accumulate:
        out = as_dtype(host_normal((vocab, dim), seed + 1), grad_t).cuda()
        base = to_np(out)
    else:
        out = torch.full((vocab, dim), float("nan"), dtype=grad_t, device="cuda")   # every row is written
    nso.embedding_grad(t, rows, vocab, scale=scale, padding_idx=padding, out=out, accumulate=accumulate)
    torch.cuda.synchronize()
    g, mag, n = F.embedding_grad_ref(tok, to_np(rows).reshape(tok.size, dim), vocab, scale, padding, base)
    half = ULP if grad_t == FP else 2.0 ** -8
    bound = (np.maximum(n - 1, 0)[:, None] + 1) * ULP * 1.01 * mag + half * np.abs(g)
    if accumulate:
        bound = bound + ULP * (np.abs(base) + mag) + half * (n[:, None] + 1) * ULP * mag
    else:
        bound = bound + half * (n[:, None] + 1) * ULP * mag
    got = to_np(out)
    bad = ~(np.abs(got - g) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], g[bad][:5])
    untouched = n == 0
    assert np.array_equal(got[untouched], np.zeros_like(g)[untouched] if base is None else base[untouched])
    return out


LOOKUPS = [(1, 1, 1), (1, 100, 64), (5, 7, 3), (33, 50, 8), (64, 129, 513), (1000, 97, 768), (300, 1000, 4096), (17, 11, 8200)]


@pytest.mark.parametrize("bits", [32, 64])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,vocab,dim", LOOKUPS)
def test_lookup(n, vocab, dim, dtype, bits):
    import newton_schulz_orthogonalized_amd as nso
    tok = _tokens("outside" if n > 3 else "uniform", n, vocab, n)
    w = as_dtype(host_normal((vocab, dim), 70000 + n, 0.02), dtype).cuda()
    t = torch.from_numpy(tok).to(torch.int64 if bits == 64 else torch.int32).cuda()
    for scale in (1.0, 0.3, -64.0):
        out = nso.embedding(t, w, scale=scale)
        torch.cuda.synchronize()
        want = F.embedding_ref(tok, to_np(w).astype(np.float32), np.float32(scale)).astype(np.float32)
        ok = (tok >= 0) & (tok < vocab)
        exp = O.bf16_round(want[ok]) if dtype == BF else want[ok].astype(np.float64)
        got = to_np(out)
        assert np.array_equal(got[ok], exp), scale
        assert np.isnan(got[~ok]).all()


@pytest.mark.parametrize("dtype,dim", [(BF, 4096), (BF, 4101), (FP, 2048), (FP, 2051)])
def test_lookups_beyond_the_caches(dtype, dim):
    """Outputs just below and above the size from which they are written past
    the caches (128 MB), guarded at both ends; the rows bit for bit, or one
    float32 product and rounding; a token outside the table is a row of NaN."""
    import newton_schulz_orthogonalized_amd as nso
    w = as_dtype(host_normal((37, dim), 70500), dtype).cuda()
    size = dim * w.element_size()
    for n in ((128 << 20) // size - 1, (128 << 20) // size + 1, (300 << 20) // size):
        print(f"[lookup] {n} x {dim} {dtype}", flush=True)
        tok = (torch.arange(n, device="cuda") * 7919) % 37
        buf = torch.full((n * dim + 16,), 7.0, dtype=dtype, device="cuda")
        out = buf[8:-8].view(n, dim)
        for scale in (1.0, -0.3):
            nso.embedding(tok, w, scale=scale, out=out)
            assert torch.equal(out, (w if scale == 1.0 else (w.float() * scale).to(dtype))[tok])
        tok[n // 2], tok[n - 1] = 37, -1
        nso.embedding(tok, w, out=out)
        bad = out.isnan().any(1)
        assert int(bad.sum()) == 2 and bool(out[n // 2].isnan().all()) and bool(out[n - 1].isnan().all())
        assert bool((buf[:8] == 7).all()) and bool((buf[-8:] == 7).all())


def test_lookup_copies_every_bit_and_takes_any_alignment():
    """Scale 1 copies infinities, NaN payloads and negative zeros; views that
    start at odd elements; tokens of any shape; an output buffer of one's own."""
    import newton_schulz_orthogonalized_amd as nso
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    for dim in (64, 100, 1):
        flat = bits[:65536 // dim * dim].cuda()
        buf = torch.zeros(flat.numel() + 3, dtype=torch.int16, device="cuda")
        buf[3:] = flat
        w = buf[3:].view(BF).view(-1, dim)
        tok = torch.randperm(w.shape[0], device="cuda").view(-1, 1)
        out = torch.zeros(tok.numel() * dim + 1, dtype=BF, device="cuda")[1:].view(*tok.shape, dim)
        nso.embedding(tok, w, out=out)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), w.view(torch.int16)[tok])


@pytest.mark.parametrize("bits", [32, 64])
@pytest.mark.parametrize("row_t,grad_t", [(BF, BF), (BF, FP), (FP, FP), (FP, BF)])
@pytest.mark.parametrize("kind", ["uniform", "skewed", "one", "outside", "sorted"])
@pytest.mark.parametrize("n,vocab,dim", [(1, 1, 1), (7, 3, 5), (64, 200, 64), (1025, 300, 100), (3000, 50, 513)])
def test_gradient(n, vocab, dim, kind, row_t, grad_t, bits):
    print(f"[rowgrad] {n} {vocab} {dim} {kind} {row_t} {grad_t} {bits}", flush=True)
    _check_grad(_tokens(kind, n, vocab, n + dim), vocab, dim, row_t, grad_t, 71000, scale=0.5, bits=bits)


@pytest.mark.parametrize("n,vocab,dim", [
    (8192, 5000, 8), (8192, 1 << 19, 2), (8193, 1 << 19, 2), (12288, 3000, 8), (12289, 3000, 8), (16383, 5000, 16),
    (16384, 300000, 8), (16385, 5000, 24), (40000, 70000, 8), (70000, 9, 16), (100003, 131072, 3), (20000, 1 << 19, 2),
    (33000, 1 << 20, 1), (131073, 5000, 2), (262144, 300, 600), (262145, 5000, 2), (524288, 40000, 3), (524289, 40000, 3), (2200001, 70, 1)])
def test_gradient_of_long_batches_and_large_tables(n, vocab, dim):
    print(f"[rowgrad] long {n} {vocab} {dim}", flush=True)
    for kind in ("skewed", "outside", "one") if n < 1 << 20 else ("outside",):
        _check_grad(_tokens(kind, n, vocab, n), vocab, dim, BF, FP, 72000)


@pytest.mark.parametrize("n,vocab,dim,grad_t", [
    (1, 300001, 256, BF), (100, 100003, 513, FP), (9000, 128256, 1024, BF), (20000, 50257, 2048, FP), (70000, 300000, 200, BF),
    (300000, 2000003, 64, BF), (64, 70, 1 << 20, BF), (5000, 5000000, 17, FP)])
def test_gradients_of_large_tables(n, vocab, dim, grad_t):
    """Tables whose zeros take part of the call's time: every row that no token
    names is zero, the others are those of a call that adds to zeros."""
    import newton_schulz_orthogonalized_amd as nso
    print(f"[rowgrad] table {n} {vocab} {dim}", flush=True)
    rows = as_dtype(host_normal((n, 1), 74300), BF).cuda() * torch.arange(1, dim + 1, device="cuda").to(BF)
    for kind in ("skewed", "outside", "sorted", "one"):
        t = torch.from_numpy(_tokens(kind, n, vocab, n)).cuda()
        got = torch.full((vocab, dim), float("nan"), dtype=grad_t, device="cuda")
        guard = torch.full((vocab * dim + 64,), -3.0, dtype=grad_t, device="cuda")
        for out in (got, guard[32:-32].view(vocab, dim)):
            nso.embedding_grad(t, rows, vocab, out=out, scale=0.5, padding_idx=1)
        want = nso.embedding_grad(t, rows, vocab, out=torch.zeros_like(got), scale=0.5, padding_idx=1, accumulate=True)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(got, guard[32:-32].view(vocab, dim)), kind
        assert bool((guard[:32] == -3).all()) and bool((guard[-32:] == -3).all())
        named = torch.zeros(vocab, dtype=torch.bool, device="cuda")
        named[t[(t >= 0) & (t < vocab) & (t != 1)]] = True
        assert not bool(got[~named].any()) and bool(got[named].any()) == bool(named.any())


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("padding", [None, 0, 40])
@pytest.mark.parametrize("grad_t", [BF, FP])
def test_padding_accumulation_and_batches(grad_t, padding, accumulate):
    tok = _tokens("skewed", 6 * 50, 41, 5)
    _check_grad(tok, 41, 72, BF, grad_t, 73000, scale=-2.5, padding=padding, accumulate=accumulate, shape=(6, 50))


def test_wide_rows():
    _check_grad(_tokens("skewed", 700, 60, 1), 60, 4096, BF, BF, 74000)
    _check_grad(_tokens("skewed", 90, 12, 1), 12, 20001, FP, FP, 74100)


def test_no_tokens_and_nothing_valid():
    import newton_schulz_orthogonalized_amd as nso
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    g = nso.embedding_grad(none, torch.zeros(0, 16, device="cuda"), 9)
    assert g.shape == (9, 16) and bool((g == 0).all())
    keep = torch.ones(9, 16, device="cuda")
    nso.embedding_grad(none, torch.zeros(0, 16, device="cuda"), 9, out=keep, accumulate=True)
    assert bool((keep == 1).all())
    assert nso.embedding(none, keep).shape == (0, 16)
    _check_grad(np.full(300, -100), 9, 16, FP, FP, 75000)
    _check_grad(np.full(300, 4), 9, 16, FP, FP, 75000, padding=4)


def test_padding_rows_of_nan_do_not_matter():
    import newton_schulz_orthogonalized_amd as nso
    tok = torch.tensor([1, 2, -5, 1, 3], device="cuda")
    rows = torch.ones(5, 40, device="cuda")
    rows[1], rows[2] = float("nan"), float("inf")
    g = nso.embedding_grad(tok, rows, 5, padding_idx=2)
    assert g[:, 0].tolist() == [0.0, 2.0, 0.0, 1.0, 0.0] and bool(g.isfinite().all())
    rows[0, 7] = float("nan")
    g = nso.embedding_grad(tok, rows, 5, padding_idx=2)
    assert bool(g[1, 7].isnan()) and int(g.isnan().sum()) == 1


def test_rows_behind_the_buffers_are_left_alone():
    import newton_schulz_orthogonalized_amd as nso
    for dim in (5, 64, 520):
        buf = torch.full((12 * dim,), 7.0, dtype=BF, device="cuda")
        nso.embedding_grad(torch.tensor([0, 3, 9], device="cuda"), torch.ones(3, dim, device="cuda"), 10,
                           out=buf[dim:11 * dim].view(10, dim))
        out = torch.full((5 * dim,), 7.0, dtype=FP, device="cuda")
        nso.embedding(torch.tensor([0, 3, 9], device="cuda"), torch.ones(10, dim, device="cuda"),
                      out=out[dim:4 * dim].view(3, dim))
        torch.cuda.synchronize()
        assert bool((buf[:dim] == 7).all()) and bool((buf[11 * dim:] == 7).all())
        assert bool((out[:dim] == 7).all()) and bool((out[4 * dim:] == 7).all())


def test_same_bits_again_and_on_other_streams():
    """Two calls at once on two streams, each with its own workspace, and again."""
    import newton_schulz_orthogonalized_amd as nso
    for n in (5000, 50000):
        tok = torch.from_numpy(_tokens("skewed", n, 1000, 3)).cuda()
        rows = as_dtype(host_normal((n, 96), 76000), BF).cuda()
        ref = nso.embedding_grad(tok, rows, 1000, dtype=FP)
        torch.cuda.synchronize()
        st = [torch.cuda.Stream(), torch.cuda.Stream()]
        got = []
        for k in range(6):
            st[k % 2].wait_stream(torch.cuda.current_stream())
            got.append(nso.embedding_grad(tok, rows, 1000, dtype=FP, stream=st[k % 2]))
        torch.cuda.synchronize()
        assert all(torch.equal(ref, g) for g in got)


def test_autograd():
    """Gradients through the module path: against the reference, of an expanded
    upstream gradient, twice over (accumulated by autograd), and against
    differences of the loss."""
    import newton_schulz_orthogonalized_amd as nso
    w = as_dtype(host_normal((30, 12), 77000), FP).cuda().requires_grad_()
    tok = torch.from_numpy(_tokens("skewed", 40, 30, 9).reshape(5, 8)).cuda()
    up = as_dtype(host_normal((5, 8, 12), 77001), FP).cuda()
    y = nso.embedding(tok, w, scale=3.0, padding_idx=1)
    y.backward(up)
    g, mag, n = F.embedding_grad_ref(to_np(tok).astype(int), to_np(up).reshape(40, 12), 30, 3.0, 1)
    assert np.all(np.abs(to_np(w.grad) - g) <= (n[:, None] + 2) * ULP * 1.01 * mag)
    first = w.grad.clone()
    nso.embedding(tok, w, scale=3.0, padding_idx=1).backward(up)
    assert torch.equal(w.grad, first * 2)
    w.grad = None
    nso.embedding(tok, w).sum().backward()          # upstream gradient of stride 0
    _, _, n = F.embedding_grad_ref(to_np(tok).astype(int), np.ones((40, 12)), 30)
    assert np.array_equal(to_np(w.grad), np.repeat(n[:, None], 12, 1).astype(float))
    # differences: the loss is linear in w, so a step of 1 gives the gradient up
    # to the rounding of sums of 40 * 12 products
    w.grad = None
    loss = lambda x: (nso.embedding(tok, x, scale=3.0).double() * up.double()).sum()  # noqa: E731
    loss(w).backward()
    v = int(tok[0, 0])
    d = w.detach().clone()
    d[v, 5] += 1.0
    with torch.no_grad():
        diff = float(loss(d) - loss(w))
    assert abs(diff - float(w.grad[v, 5])) <= 1e-4 * max(1.0, abs(diff))
    assert not nso.embedding(tok, w.detach()).requires_grad


def test_captured_and_replayed():
    """Lookup and gradient in one graph, replayed with new tokens, rows and
    weights between the program's own work; an eager graph of the same leaf
    lives meanwhile."""
    import newton_schulz_orthogonalized_amd as nso
    for n in (700, 20000):
        w = as_dtype(host_normal((500, 64), 78000), BF).cuda()
        leaf = w.clone().requires_grad_()
        tok = torch.from_numpy(_tokens("skewed", n, 500, 3)).cuda()
        up = as_dtype(host_normal((n, 64), 78001), BF).cuda()
        alive = nso.embedding(tok.clone(), leaf)
        out = torch.zeros(n, 64, dtype=BF, device="cuda")
        grad = torch.zeros(500, 64, dtype=FP, device="cuda")
        nso.embedding(tok, w, out=out)
        nso.embedding_grad(tok, up, 500, out=grad)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            nso.embedding(tok, w, scale=2.0, out=out)
            nso.embedding_grad(tok, up, 500, out=grad)
        for k in range(4):
            tok.copy_(torch.from_numpy(_tokens("skewed", n, 500, 10 + k)))
            up.mul_(-0.5)
            w.add_(0.25)
            graph.replay()
            torch.cuda.synchronize()
            o2 = nso.embedding(tok, w, scale=2.0)
            g2 = nso.embedding_grad(tok, up, 500, dtype=FP)
            torch.cuda.synchronize()
            assert torch.equal(out, o2) and torch.equal(grad, g2), (n, k)
        alive.sum().backward()
        assert leaf.grad is not None


def test_refusals_on_the_gpu():
    import newton_schulz_orthogonalized_amd as nso
    from newton_schulz_orthogonalized_amd import _lib
    w = torch.ones(10, 8, device="cuda")
    tok = torch.zeros(10, dtype=torch.int64, device="cuda")
    with pytest.raises(_lib.MuonError) as e:
        nso.embedding(tok, w, out=w)
    assert e.value.status == _lib.MU_ERR_LAYOUT
    with pytest.raises(_lib.MuonError):
        nso.embedding_grad(tok, w, 10, out=w)
    with pytest.raises(_lib.MuonError):
        nso.embedding(tok, w, scale=float("nan"))
    with pytest.raises(ValueError):
        nso.embedding(tok.cpu(), w)
    with pytest.raises(ValueError):
        nso.embedding(tok, w.t())
    with pytest.raises(TypeError):
        nso.embedding(tok.float(), w)
    with pytest.raises(TypeError):
        nso.embedding(tok, w.half())
    torch.cuda.synchronize()
    assert bool((w == 1).all())


def test_profiled_bytes_of_the_gradient():
    """Many tokens on few rows: the rows are read once, the gradient's zeros and
    its at most `vocab` sums written once each."""
    import newton_schulz_orthogonalized_amd as nso
    from newton_schulz_orthogonalized_amd import _lib
    n, vocab, dim = 4000, 10, 256
    tok = torch.from_numpy(_tokens("uniform", n, vocab, 1)).cuda()
    rows = torch.ones(n, dim, dtype=BF, device="cuda")
    for accumulate in (False, True):
        out = torch.zeros(vocab, dim, device="cuda")
        _lib.mu_profile_enable(True)
        try:
            nso.embedding_grad(tok, rows, vocab, out=out, accumulate=accumulate)
            torch.cuda.synchronize()
        finally:
            _lib.mu_profile_enable(False)
        p = _lib.mu_profile_read(_lib.MU_K_ROWGRAD)
        # tokens 8 bytes, sorted words 8 written and read
        assert p["bytes"] == n * (8 + 8 + 8) + n * dim * 2 + 2 * vocab * dim * 4 and p["launches"] == 3


@pytest.mark.parametrize("grad_t,accumulate", [(FP, False), (FP, True), (BF, False)])
@pytest.mark.parametrize("n,vocab,dim", [(12289, 3, 24), (70000, 9, 16), (100003, 5000, 3), (131073, 4, 2), (262144, 300, 600),
                                         (524289, 40000, 3), (65536, 7, 1030), (2200001, 70, 1)])
def test_every_token_of_long_batches_counts(n, vocab, dim, grad_t, accumulate):
    """Small positive integers, whose float32 sums are exact in any order (all
    below 2^24), so one row left out, counted twice or put elsewhere shows: runs
    over thousands of chunks and of chunks longer than 16, joined by quarters."""
    import newton_schulz_orthogonalized_amd as nso
    print(f"[rowgrad] exact {n} {vocab} {dim} {grad_t} {accumulate}", flush=True)
    rows = (np.arange(n)[:, None] * (np.arange(dim)[None, :] + 3) % 5 + 1).astype(np.float32)
    assert 5 * n + 9 < 2 ** 24
    r = torch.from_numpy(rows).to(BF).cuda()
    for kind in ("one", "skewed", "sorted", "outside"):
        tok = _tokens(kind, n, vocab, n + 1)
        t = torch.from_numpy(tok).cuda()
        base = np.zeros((vocab, dim))
        out = torch.full((vocab, dim), float("nan"), dtype=grad_t, device="cuda")
        if accumulate:
            base = (np.arange(vocab * dim).reshape(vocab, dim) % 9).astype(np.float64)
            out.copy_(torch.from_numpy(base))
        nso.embedding_grad(t, r, vocab, out=out, accumulate=accumulate)
        torch.cuda.synchronize()
        ok = (tok >= 0) & (tok < vocab)
        want = base + np.stack([np.bincount(tok[ok], weights=rows[ok, c], minlength=vocab) for c in range(dim)], 1)
        got = to_np(out)
        assert np.array_equal(got, O.bf16_round(want) if grad_t == BF else want), kind
