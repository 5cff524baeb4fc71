"""GPU parity of the global gradient norm and clipping against a float64
reference, alone and inside the optimizer steps.

Tolerances: the norm is a float64 sum rounded once to float32 (2^-24 relative,
plus the float64 rounding); the factor likewise; a scaled gradient is one
float32 product of that factor (2 * 2^-24) rounded to its type (bfloat16 2^-8).
"""

import math

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


def _list(sizes, types, seed, std=1e-3, shift=0):
    out = []
    for i, (n, t) in enumerate(zip(sizes, types)):
        shape = n if isinstance(n, tuple) else (n,)
        buf = torch.zeros(math.prod(shape) + shift, dtype=t, device="cuda")
        v = buf[shift:].view(shape)
        v.copy_(as_dtype(host_normal(shape, seed + i, std), t))
        out.append(v)
    return out


def _check(grads, max_norm, outs, eps=1e-6):
    """Norm, factor and outputs of clip_grads against the reference."""
    import newton_schulz_orthogonalized_amd as nso
    host = [to_np(g) for g in grads]
    scale = torch.full((), -1.0, device="cuda")
    norm = nso.clip_grads(grads, max_norm, outs=outs, eps=eps, scale_out=scale)
    torch.cuda.synchronize()
    want = F.grad_norm_ref(host)
    # the bounds are float32 arguments: 0.2524.. itself is up to 2^-24 away from the one the call takes
    c = F.clip_scale_ref(want, float(np.float32(max_norm)), float(np.float32(eps)))
    assert abs(float(norm) - want) <= want * ULP * 1.001
    assert abs(float(scale) - c) <= c * ULP * 1.001
    for h, o in zip(host, grads if outs is None else outs):
        half = ULP if o.dtype == FP else 2.0 ** -8
        ref = c * h
        if outs is None and c == 1.0:
            assert np.array_equal(to_np(o), h)
        else:
            assert np.all(np.abs(to_np(o) - ref) <= np.abs(ref) * (half + 2.1 * ULP))
    return float(norm)


SIZES = [1, 7, 8, 9, 255, 2048, 8191, 8192, 8193, 16385, (33, 77), (128, 256), 100003, 0]


@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("types", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("where", ["in_place", "same", "other"])
def test_clip_of_odd_sizes_and_alignments(types, where, shift):
    print(f"[clip] {types} {where} shift {shift}", flush=True)
    ts = [{"f32": FP, "bf16": BF, "mixed": (FP, BF)[i % 2]}[types] for i in range(len(SIZES))]
    g = _list(SIZES, ts, 50000, shift=shift)
    if where == "in_place":
        outs = None
    else:
        to = ts if where == "same" else [BF if t is FP else FP for t in ts]
        outs = _list(SIZES, to, 51000, shift=shift)
    n = _check(g, 0.1, outs)
    assert n > 0.1


@pytest.mark.parametrize("size", [1, 64, 8192, 70000])
def test_below_the_bound_keeps_the_gradients(size):
    g = _list([size], [BF], 52000)
    _check(g, 1e3, None)
    o = _list([size], [FP], 52001)
    _check(g, 1e3, o)


@pytest.mark.parametrize("chunks", [11, 12, 13, 31, 32, 33, 34])
def test_around_the_sizes_of_one_workgroup(chunks):
    import newton_schulz_orthogonalized_amd as nso
    for sizes in ([8192 * chunks], [8192 * chunks - 5], [5] + [8192] * (chunks - 1), [8192 * (chunks - 1) - 1, 3, 1]):
        g = _list(sizes, [(FP, BF)[i % 2] for i in range(len(sizes))], 52100, shift=1)
        want = F.grad_norm_ref([to_np(x) for x in g])
        assert abs(float(nso.grad_norm(g)) - want) <= want * ULP * 1.001
        _check(g, want / 2, _list(sizes, [FP] * len(sizes), 52200))
        _check(g, want / 2, None)


@pytest.mark.parametrize("types,where", [((FP, FP), "in_place"), ((FP, BF), "other"), ((BF, BF), "other")])
def test_lists_beyond_the_caches(types, where):
    """More than 256 MB, at odd elements and sizes; the reference on the GPU, in
    float64 for the norm, and the one float32 product and rounding exactly."""
    import newton_schulz_orthogonalized_amd as nso
    g = []
    for n in (8192, 50_000_001, 41_234_567, 7):
        x = torch.zeros(n + 3, dtype=types[0], device="cuda")[3:]
        i = torch.arange(n, device="cuda", dtype=torch.int64)
        x.copy_(((i * 7919) % 2003 - 1001).float() / 4096)
        g.append(x)
    want = math.sqrt(sum(float(x.double().square().sum()) for x in g))
    outs = None if where == "in_place" else [torch.zeros(x.numel() + 1, dtype=types[1], device="cuda")[1:] for x in g]
    keep = [x.clone() for x in g]
    scale = torch.zeros((), device="cuda")
    norm = nso.clip_grads(g, 3.0, outs=outs, scale_out=scale)
    torch.cuda.synchronize()
    assert abs(float(norm) - want) <= want * ULP * 1.001 and float(scale) < 1.0
    for k, x, o in zip(keep, g, g if outs is None else outs):
        assert torch.equal(o, (k.float() * scale).to(o.dtype))
        assert outs is None or torch.equal(x, k)


def test_norm_of_many_tensors_and_beyond_one_launch():
    """More tensors than one launch takes, single elements among them, and the
    same tensor twice (it counts twice)."""
    import newton_schulz_orthogonalized_amd as nso
    sizes = [1 + (i * 37) % 500 for i in range(517)]
    g = _list(sizes, [(FP, BF)[i % 3 == 0] for i in range(517)], 53000)
    want = F.grad_norm_ref([to_np(x) for x in g])
    assert abs(float(nso.grad_norm(g)) - want) <= want * ULP * 1.001
    _check(g, want / 3, _list(sizes, [FP] * 517, 54000))
    one = float(nso.grad_norm([g[5], g[5]]))
    assert abs(one - math.sqrt(2) * F.grad_norm_ref([to_np(g[5])])) <= one * 2 * ULP


@pytest.mark.parametrize("std", [1e-38, 1e-20, 1e20, 1e37])
def test_magnitudes_whose_squares_leave_float32(std):
    import newton_schulz_orthogonalized_amd as nso
    g = _list([1000, 30000], [FP, FP], 55000, std=std)
    want = F.grad_norm_ref([to_np(x) for x in g])
    scale = torch.zeros((), device="cuda")
    norm = float(nso.grad_norm(g, max_norm=1.0, scale_out=scale))
    # a norm of 2^128 (1 - 2^-25) or more is infinity in float32; the factor is formed from the float64 norm
    assert math.isinf(norm) if want >= 2.0 ** 128 * (1 - 2.0 ** -25) else abs(norm - want) <= want * ULP * 1.001
    c = F.clip_scale_ref(want, 1.0)
    assert abs(float(scale) - c) <= c * ULP * 1.001 + 2.0 ** -150   # half a step of the smallest float32


def test_zero_empty_and_not_finite():
    import newton_schulz_orthogonalized_amd as nso
    z = [torch.zeros(100, device="cuda"), torch.zeros(0, device="cuda", dtype=BF)]
    assert _check(z, 1.0, None) == 0.0
    assert _check(z, 0.0, None, eps=0.0) == 0.0
    assert float(nso.grad_norm([])) == 0.0 and float(nso.clip_grads([], 1.0)) == 0.0
    assert float(nso.grad_norm([z[1]])) == 0.0
    for bad, where in ((float("nan"), 17), (float("inf"), 9000), (-float("inf"), 0)):
        g = torch.ones(20000, device="cuda", dtype=BF)
        g[where] = bad
        o = torch.zeros(20000, device="cuda")
        scale = torch.zeros((), device="cuda")
        norm = float(nso.clip_grads([g], 1.0, outs=[o], scale_out=scale))
        if math.isnan(bad):
            assert math.isnan(norm) and math.isnan(float(scale)) and bool(o.isnan().all())
        else:
            assert math.isinf(norm) and float(scale) == 0.0
            assert bool(o[where].isnan()) and float(o.nan_to_num(0.0).abs().max()) == 0.0   # 0 * inf, 0 * 1


@pytest.mark.parametrize("n", [100, 8192 * 40])   # one launch, several
def test_no_bound_keeps_the_gradients(n):
    """max_norm = inf, grad_norm's default: the factor is 1 for any norm but NaN,
    an infinite one too (infinity over infinity clips nothing)."""
    import newton_schulz_orthogonalized_amd as nso
    for bad in (0.0, 3.0, 1e30, float("inf"), -float("inf"), float("nan")):
        g = torch.ones(n, device="cuda")
        g[n // 2] = bad
        keep, scale, o = g.clone(), torch.full((), -1.0, device="cuda"), torch.zeros_like(g)
        norm = float(nso.grad_norm([g], scale_out=scale))
        assert math.isnan(float(scale)) if math.isnan(bad) else float(scale) == 1.0, bad
        assert math.isinf(norm) == math.isinf(bad) and math.isnan(norm) == math.isnan(bad)
        nso.clip_grads([g], math.inf, outs=[o])
        nso.clip_grads([g], math.inf)
        for x in (o, g):
            assert bool(x.isnan().all()) if math.isnan(bad) else torch.equal(x, keep), bad


def test_same_bits_again_and_on_another_stream():
    import newton_schulz_orthogonalized_amd as nso
    g = _list([200000, 77777, 5], [BF, FP, BF], 56000)
    a = nso.grad_norm(g)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    b = nso.grad_norm(g, stream=st)
    with torch.cuda.stream(st):
        c = nso.grad_norm(g)
    torch.cuda.synchronize()
    assert float(a) == float(b) == float(c)


def test_captured_and_replayed():
    """A graph of norm and clip follows the gradients' values at each replay."""
    import newton_schulz_orthogonalized_amd as nso
    sizes = [30000, 9, 123457] + [50] * 200
    types = [FP, BF, BF] + [FP] * 200
    g = _list(sizes, types, 57000)
    o = [torch.zeros_like(x) for x in g]
    norm, scale = torch.zeros((), device="cuda"), torch.zeros((), device="cuda")
    nso.clip_grads(g, 0.05, outs=o, norm_out=norm, scale_out=scale)   # warm
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nso.clip_grads(g, 0.05, outs=o, norm_out=norm, scale_out=scale)
    for k in range(4):
        for x in g:
            x.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        o2 = [torch.zeros_like(x) for x in g]
        n2 = nso.clip_grads(g, 0.05, outs=o2)
        torch.cuda.synchronize()
        assert float(norm) == float(n2), k
        assert all(torch.equal(a, b) for a, b in zip(o, o2)), k


def test_refusals_on_the_gpu():
    import newton_schulz_orthogonalized_amd as nso
    from newton_schulz_orthogonalized_amd import _lib
    x = torch.ones(64, device="cuda")
    for call in (lambda: nso.clip_grads([x, x], 1.0), lambda: nso.clip_grads([x], 1.0, outs=[x.view(BF)[:64]]),
                 lambda: nso.clip_grads([x[:32]], 1.0, outs=[x[16:48]])):
        with pytest.raises(_lib.MuonError) as e:
            call()
        assert e.value.status == _lib.MU_ERR_LAYOUT
    with pytest.raises(_lib.MuonError) as e:
        nso.grad_norm([x], workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert e.value.status == _lib.MU_ERR_WORKSPACE
    with pytest.raises(_lib.MuonError):
        nso.clip_grads([x], -1.0)
    with pytest.raises(ValueError):
        nso.grad_norm([x, torch.ones(4)])
    torch.cuda.synchronize()
    assert bool((x == 1).all())


# ---------------------------------------------------------------------------
# Inside the steps
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,precision", [(FP, "f32"), (BF, "bf16")])
def test_muon_step_with_a_factor(dtype, precision):
    """The step takes c * g in float32: bit for bit the step of gradients that
    hold c * g already (c a power of two, exact in both types), and with c = 1
    the plain step; a factor read at launch follows its tensor."""
    import newton_schulz_orthogonalized_amd as nso
    shapes = [(96, 160), (160, 96), (33, 77)]
    c = torch.ones((), device="cuda")
    runs = {}
    for name in ("plain", "one", "half", "scaled"):
        w = [as_dtype(host_normal(s, 58000 + i, 0.02), dtype).cuda() for i, s in enumerate(shapes)]
        g = [as_dtype(host_normal(s, 58100 + i, 1e-3), dtype).cuda() for i, s in enumerate(shapes)]
        m = [as_dtype(host_normal(s, 58200 + i, 1e-3), FP).cuda() for i, s in enumerate(shapes)]
        if name == "half":
            g = [x * 0.5 for x in g]
        for k in range(3):   # the third call replays a graph
            c.fill_(0.5 if name == "scaled" else 1.0)
            nso.muon_step(w, g, m, lr=0.02, weight_decay=0.01, precision=precision,
                          grad_scale=None if name in ("plain", "half") else c)
        torch.cuda.synchronize()
        runs[name] = (w, m)
    for a, b in (("plain", "one"), ("half", "scaled")):
        for x, y in zip(runs[a][0] + runs[a][1], runs[b][0] + runs[b][1]):
            assert torch.equal(x, y), (a, b)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_adamw_step_with_a_factor(dtype):
    import newton_schulz_orthogonalized_amd as nso
    sizes = [5, 8192, 70001, 131072]
    c = torch.full((), 0.3, device="cuda")

    def run(scale, grad_scale, steps=1):
        p = [as_dtype(host_normal(n, 59000 + i, 0.02), dtype).cuda() for i, n in enumerate(sizes)]
        g = [as_dtype(host_normal(n, 59100 + i, 1e-3) * scale, dtype).cuda() for i, n in enumerate(sizes)]
        m = [torch.zeros(n, device="cuda") for n in sizes]
        v = [torch.zeros(n, device="cuda") for n in sizes]
        h = [(to_np(a), to_np(b)) for a, b in zip(p, g)]
        nso.adamw_step(p, g, m, v, lr=1e-3, weight_decay=0.01, step=1, grad_scale=grad_scale)
        torch.cuda.synchronize()
        return p, m, v, h
    a = run(1.0, None)
    b = run(1.0, torch.ones((), device="cuda"))
    for x, y in zip(a[0] + a[1] + a[2], b[0] + b[1] + b[2]):
        assert torch.equal(x, y)
    p, m, v, h = run(1.0, c)
    cf = float(c)
    for i, n in enumerate(sizes):
        pr, mr, vr = O.adamw_ref(h[i][0], cf * h[i][1], np.zeros(n), np.zeros(n), lr=1e-3, weight_decay=0.01, beta1=0.9,
                                 beta2=0.95, eps=1e-8, step=1)
        # float32 chain: the product c g, (1 - beta) rounded, two products, a sum
        assert np.all(np.abs(to_np(m[i]) - mr) <= 8 * ULP * np.abs(mr) + 1e-45)
        assert np.all(np.abs(to_np(v[i]) - vr) <= 8 * ULP * np.abs(vr) + 1e-45)


class Tiny(torch.nn.Module):
    def __init__(self, vocab=101, d=64, sparse=False):
        super().__init__()
        self.wte = torch.nn.Embedding(vocab, d, sparse=sparse)
        self.a = torch.nn.Linear(d, 3 * d, bias=True)
        self.b = torch.nn.Linear(3 * d, d, bias=False)
        self.lm_head = torch.nn.Linear(d, vocab, bias=False)


def _model(sparse=False, dtype=FP):
    m = Tiny(sparse=sparse).to("cuda", dtype)
    for i, p in enumerate(m.parameters()):
        p.data.copy_(as_dtype(host_normal(tuple(p.shape), 60000 + i, 0.02), dtype))
    return m


def _opt(m, **kw):
    import newton_schulz_orthogonalized_amd as nso
    muon, adamw = nso.split_params(m)
    return nso.MuonAdamW([{"params": muon, "kind": "muon"}, {"params": adamw, "kind": "adamw"}], lr=0.02,
                         weight_decay=0.01, adamw_lr=3e-3, precision="f32", **kw)


def test_optimizer_clips_all_groups_together():
    """MuonAdamW(max_grad_norm): the norm over both groups, the clipped step
    equal bit for bit to the functional calls with that factor, p.grad kept."""
    import newton_schulz_orthogonalized_amd as nso
    a, b = _model(), _model()
    opt = _opt(a, max_grad_norm=0.05)
    muon, adamw = nso.split_params(b)
    mom = [torch.zeros_like(p) for p in muon]
    m1, m2 = [torch.zeros_like(p) for p in adamw], [torch.zeros_like(p) for p in adamw]
    for step in range(3):
        for i, (p, q) in enumerate(zip(a.parameters(), b.parameters())):
            g = as_dtype(host_normal(tuple(p.shape), 61000 + 10 * step + i, 1e-3 * (1 + step)), FP).cuda()
            p.grad, q.grad = g.clone(), g.clone()
        keep = [p.grad.clone() for p in a.parameters()]
        opt.step()
        scale = torch.zeros((), device="cuda")
        norm = nso.grad_norm([p.grad for p in muon + adamw], max_norm=0.05, scale_out=scale)
        nso.muon_step([p.data for p in muon], [p.grad for p in muon], mom, lr=0.02, weight_decay=0.01, precision="f32",
                      grad_scale=scale)
        nso.adamw_step([p.data for p in adamw], [p.grad for p in adamw], m1, m2, lr=3e-3, weight_decay=0.0, step=step + 1,
                       grad_scale=scale)
        torch.cuda.synchronize()
        assert float(opt.grad_norm) == float(norm) and float(scale) < 1.0
        assert all(torch.equal(p.grad, k) for p, k in zip(a.parameters(), keep))
        for (n, p), q in zip(a.named_parameters(), b.parameters()):
            assert torch.equal(p, q), (step, n)


def test_optimizer_without_a_bound_is_the_plain_step():
    a, b = _model(), _model()
    oa, ob = _opt(a), _opt(b, max_grad_norm=1e9)
    for i, (p, q) in enumerate(zip(a.parameters(), b.parameters())):
        g = as_dtype(host_normal(tuple(p.shape), 62000 + i, 1e-3), FP).cuda()
        p.grad, q.grad = g, g.clone()
    oa.step()
    ob.step()
    torch.cuda.synchronize()
    assert oa.grad_norm is None and float(ob.grad_norm) > 0
    assert all(torch.equal(p, q) for p, q in zip(a.parameters(), b.parameters()))


@pytest.mark.parametrize("clip", [None, 1e-4])
def test_optimizer_takes_sparse_embedding_gradients(clip):
    """nn.Embedding(sparse=True) under MuonAdamW: the step of the dense
    gradient, repeated tokens summed, untouched rows decayed by their moments."""
    a, b = _model(sparse=True), _model()
    oa, ob = _opt(a, max_grad_norm=clip), _opt(b, max_grad_norm=clip)
    for step in range(3):
        rng = np.random.default_rng(63 + step)
        tok = torch.from_numpy(rng.integers(0, 101, (4, 33))).cuda()
        # integers: their sums are exact in any order, so both gradients are the same bits
        up = torch.from_numpy(rng.integers(-4, 5, (4, 33, 64)).astype(np.float32)).cuda() / 1024
        for m in (a, b):
            m.zero_grad(set_to_none=True)
            m.wte(tok).backward(up)
            for i, (n, p) in enumerate(m.named_parameters()):
                if n != "wte.weight":
                    p.grad = as_dtype(host_normal(tuple(p.shape), 64000 + 10 * step + i, 1e-3), FP).cuda()
        assert a.wte.weight.grad.is_sparse and not b.wte.weight.grad.is_sparse
        oa.step()
        ob.step()
        torch.cuda.synchronize()
        for (n, p), q in zip(a.named_parameters(), b.parameters()):
            assert torch.equal(p, q), (step, n)


def test_optimizer_refuses_a_sparse_matrix_gradient():
    m = _model()
    opt = _opt(m)
    for p in m.parameters():
        p.grad = torch.zeros_like(p)
    before = [p.detach().clone() for p in m.parameters()]
    m.a.weight.grad = torch.zeros_like(m.a.weight).to_sparse()
    with pytest.raises(ValueError, match="sparse"):
        opt.step()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(m.parameters(), before))


def test_optimizer_copies_of_gradients_end_with_their_group():
    """Gradients that are not contiguous are copied for the step: without a bound
    on the norm one group's copies at a time, and none after the step."""
    import newton_schulz_orthogonalized_amd as nso
    shape, groups = (1024, 2048), 4
    copy = shape[0] * shape[1] * 4
    ps = [torch.nn.Parameter(torch.zeros(shape, device="cuda")) for _ in range(groups)]
    for p in ps:
        p.grad = torch.ones(shape[::-1], device="cuda").t()
    for clip, most in ((None, 1.5), (1.0, groups + 0.5)):
        opt = nso.MuonAdamW([{"params": [p], "kind": "muon" if i % 2 else "adamw"} for i, p in enumerate(ps)],
                            max_grad_norm=clip)
        opt.step()           # states and workspaces are made
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        opt.step()
        torch.cuda.synchronize()
        assert torch.cuda.max_memory_allocated() - before < most * copy, clip
        assert torch.cuda.memory_allocated() - before < copy // 2


@pytest.mark.parametrize("clip", [None, 1.0])
def test_optimizer_keeps_no_dense_gradient_of_a_sparse_one(clip):
    import newton_schulz_orthogonalized_amd as nso
    emb = torch.nn.Embedding(20000, 128, sparse=True, device="cuda")
    table = 20000 * 128 * 4
    opt = nso.MuonAdamW([{"params": [emb.weight], "kind": "adamw"}], max_grad_norm=clip)
    tok = torch.arange(64, device="cuda")
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for _ in range(2):
        emb(tok).sum().backward()
        opt.step()
        opt.zero_grad(set_to_none=True)
    torch.cuda.synchronize()
    # the two moments, nothing else of the table's size
    assert abs(torch.cuda.memory_allocated() - before - 2 * table) < table // 2


@pytest.mark.parametrize("dtype,precision", [(FP, "f32"), (BF, "bf16")])
def test_replayed_steps_follow_the_factor(dtype, precision):
    """One list of buffers, whose calls replay a graph from the second one on:
    factors that change in place, a factor at another address, none, and back,
    each step bit for bit the plain step of gradients times that power of two."""
    import newton_schulz_orthogonalized_amd as nso
    from newton_schulz_orthogonalized_amd import _lib
    shapes = [(96, 160), (160, 96), (33, 77), (256, 256)]
    mk = lambda seed, std, t: [as_dtype(host_normal(s, seed + i, std), t).cuda() for i, s in enumerate(shapes)]  # noqa: E731
    w, g, m = mk(65000, 0.02, dtype), mk(65100, 1e-3, dtype), mk(65200, 1e-3, FP)
    w2, g2, m2 = ([x.clone() for x in t] for t in (w, g, m))
    ws = _lib.workspace(nso.muon_workspace_bytes(w, g, m, precision=precision), "cuda")
    a, b = torch.zeros((), device="cuda"), torch.zeros(1, device="cuda")
    kw = dict(lr=0.02, weight_decay=0.01, precision=precision)
    for step, (t, c) in enumerate([(a, 0.5), (a, 0.5), (a, 0.25), (a, 1.0), (b, 0.125), (b, 0.5), (None, 1.0), (a, 0.25),
                                   (None, 1.0), (b, 2.0), (a, 0.5)]):
        if t is not None:
            a.fill_(-1.0), b.fill_(-1.0)     # what the step must not read
            t.fill_(c)
        for x, y in zip(g, g2):
            y.copy_(x * c)
        nso.muon_step(w, g, m, grad_scale=t, workspace=ws, **kw)
        nso.muon_step(w2, g2, m2, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(w + m, w2 + m2)), (step, c)


def test_thousands_of_tensors():
    """Lists of dozens of launches of both kernels, of large and small tensors;
    the sums in float64 and the one product and rounding exactly."""
    import newton_schulz_orthogonalized_amd as nso
    sizes = [1 + (i * 7919) % 997 if i % 50 else 30000 + i for i in range(5000)]
    flat = (((torch.arange(sum(sizes), device="cuda") * 7919) % 2003 - 1001).float() / 4096)
    g = list(flat.split(sizes))
    for i in range(0, 5000, 3):
        g[i] = g[i].to(BF)
    want = math.sqrt(sum(float(x.double().square().sum()) for x in g))
    assert abs(float(nso.grad_norm(g)) - want) <= want * ULP * 1.001
    outs = [torch.zeros(x.numel(), dtype=(FP, BF)[i % 2], device="cuda") for i, x in enumerate(g)]
    scale = torch.zeros((), device="cuda")
    norm = nso.clip_grads(g, 3.0, outs=outs, scale_out=scale)
    torch.cuda.synchronize()
    assert abs(float(norm) - want) <= want * ULP * 1.001
    assert abs(float(scale) - 3.0 / (want + 1e-6)) <= 3.0 / want * ULP * 1.001
    for i, (x, o) in enumerate(zip(g, outs)):
        assert torch.equal(o, (x.float() * scale).to(o.dtype)), i
