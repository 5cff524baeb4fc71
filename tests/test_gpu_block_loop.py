"""The parts of a transformer block together, as a training loop has them: the
first norm, projections, rotary positions, the max logits of QK-Clip, attention,
the gate and norms around the block, the gated feed-forward product, the backward
pass, and the MuonAdamW step with QK-Clip; the gradients against the same block in
float64 torch operations.

Tolerances (norm of the difference over the norm): in float32, 24 operations of
both passes, each within 2 K U (K = 64 terms, U = 2^-24) of magnitudes that
cancel to no less than a sixteenth: 24 * 128 * 16 U < 2^-8. In bfloat16 24
roundings of 2^-8 each, as independent errors: their root of 24 times 2^-8, taken
four times for what cancels.
"""

import math

import pytest
import torch

from gpu_util import need_gpu
from oracle import block_oracle as B
from workloads import as_dtype, host_normal

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32
BATCH, SEQ, DIM, HQ, HK, HEAD, PART, HIDDEN = 2, 40, 64, 4, 2, 16, 12, 88


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    import newton_schulz_orthogonalized_amd  # noqa: F401  (fails loudly without the library)
    yield


def _weights(dtype):
    shapes = {"wq": (HQ * HEAD, DIM), "wk": (HK * HEAD, DIM), "wv": (HK * HEAD, DIM), "wo": (DIM, HQ * HEAD),
              "w_gate": (HIDDEN, DIM), "w_up": (HIDDEN, DIM), "w_down": (DIM, HIDDEN)}
    ps = {k: as_dtype(host_normal(s, 95000 + i, s[1] ** -0.5), dtype).cuda() for i, (k, s) in enumerate(shapes.items())}
    for i in range(4):
        ps[f"norm{i}"] = as_dtype(host_normal((DIM,), 95020 + i, 0.1) + 1, dtype).cuda()
    ps["gate"] = as_dtype(host_normal((BATCH, DIM), 95030), dtype).cuda()
    return {k: v.requires_grad_() for k, v in ps.items()}


def _attend(q, k, v):
    """Causal attention in torch operations: [batch, length, heads, head]."""
    k, v = (t.repeat_interleave(HQ // HK, 2) for t in (k, v))
    s = (q[:, :, None] * k[:, None]).sum(-1) / math.sqrt(HEAD)            # [batch, i, j, heads]
    i = torch.arange(SEQ, device=q.device)
    p = torch.softmax(s.masked_fill((i[None, :] > i[:, None])[None, :, :, None], float("-inf")), 2)
    return (p[..., None] * v[:, None]).sum(2).flatten(2)


def _own(x, ps, freqs, logits=None):
    import newton_schulz_orthogonalized_amd as nso
    n = nso.rms_norm(x, ps["norm0"])
    q, k, v = ((n @ ps[w].t()).unflatten(-1, (-1, HEAD)) for w in ("wq", "wk", "wv"))
    q, k = nso.rotary(q, k, freqs=freqs, scale=1.25)
    if logits is not None:
        nso.qk_max_logits(q.detach(), k.detach(), out=logits, accumulate=True)
    r, n = nso.residual_norm(x, _attend(q, k, v) @ ps["wo"].t(), gate=ps["gate"], post_weight=ps["norm1"], pre_weight=ps["norm2"],
                             residual_scale=0.5)
    h = nso.gated_mlp(n, ps["w_gate"], ps["w_up"])
    return nso.residual_norm(r, h @ ps["w_down"].t(), pre_weight=ps["norm3"])


def _plain(x, ps, freqs):
    """The same in float64 torch operations on the CPU."""
    def norm(v, w):
        return v / (v.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w

    def turn(v):
        a = (torch.arange(SEQ, dtype=torch.float64)[:, None] * freqs)[None, :, None]
        p, q = v[..., :PART // 2], v[..., PART // 2:PART]
        return torch.cat((1.25 * (p * a.cos() - q * a.sin()), 1.25 * (q * a.cos() + p * a.sin()), v[..., PART:]), -1)
    n = norm(x, ps["norm0"])
    q, k, v = ((n @ ps[w].t()).unflatten(-1, (-1, HEAD)) for w in ("wq", "wk", "wv"))
    q, k = turn(q), turn(k)
    r = 0.5 * x + ps["gate"][:, None] * norm(_attend(q, k, v) @ ps["wo"].t(), ps["norm1"])
    n = norm(r, ps["norm2"])
    g = n @ ps["w_gate"].t()
    r = r + (g / (1 + torch.exp(-g)) * (n @ ps["w_up"].t())) @ ps["w_down"].t()
    causal = torch.ones(SEQ, SEQ, dtype=torch.bool).tril()
    logits = torch.stack([((q[:, :, h] @ k[:, :, h * HK // HQ].transpose(1, 2)).abs() * causal).max() for h in range(HQ)])
    return (r, norm(r, ps["norm3"])), logits / math.sqrt(HEAD)


@pytest.mark.parametrize("dtype,tol", [(FP, 2.0 ** -8), (BF, 4 * math.sqrt(24) * 2.0 ** -8)])
@pytest.mark.parametrize("side_stream", [False, True])
def test_a_block_trains(dtype, tol, side_stream):
    import newton_schulz_orthogonalized_amd as nso
    ps = _weights(dtype)
    x = as_dtype(host_normal((BATCH, SEQ, DIM), 95100), dtype).cuda().requires_grad_()
    ups = [as_dtype(host_normal((BATCH, SEQ, DIM), 95110 + i), dtype).cuda() for i in range(2)]
    freqs = nso.rotary_frequencies(PART, base=100.0)
    muon = [k for k, v in ps.items() if v.dim() == 2 and k != "gate"]
    opt = nso.MuonAdamW([{"params": [ps[k] for k in muon], "kind": "muon"},
                         {"params": [v for k, v in ps.items() if k not in muon], "kind": "adamw"}], max_grad_norm=1.0,
                        adamw_lr=0.03,   # more than half a bfloat16 step of 1
                        precision="f32" if dtype == FP else "bf16")
    stream = torch.cuda.Stream() if side_stream else torch.cuda.current_stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(2):
            host = {k: v.detach().double().cpu().requires_grad_() for k, v in ps.items()}
            hx = x.detach().double().cpu().requires_grad_()
            opt.zero_grad(set_to_none=True)
            x.grad = None
            logits = torch.zeros(HQ, device="cuda")
            res = _own(x, ps, freqs, logits)
            torch.autograd.backward(res, ups)
            ref, best = _plain(hx, host, torch.from_numpy(B.frequencies_ref(PART, 100.0)))
            torch.autograd.backward(ref, [u.double().cpu() for u in ups])
            torch.cuda.synchronize()

            def close(got, want, what):
                err = float((got.detach().double().cpu() - want.detach()).norm() / want.detach().norm())
                assert err <= tol, (what, err)
            for got, want, what in zip(res, ref, ("residual", "normed")):
                close(got, want, what)
            close(logits, best, "logits")
            close(x.grad, hx.grad, "x")
            for k in ps:
                close(ps[k].grad, host[k].grad, k)
            before = {k: v.detach().clone() for k, v in ps.items()}
            opt.step()
            nso.qk_clip([ps["wq"].detach()], [ps["wk"].detach()], [logits], q_heads=HQ, k_heads=HK)
            torch.cuda.synchronize()
            for k, v in ps.items():
                assert bool(v.isfinite().all()) and not torch.equal(v, before[k]), k


def test_captured_forward_and_backward():
    """The own calls of a block, forward and backward, captured and replayed
    between eager work, each replay against the eager result."""
    import newton_schulz_orthogonalized_amd as nso
    t, d, f = 90, 64, 72
    r, y = (as_dtype(host_normal((t, d), 95200 + i), BF).cuda() for i in range(2))
    w = as_dtype(host_normal((d,), 95210, 0.1) + 1, BF).cuda()
    wg, wu = (as_dtype(host_normal((f, d), 95220 + i, d ** -0.5), BF).cuda() for i in range(2))
    up, freqs = as_dtype(host_normal((t, f), 95230), BF).cuda(), nso.rotary_frequencies(24)

    def step():
        ts = [v.detach().requires_grad_() for v in (r, y, w, wg, wu)]     # leaves of this pass alone
        _, n = nso.residual_norm(ts[0], ts[1], post_weight=ts[2], pre_weight=ts[2])
        h = nso.gated_mlp(n, ts[3], ts[4])
        o = nso.rotary(h.view(t, 3, 24), freqs=freqs)
        return [o.detach(), *torch.autograd.grad(o, ts, up.view(t, 3, 24))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = step()
    for _ in range(4):
        y.mul_(0.75)
        wu.mul_(-1)
        g.replay()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(cap, want))
