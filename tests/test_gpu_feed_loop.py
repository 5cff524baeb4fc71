"""The calls that feed the step together, as a training loop has them: lookup,
its gradient through autograd over two micro-batches, the max logits kept over
them, MuonAdamW with a bound on the gradient norm, then QK-Clip; each stage
against the float64 reference on the values that the GPU had before it.

The forward and backward passes work on small integers, whose sums are exact in
float32 in any order, so the gradients must be equal. Tolerances: the norm half
a step (2^-24) of float32 and its float64 rounding. A momentum is a product
c g, (1 - mu), a product, a sum: 8 half steps of its terms. AdamW moves an element
by lr m / sqrt(v): in two steps m is off by at most 8 half steps of the larger
gradient over its correction 0.19, sqrt(v) at least 0.69 of that gradient, and
roots, quotients and corrections add 16: 80 half steps of lr, taken as 128, and
2 of the parameter. The orthogonal direction is within the float32 bound of the
Muon tests, and a clipped weight is a quotient and a product: 4 half steps.
"""

import numpy as np
import pytest
import torch

from gpu_util import need_gpu, to_np
from oracle import feed_oracle as F
from oracle import muon_oracle as O

pytestmark = pytest.mark.gpu

ULP = 2.0 ** -24
F32_TOL = 1e-4
VOCAB, DIM, HQ, HK, D = 90, 48, 4, 2, 16
LR, ALR, WD = 0.5, 0.25, 0.01


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    import newton_schulz_orthogonalized_amd  # noqa: F401  (fails loudly without the library)
    yield


def _ints(rng, *shape, top=3):
    return torch.from_numpy(rng.integers(-top, top + 1, shape).astype(np.float32)).cuda()


@pytest.mark.parametrize("side_stream", [False, True])
def test_a_loop_of_all_calls(side_stream):
    """side_stream: the whole loop on a side stream."""
    import newton_schulz_orthogonalized_amd as nso
    rng = np.random.default_rng(90000)
    table = _ints(rng, VOCAB, DIM).requires_grad_()
    wq, wk = _ints(rng, HQ * D, DIM).requires_grad_(), _ints(rng, HK * D, DIM).requires_grad_()
    opt = nso.MuonAdamW([{"params": [wq, wk], "kind": "muon"}, {"params": [table], "kind": "adamw"}], lr=LR,
                        weight_decay=WD, adamw_lr=ALR, precision="f32", max_grad_norm=40.0)
    stream = torch.cuda.Stream() if side_stream else torch.cuda.current_stream()
    stream.wait_stream(torch.cuda.current_stream())
    moments = [np.zeros((VOCAB, DIM)), np.zeros((VOCAB, DIM))]
    mom = [np.zeros((HQ * D, DIM)), np.zeros((HK * D, DIM))]
    with torch.cuda.stream(stream):
        for step in range(2):
            with torch.no_grad():     # integers again, so that this step's sums are exact too
                for p in (table, wq, wk):
                    p.copy_(p.round().clamp_(-4, 4))
            torch.cuda.synchronize()
            w0 = [to_np(p) for p in (wq, wk, table)]
            logits = torch.zeros(HQ, device="cuda")
            ref_g = [np.zeros_like(w) for w in w0]
            best = np.zeros(HQ)
            opt.zero_grad(set_to_none=True)
            for mb in range(2):
                b, s = 3, 37 + mb
                tok = torch.from_numpy(rng.integers(0, VOCAB, (b, s))).cuda()
                lens = np.array([s, 5, 0])
                seen = torch.from_numpy((np.arange(s)[None] < lens[:, None]).astype(np.float32)).cuda()[..., None]
                uq, uk, ux = _ints(rng, b, s, HQ * D) * seen, _ints(rng, b, s, HK * D) * seen, _ints(rng, b, s, DIM) * seen
                x = nso.embedding(tok, table, scale=2.0, padding_idx=7)
                q, k = x @ wq.t(), x @ wk.t()
                nso.qk_max_logits(q.view(b, s, HQ, D), k.view(b, s, HK, D), out=logits, accumulate=True, scale=0.25,
                                  lengths=torch.from_numpy(lens.astype(np.int32)).cuda())
                ((q * uq).sum() + (k * uk).sum() + (x * ux).sum()).backward()
                # the reference
                hx = F.embedding_ref(to_np(tok).astype(int).ravel(), w0[2], 2.0)
                hq, hk = hx @ w0[0].T, hx @ w0[1].T
                gq, gk = to_np(uq).reshape(b * s, -1), to_np(uk).reshape(b * s, -1)
                ref_g[0] += gq.T @ hx
                ref_g[1] += gk.T @ hx
                rows = gq @ w0[0] + gk @ w0[1] + to_np(ux).reshape(b * s, -1)
                ref_g[2] += F.embedding_grad_ref(to_np(tok).astype(int).ravel(), rows, VOCAB, 2.0, 7)[0]
                hq, hk = hq.reshape(b, s, HQ, D), hk.reshape(b, s, HK, D)
                best = np.maximum(best, F.qk_max_logits_ref([(hq[i, :n], hk[i, :n]) for i, n in enumerate(lens)], HQ // HK,
                                                            0.25, True)[0])
            torch.cuda.synchronize()
            assert max(np.abs(g).max() for g in ref_g) < 2 ** 22 and best.max() < 2 ** 20     # exact indeed
            for p, g in zip((wq, wk, table), ref_g):
                assert np.array_equal(to_np(p.grad), g)
            assert np.array_equal(to_np(logits), best)
            opt.step()
            torch.cuda.synchronize()
            norm = F.grad_norm_ref(ref_g)
            c = F.clip_scale_ref(norm, 40.0)
            assert c < 1 and abs(float(opt.grad_norm) - norm) <= norm * ULP * 1.001
            for i, p in enumerate((wq, wk)):
                r = O.muon_step_ref(w0[i], c * ref_g[i], mom[i], lr=LR, weight_decay=WD)
                got = to_np(opt.state[p]["momentum_buffer"])
                assert np.all(np.abs(got - r["m"]) <= 8 * ULP * (np.abs(mom[i]) + 0.05 * c * np.abs(ref_g[i])))
                mom[i] = got
                assert np.linalg.norm(to_np(p) - r["w"]) <= LR * F32_TOL * np.linalg.norm(r["o"]) + 2 * ULP * np.linalg.norm(w0[i])
            t, m, v = O.adamw_ref(w0[2], c * ref_g[2], *moments, lr=ALR, weight_decay=0.0, beta1=0.9, beta2=0.95, eps=1e-8,
                                  step=step + 1)
            assert np.all(np.abs(to_np(table) - t) <= 128 * ULP * ALR + 2 * ULP * np.abs(w0[2]))
            moments = [m, v]
            before = [to_np(wq), to_np(wk)]
            tau = float(np.sort(best)[1:3].mean())
            want_q, want_k, gamma = O.qk_clip_ref(*before, to_np(logits), q_heads=HQ, k_heads=HK, tau=tau)
            nso.qk_clip([wq], [wk], [logits], q_heads=HQ, k_heads=HK, tau=tau)
            torch.cuda.synchronize()
            assert int((np.asarray(gamma) < 1).sum()) >= 1
            for p, want in ((wq, want_q), (wk, want_k)):
                assert np.all(np.abs(to_np(p) - want) <= 4 * ULP * np.abs(want))
