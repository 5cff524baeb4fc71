"""Float64 references of the operators that feed the optimizer step: gradient
norm and clipping, the embedding and its gradient, attention max logits. Plain
loops and numpy, no code shared with the package."""

from __future__ import annotations

import numpy as np


def grad_norm_ref(grads) -> float:
    """Global 2-norm of a list of arrays (exponent-scaled, so that no square
    over- or underflows)."""
    top = max((float(np.max(np.abs(g))) for g in grads if g.size), default=0.0)
    if top == 0.0 or not np.isfinite(top):
        return float(top) if not any(np.isnan(g).any() for g in grads) else float("nan")
    e = 2.0 ** np.floor(np.log2(top))
    return float(e * np.sqrt(sum(np.sum((np.asarray(g, np.float64) / e) ** 2) for g in grads)))


def clip_scale_ref(norm: float, max_norm: float, eps: float = 1e-6) -> float:
    if np.isnan(norm):
        return float("nan")
    d = norm + eps
    return 1.0 if d == 0.0 else min(1.0, max_norm / d)


def embedding_ref(tokens, weight, scale: float = 1.0):
    """scale * weight[tokens]; NaN rows for tokens outside the table."""
    tokens = np.asarray(tokens).reshape(-1)
    out = np.full((tokens.size, weight.shape[1]), np.nan)
    for t, v in enumerate(tokens):
        if 0 <= v < weight.shape[0]:
            out[t] = scale * weight[v]
    return out


def embedding_grad_ref(tokens, rows, vocab: int, scale: float = 1.0, padding_idx=None, base=None):
    """(gradient, the same sums of magnitudes, terms per row): the last two bound
    what a float32 sum in any order may be off by."""
    tokens = np.asarray(tokens).reshape(-1)
    rows = np.asarray(rows, np.float64).reshape(tokens.size, -1)
    g = np.zeros((vocab, rows.shape[1]))
    mag = np.zeros_like(g)
    n = np.zeros(vocab, dtype=np.int64)
    for t, v in enumerate(tokens):
        if 0 <= v < vocab and v != padding_idx:
            g[v] += rows[t]
            mag[v] += np.abs(rows[t])
            n[v] += 1
    g *= scale
    mag *= abs(scale)
    if base is not None:
        g += base
    return g, mag, n


def qk_max_logits_ref(seqs, group: int, scale: float, causal: bool):
    """seqs: list of (q [nq, Hq, D], k [nk, Hk, D]). Returns (max |scale q.k| of
    each query head over the visible pairs, the largest sum of |q_d k_d| times
    |scale| among them)."""
    hq = seqs[0][0].shape[1]
    best, mag = np.zeros(hq), np.zeros(hq)
    for q, k in seqs:
        nq, nk = q.shape[0], k.shape[0]
        if nq == 0 or nk == 0:
            continue
        seen = np.ones((nq, nk), bool)
        if causal:
            seen = np.arange(nk)[None, :] <= np.arange(nq)[:, None] + nk - nq
        if not seen.any():
            continue
        for h in range(hq):
            with np.errstate(invalid="ignore", over="ignore"):
                s = np.abs(scale * (q[:, h] @ k[:, h // group].T))[seen]
                m = abs(scale) * (np.abs(q[:, h]) @ np.abs(k[:, h // group]).T)[seen]
            best[h] = np.maximum(best[h], s.max())
            mag[h] = np.maximum(mag[h], m.max())
    return best, mag
