"""Float64 references of the parts of a transformer block between its products:
rotary positions, the norms around a block with its gate and residual scale, the
gated feed-forward product, and their gradients. Plain numpy, no code shared with
the package."""

from __future__ import annotations

import math

import numpy as np

erf = np.vectorize(math.erf, otypes=[np.float64])


def frequencies_ref(part, base=10000.0, factor=1.0, original_length=None, low=1.0, high=32.0):
    """One frequency at a time."""
    out = []
    for i in range(part // 2):
        f = math.exp(-2.0 * i / part * math.log(base))
        if original_length is None:
            f /= factor
        else:
            r = original_length * f / (2 * math.pi)
            if r <= low:
                f /= factor
            elif r < high:
                y = (r - low) / (high - low)
                f = (1 - y) * f / factor + y * f
        out.append(f)
    return np.array(out)


def rotary_ref(x, pos, freqs, interleaved=False, scale=1.0, inverse=False):
    """x [batch, length, heads, dim], pos [batch, length]. Returns (result, |a| + |b|
    of the pair behind each element, 0 for elements that are copied)."""
    out, mag = np.array(x, np.float64), np.zeros(x.shape)
    half = len(freqs)
    for i in range(half):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        angle = pos.astype(np.float64) * freqs[i]
        c, s = np.cos(angle)[..., None], np.sin(angle)[..., None]
        if inverse:
            s = -s
        a, b = x[..., ia], x[..., ib]
        out[..., ia] = scale * (a * c - b * s)
        out[..., ib] = scale * (b * c + a * s)
        mag[..., ia] = mag[..., ib] = abs(scale) * (np.abs(a) + np.abs(b))
    return out, mag


def _w(w, dim):
    return np.ones(dim) if w is None else w


def residual_norm_ref(r, y, gate=None, post_norm=False, post=None, pre=None, a=1.0, eps=1e-6):
    """(new_residual, normed, |a r| + |update's share|) of rows [rows, dim]; gate [groups, dim]."""
    dim = r.shape[1]
    ar = a * r
    p = np.zeros_like(r)
    if y is not None:
        p = y / np.sqrt(np.mean(y * y, 1, keepdims=True) + eps) * _w(post, dim) if post_norm else y.copy()
        if gate is not None:
            p = p * np.repeat(gate, r.shape[0] // max(gate.shape[0], 1), 0)
    new = ar + p
    return new, new / np.sqrt(np.mean(new * new, 1, keepdims=True) + eps) * _w(pre, dim), np.abs(ar) + np.abs(p)


def residual_norm_grad_ref(dr, dn, new, y, gate=None, post_norm=False, post=None, pre=None, a=1.0, eps=1e-6):
    """Gradients row by row, with for each the sum of magnitudes that bounds its
    float32 error: {name: (gradient, magnitudes)}."""
    rows, dim = new.shape
    groups = 1 if gate is None else gate.shape[0]
    per = rows // groups if groups else 0
    zero = np.zeros(dim)
    out = {"r": (np.zeros_like(new), np.zeros_like(new)), "y": (np.zeros_like(new), np.zeros_like(new)),
           "pre": (zero.copy(), zero.copy()), "post": (zero.copy(), zero.copy()),
           "gate": (np.zeros((groups, dim)), np.zeros((groups, dim)))}
    wp, wq = _w(post, dim), _w(pre, dim)
    for i in range(rows):
        g = np.ones(dim) if gate is None else gate[i // per]
        v, n = new[i], zero if dn is None else dn[i]
        d, md = (zero, zero) if dr is None else (dr[i], np.abs(dr[i]))
        if dn is not None:
            s = 1.0 / math.sqrt(np.mean(v * v) + eps)
            t = n * wq
            d = d + s * t - s ** 3 * np.mean(t * v) * v
            md = md + np.abs(s * t) + s ** 3 * np.mean(np.abs(t * v)) * np.abs(v)
            out["pre"][0][:] += n * v * s
            out["pre"][1][:] += np.abs(n * v * s)
        out["r"][0][i], out["r"][1][i] = a * d, abs(a) * md
        if y is None:
            continue
        f = 1.0 / math.sqrt(np.mean(y[i] * y[i]) + eps) if post_norm else 1.0
        hat = y[i] * f
        out["gate"][0][i // per if gate is not None else 0] += d * hat * wp
        out["gate"][1][i // per if gate is not None else 0] += md * np.abs(hat * wp)
        out["post"][0][:] += d * g * hat
        out["post"][1][:] += md * np.abs(g * hat)
        u, mu = d * g * wp, md * np.abs(g * wp)
        out["y"][0][i], out["y"][1][i] = f * u, f * mu
        if post_norm:
            out["y"][0][i] -= f ** 3 * np.mean(u * y[i]) * y[i]
            out["y"][1][i] += f ** 3 * np.mean(mu * np.abs(y[i])) * np.abs(y[i])
    return out


def activation_ref(g, kind):
    """(act(g), act'(g), argument of the exponential in it)."""
    if kind == "silu":
        s = 1.0 / (1.0 + np.exp(-g))
        return g * s, s + g * s * (1 - s), np.abs(g)
    if kind == "gelu":
        phi = 0.5 * (1.0 + erf(g / math.sqrt(2.0)))
        return g * phi, phi + g * np.exp(-g * g / 2) / math.sqrt(2 * math.pi), g * g
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        z = c * (g + 0.044715 * g ** 3)
        t = np.tanh(z)
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g), 8 * np.abs(z)
    return np.maximum(g, 0.0), (g > 0).astype(np.float64), np.zeros_like(g)


def gated_mlp_ref(x, wg, wu, kind="silu"):
    """(h, g, u, sums of magnitudes of g and of u)."""
    g, u = x @ wg.T, x @ wu.T
    return activation_ref(g, kind)[0] * u, g, u, np.abs(x) @ np.abs(wg).T, np.abs(x) @ np.abs(wu).T


def gated_mlp_grad_ref(dh, x, wg, wu, g, u, kind="silu"):
    """(dx, d_gate, d_up, dg, du)."""
    act, slope, _ = activation_ref(g, kind)
    dg, du = dh * u * slope, dh * act
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dg, du
