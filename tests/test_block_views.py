"""Which views mu_rotary takes as sharing elements, on a machine without a GPU: a
call whose views it accepts ends at the launch (status 5: no GPU), one that it
refuses before that (status 3). Against the sets of the elements' addresses."""

import ctypes
import random

import pytest
import torch

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="its addresses must not reach a kernel")

A = 0x7f0000000000   # never dereferenced
FREQS = 0x7e0000000000


def _status(q, k, dim, batch, length):
    """mu_rotary in place on views (offset, heads, stride_b, stride_s, stride_h) of one bfloat16 buffer."""
    from newton_schulz_orthogonalized_amd import _lib as lib
    a = lib.MuRotaryArgs(freqs=FREQS, positions=None, offset=0, batch=batch, len=length, n=2, dim=dim, part=2, position_bits=0,
                         shared_positions=0, interleaved=0, inverse=0, dtype=lib.MU_BF16, scale=1.0, pad0=0)
    for i, (at, heads, *s) in enumerate((q, k)):
        a.x[i] = lib.MuRotaryTensor(A + 2 * at, A + 2 * at, *s, *s, heads, 0)
    return lib.LIB.mu_rotary(ctypes.byref(a), None)


def _elements(view, dim, batch, length):
    at, heads, sb, ss, sh = view
    return [at + b * sb + s * ss + h * sh + d for b in range(batch) for s in range(length) for h in range(heads) for d in range(dim)]


def _views(t):
    """(offset, heads, strides) of a [batch, length, heads, dim] view."""
    return t.storage_offset(), t.shape[2], *t.stride()[:3]


def _fused(kind, b, s, hq, hk, d):
    """q and k as views of one projection's result."""
    if kind == "columns":                                    # [b, s, heads, dim]: ranges of heads
        t = torch.empty(b, s, hq + 2 * hk, d)
        return t[:, :, :hq], t[:, :, hq:hq + hk]
    if kind == "head by head":                               # [b, s, heads, 3, dim]
        t = torch.empty(b, s, hq, 3, d)
        return t[..., 0, :], t[..., 1, :]
    if kind == "heads first":                                # [b, heads, s, dim]
        t = torch.empty(b, hq + 2 * hk, s, d).transpose(1, 2)
        return t[:, :, :hq], t[:, :, hq:hq + hk]
    if kind == "heads first, side by side":                  # [b, heads, s, 3, dim]
        t = torch.empty(b, hq, s, 3, d).transpose(1, 2)
        return t[..., 0, :], t[..., 1, :]
    if kind == "groups":                                     # [b, s, k heads, queries of one, its key, dim]
        t = torch.empty(b, s, hk, 3, d)
        return t[..., 0, :], t[..., 2, :]
    t = torch.empty(b, s, 2, hq, d)                          # "one row behind the other"
    return t[:, :, 0], t[:, :, 1]


KINDS = ["columns", "head by head", "heads first", "heads first, side by side", "groups", "one row behind the other"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("b,s,hq,hk,d", [(1, 1, 1, 1, 8), (2, 5, 4, 2, 8), (3, 1, 4, 4, 16), (1, 7, 2, 1, 10), (64, 1, 32, 4, 128)])
def test_views_of_a_projection_are_apart(kind, b, s, hq, hk, d):
    q, k = _fused(kind, b, s, hq, hk, d)
    vq, vk = _views(q), _views(k)
    assert _status(vq, vk, d, b, s) == 5 and _status(vk, vq, d, b, s) == 5
    # one element further on, the key's last of a head is the next one's first, or lies outside
    moved = (vk[0] - 1, *vk[1:])
    shared = set(_elements(vq, d, b, s)) & set(_elements(moved, d, b, s))
    assert _status(vq, moved, d, b, s) == (3 if shared else 5)


def test_views_of_one_buffer_at_random():
    """Strides that nest, the same for both but where a size is one; any offset."""
    rng, seen = random.Random(97000), {3: 0, 5: 0}
    for _ in range(3000):
        b, s, hq, hk, d = (rng.randint(1, 4) for _ in range(5))
        d = max(d, 2)
        dims = {"b": b, "s": s, "h": max(hq, hk)}
        strides, extent = {}, d
        for name in rng.sample(sorted(dims), 3):
            strides[name] = extent + rng.choice([0, 0, 1, 3, d, 2 * d])
            extent = strides[name] * dims[name]

        def of(at, heads):
            return (at, heads, *(strides[n] if size > 1 else rng.randint(0, 40) for n, size in (("b", b), ("s", s), ("h", heads))))
        q, k = of(0, hq), of(rng.randint(0, extent), hk)
        eq, ek = _elements(q, d, b, s), _elements(k, d, b, s)
        assert len(set(eq)) == len(eq) and len(set(ek)) == len(ek)
        got = _status(q, k, d, b, s)
        assert got == (3 if set(eq) & set(ek) else 5), (q, k, b, s, d)
        seen[got] += 1
    assert min(seen.values()) > 300


def test_views_of_unlike_strides_never_pass_where_they_meet():
    """What is refused beyond them are views of one memory range with unlike strides."""
    rng, met = random.Random(97001), 0
    for _ in range(3000):
        b, s, hq, hk, d = (rng.randint(1, 3) for _ in range(5))
        d = max(d, 2)
        views = []
        for heads in (hq, hk):
            extent, strides = d, {}
            for name in rng.sample("bsh", 3):
                strides[name] = extent + rng.choice([0, 1, d])
                extent = strides[name] * {"b": b, "s": s, "h": heads}[name]
            views.append((rng.randint(0, 30), heads, strides["b"], strides["s"], strides["h"]))
        q, k = views
        if set(_elements(q, d, b, s)) & set(_elements(k, d, b, s)):
            met += 1
            assert _status(q, k, d, b, s) == 3, (q, k, b, s, d)
    assert met > 300
