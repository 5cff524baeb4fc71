"""Rotary positions in place on the views that fused projections give: queries and
keys head by head, heads first, grouped. Against the call into buffers of its own,
whose results test_gpu_rotary.py compares with the reference; what lies between
the views keeps its bits."""

import pytest
import torch

from gpu_util import need_gpu
from test_block_views import KINDS, _fused

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    import newton_schulz_orthogonalized_amd  # noqa: F401  (fails loudly without the library)
    yield


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("b,s,hq,hk,d,part", [(2, 70, 4, 2, 32, 32), (3, 1, 8, 8, 90, 70), (1, 33, 2, 1, 128, 64)])
def test_in_place(kind, b, s, hq, hk, d, part, dtype, interleaved):
    import newton_schulz_orthogonalized_amd as nso
    places = _fused(kind, b, s, hq, hk, d)
    g = torch.Generator(device="cuda")
    g.manual_seed(97100)
    buf = torch.empty(places[0].untyped_storage().nbytes() // 4, dtype=dtype, device="cuda").normal_(generator=g)
    q, k = (buf.as_strided(t.shape, t.stride(), t.storage_offset()) for t in places)
    freqs = nso.rotary_frequencies(part)
    want = nso.rotary(q, k, freqs=freqs, interleaved=interleaved)
    expect = buf.clone()
    for t, w in zip(places, want):
        expect.as_strided(t.shape, t.stride(), t.storage_offset()).copy_(w)
    # into views of another buffer, then in place
    other = torch.full_like(buf, 7.0)
    outs = tuple(other.as_strided(t.shape, t.stride(), t.storage_offset()) for t in places)
    nso.rotary(q, k, freqs=freqs, interleaved=interleaved, out=outs)
    untouched = torch.ones_like(buf, dtype=torch.bool)
    for t in places:
        untouched.as_strided(t.shape, t.stride(), t.storage_offset()).fill_(False)
    assert torch.equal(other, torch.where(untouched, torch.full_like(buf, 7.0), expect))
    nso.rotary(q, k, freqs=freqs, interleaved=interleaved, out=(q, k))
    assert torch.equal(buf, expect)
