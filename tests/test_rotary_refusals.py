"""Calls of rotary whose results would silently lack something, refused on a
machine without a GPU: a gradient or tangent of the frequencies, and an offset
that does not fit the call's field."""

import pytest
import torch


def _args(offset):
    import newton_schulz_orthogonalized_amd as nso
    from newton_schulz_orthogonalized_amd import _lib
    q = torch.zeros(2, 5, 4, 16)
    return _lib.rotary_args((q,), (torch.empty_like(q),), nso.rotary_frequencies(16, device="cpu"), None, offset, False, False, 1.0)


@pytest.mark.parametrize("needs", ["freqs", "both"])
def test_no_gradient_of_the_frequencies(needs):
    import newton_schulz_orthogonalized_amd as nso
    q = torch.zeros(2, 5, 4, 16, requires_grad=needs == "both")
    freqs = nso.rotary_frequencies(16, device="cpu").requires_grad_()
    with pytest.raises(NotImplementedError, match="freqs"):
        nso.rotary(q, freqs=freqs)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):     # nothing asked for: on to the next check
        nso.rotary(q, freqs=freqs)


def test_no_tangent_of_the_frequencies():
    import newton_schulz_orthogonalized_amd as nso
    with torch.autograd.forward_ad.dual_level():
        f = nso.rotary_frequencies(16, device="cpu")
        with pytest.raises(NotImplementedError):
            nso.rotary(torch.zeros(2, 5, 4, 16), freqs=torch.autograd.forward_ad.make_dual(f, f))


@pytest.mark.parametrize("offset", [(1 << 52) + 1, -(1 << 52) - 1, 1 << 64, (1 << 64) + 7, -(1 << 64)])
def test_offsets_out_of_range(offset):
    with pytest.raises(ValueError, match="offset"):
        _args(offset)


def test_offsets_in_range():
    for offset in (0, 7, -3, 1 << 52, -(1 << 52)):
        assert _args(offset).offset == offset
