"""What the backward passes of the block's calls hold while a kernel is launched:
the dense copy of a gradient that autograd hands in transposed or expanded has to
live until the launch has been made. Without a GPU, as in test_block_streams.py:
no kernel is called; the stand-in for each launch looks whether a living tensor
stands behind the address that it is given."""

import weakref

import pytest
import torch

from test_block_streams import made_and_tied  # noqa: F401  (a fixture)
from test_streams import notes  # noqa: F401  (a fixture)


@pytest.fixture
def launches(made_and_tied, monkeypatch):  # noqa: F811
    """Of each gradient call: (gradients read, those of them that nobody holds any more)."""
    from newton_schulz_orthogonalized_amd import _lib
    real_contiguous, copies, seen = torch.Tensor.contiguous, [], []
    real_empty = torch.empty

    def contiguous(t, *a, **k):
        c = real_contiguous(t, *a, **k)
        if c.data_ptr() != t.data_ptr():
            copies.append((weakref.ref(c), c.data_ptr()))
        return c

    class Library:
        def __getattr__(self, name):
            return getattr(real, name)

        def mu_residual_norm_grad(self, ref, ws, nb, stream):
            return note(ref, "grad_residual", "grad_normed")

        def mu_gated_mlp_grad(self, ref, ws, nb, stream):
            return note(ref, "grad_h")

        def mu_rotary(self, ref, stream):
            a = ref._obj
            return look([a.x[i].x for i in range(a.n)])

    def note(ref, *names):
        return look([getattr(ref._obj, n) for n in names])

    def look(addresses):
        read = [p for p in addresses if p in [at for _, at in copies]]
        seen.append((len(read), [p for p in read if not any(w() is not None and at == p for w, at in copies)]))
        copies.clear()      # (their memory may be another tensor's next)
        return 0
    real = _lib.LIB
    monkeypatch.setattr(_lib, "LIB", Library())
    monkeypatch.setattr(torch.Tensor, "contiguous", contiguous)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)      # where these tensors say they are
    monkeypatch.setattr(_lib, "device_of", lambda tensors, what: -1)
    monkeypatch.setattr(_lib, "scratch", lambda nbytes, device, stream=None: real_empty(nbytes, dtype=torch.uint8))
    return seen


def _transposed(*shape):
    return torch.randn(shape[:-2] + (shape[-1], shape[-2])).transpose(-1, -2)


def _expanded(*shape):
    return torch.randn(()).expand(shape)


@pytest.mark.parametrize("grad", [_transposed, _expanded])
def test_copies_of_gradients_live_over_the_launch(launches, grad):
    import newton_schulz_orthogonalized_amd as nso

    def leaf(*shape):
        return torch.randn(shape).requires_grad_()
    r, y, w = leaf(50, 24), leaf(50, 24), leaf(24)
    torch.autograd.backward(nso.residual_norm(r, y, pre_weight=w), (grad(50, 24), grad(50, 24)))
    torch.autograd.backward(nso.rms_norm(r, w), grad(50, 24))
    x, wg, wu = leaf(50, 24), leaf(30, 24), leaf(30, 24)
    for save in (True, False):
        torch.autograd.backward(nso.gated_mlp(x, wg, wu, save_gates=save), grad(50, 30))
    q, k = leaf(2, 5, 4, 8), leaf(2, 5, 1, 8)
    freqs = nso.rotary_frequencies(8, device="cpu")
    torch.autograd.backward(nso.rotary(q, k, freqs=freqs), (grad(2, 5, 4, 8), torch.randn(2, 5, 1, 8)))
    assert [n for n, _ in launches] == [2, 1, 1, 1, 1]
    assert [lost for _, lost in launches if lost] == []
