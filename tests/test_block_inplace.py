"""Buffers of the caller's that the block's calls write count as changed in place:
a backward pass that saved one of them refuses, as it does where torch changed
it, and does not take the new values. Without a GPU, as in test_block_streams.py:
streams are stand-ins and no kernel is called."""

import pytest
import torch

from test_block_streams import made_and_tied  # noqa: F401  (a fixture)
from test_streams import notes  # noqa: F401  (a fixture)


@pytest.fixture(autouse=True)
def _stand_ins(made_and_tied, monkeypatch):  # noqa: F811
    from newton_schulz_orthogonalized_amd import _lib
    real = torch.empty
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)      # where these tensors say they are
    monkeypatch.setattr(_lib, "device_of", lambda tensors, what: -1)
    monkeypatch.setattr(_lib, "scratch", lambda nbytes, device, stream=None: real(nbytes, dtype=torch.uint8))


def _writes():
    """name, call that writes into buffers of the caller's, those buffers."""
    import newton_schulz_orthogonalized_amd as nso
    freqs = nso.rotary_frequencies(8, device="cpu")
    q, k, o = torch.zeros(2, 5, 4, 8), torch.zeros(2, 5, 1, 8), torch.zeros(2, 5, 4, 8)
    r, y, n = (torch.zeros(6, 8) for _ in range(3))
    x, w, h, gates = torch.zeros(6, 8), torch.zeros(10, 8), torch.zeros(6, 10), torch.zeros(2, 6, 10)
    dg, du = torch.zeros(10, 8), torch.zeros(10, 8)
    return [
        ("rotary in place", lambda: nso.rotary(q, k, freqs=freqs, out=(q, k)), (q, k)),
        ("rotary", lambda: nso.rotary(q, freqs=freqs, out=o), (o,)),
        ("residual_norm in place", lambda: nso.residual_norm(r, y, out=r, normed_out=y), (r, y)),
        ("residual_norm", lambda: nso.residual_norm(r, y, out=n), (n,)),
        ("rms_norm", lambda: nso.rms_norm(r, out=r), (r,)),
        ("gated_mlp", lambda: nso.gated_mlp(x, w, w, out=h, gates_out=gates), (h, gates)),
        ("gated_mlp_grad", lambda: nso.gated_mlp_grad(h, x, w, w, d_gate=dg, d_up=du, accumulate=True), (dg, du)),
    ]


@pytest.mark.parametrize("which", range(7))
def test_written_buffers_count_as_changed(which):
    name, call, written = _writes()[which]
    before = [t._version for t in written]
    call()
    assert all(t._version > v for t, v in zip(written, before)), name


@pytest.mark.parametrize("which", range(7))
def test_a_backward_pass_refuses_what_was_overwritten(which):
    """Torch's own product saves the buffer."""
    name, call, written = _writes()[which]
    w = torch.ones(written[0].shape, requires_grad=True)
    loss = (written[0] * w).sum()
    with torch.no_grad():
        call()
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()


def test_the_calls_own_saved_tensors():
    """A residual, an update and an x that earlier calls saved, overwritten by the next ones."""
    import newton_schulz_orthogonalized_amd as nso
    w = torch.ones(8, requires_grad=True)
    wg = torch.ones(10, 8, requires_grad=True)
    for first, overwrite in (
            (lambda r, y: nso.residual_norm(r, y, pre_weight=w)[1], lambda r, y, n: nso.residual_norm(y, r, normed_out=y)),
            (lambda r, y: nso.rms_norm(r, w), lambda r, y, n: nso.rms_norm(r, out=r)),
            (lambda r, y: nso.gated_mlp(r, wg, wg), lambda r, y, n: nso.residual_norm(r, y, out=r))):
        r, y = torch.ones(6, 8), torch.ones(6, 8)
        n = first(r, y)
        with torch.no_grad():
            overwrite(r, y, n)
        with pytest.raises(RuntimeError, match="inplace"):
            n.backward(torch.ones_like(n))


def test_results_of_their_own_are_not_counted_twice():
    """Nothing of the caller's is written: inputs keep their versions."""
    import newton_schulz_orthogonalized_amd as nso
    r, y, w = torch.ones(6, 8), torch.ones(6, 8), torch.ones(10, 8)
    new, n = nso.residual_norm(r, y)
    h = nso.gated_mlp(r, w, w)
    nso.gated_mlp_grad(h, r, w, w)
    nso.residual_norm_grad(new, n, new, y)
    assert [t._version for t in (r, y, w)] == [0, 0, 0]
