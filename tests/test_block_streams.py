"""Where the block's calls allocate when they are given a stream of their own: on
that stream, results recorded on the caller's. Without a GPU, as in
test_streams.py: streams are stand-ins and no kernel is called."""

import pytest
import torch

from test_streams import FakeStream, notes  # noqa: F401  (a fixture)


@pytest.fixture
def made_and_tied(notes, monkeypatch):  # noqa: F811
    from newton_schulz_orthogonalized_amd import _lib
    for name in ("mu_rotary", "mu_residual_norm", "mu_residual_norm_grad", "mu_gated_mlp", "mu_gated_mlp_grad"):
        monkeypatch.setattr(_lib, name, lambda *a, **k: None)
    return notes


def _calls():
    import newton_schulz_orthogonalized_amd as nso
    q, k = torch.zeros(2, 5, 4, 8), torch.zeros(2, 5, 1, 8)
    freqs = nso.rotary_frequencies(8, device="cpu")
    r, w = torch.zeros(40, 32), torch.ones(32)
    x, wg, wu, dh = torch.zeros(40, 30), torch.zeros(16, 30), torch.zeros(16, 30), torch.zeros(40, 16)
    # name, call, buffers it allocates (results and workspace), results among them
    return [
        ("rotary", lambda s: nso.rotary(q, k, freqs=freqs, stream=s), 2, 2),
        ("residual_norm", lambda s: nso.residual_norm(r, r.clone(), pre_weight=w, stream=s), 2, 2),
        ("rms_norm", lambda s: nso.rms_norm(r, w, stream=s), 1, 1),
        ("residual_norm_grad", lambda s: nso.residual_norm_grad(r, r, r, r, pre_weight=w, stream=s), 4, 3),
        ("gated_mlp", lambda s: nso.gated_mlp(x, wg, wu, stream=s), 2, 1),
        ("gated_mlp_grad", lambda s: nso.gated_mlp_grad(dh, x, wg, wu, stream=s), 4, 3),
    ]


@pytest.mark.parametrize("which", range(6))
@pytest.mark.parametrize("stream,handle", [(FakeStream(22), 22), (33, 33), (0, 0)])
def test_buffers_come_from_the_launch_stream(made_and_tied, which, stream, handle):
    made, tied = made_and_tied
    name, call, buffers, results = _calls()[which]
    made.clear()
    call(stream)
    # (an unaligned scratch buffer is replaced by a second one)
    assert len(made) in (buffers, buffers + 1) and set(made) == {handle}, (name, made)
    assert tied == [11] * results, (name, tied)


@pytest.mark.parametrize("which", range(6))
def test_without_a_stream_the_current_one_is_used(made_and_tied, which, monkeypatch):
    made, tied = made_and_tied
    real = torch.empty     # (without a stream results are asked for by device number)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: real(*a, device=None, **k))
    name, call, _, _ = _calls()[which]
    made.clear()
    call(None)
    assert set(made) == {11} and tied == [], name
