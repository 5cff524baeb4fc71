"""Where the tensor-level calls allocate when they are given a stream of their
own: on that stream, behind whatever used the memory there before. Without a
GPU: streams are stand-ins, allocations are noted, and no kernel is called."""

import contextlib

import pytest
import torch


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def notes(monkeypatch):
    """(stream current at each allocation, streams recorded on buffers) of the
    calls made under this fixture; the caller's current stream is 11."""
    from newton_schulz_orthogonalized_amd import _lib
    current, made, tied = [FakeStream(11)], [], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def noting(real):
        def make(*args, device=None, **kw):
            made.append(current[-1].cuda_stream)
            return real(*args, **kw)
        return make

    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: FakeStream(h))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: FakeStream(0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 11, raising=False)
    monkeypatch.setattr(torch, "empty", noting(torch.empty))
    monkeypatch.setattr(torch, "empty_like", noting(torch.empty_like))
    monkeypatch.setattr(_lib, "device_of", lambda tensors, what: 0)
    monkeypatch.setattr(_lib, "tie_to_stream", lambda buf, s, current=None: s is None or tied.append(getattr(s, "cuda_stream", s)))
    for name in ("mu_muon_step_scaled", "mu_muon_orthogonalize", "mu_adamw_step_scaled", "mu_qk_clip", "mu_grad_norm",
                 "mu_clip_grads", "mu_embedding", "mu_embedding_grad", "mu_qk_max_logits"):
        monkeypatch.setattr(_lib, name, lambda *a, **k: None)
    return made, tied


def _calls():
    import newton_schulz_orthogonalized_amd as nso
    w, g, m, v = (torch.zeros(32, 64) for _ in range(4))
    tok = torch.zeros(32, dtype=torch.int64)
    q = torch.zeros(65, 4096, 2, 8)
    lens = torch.zeros(65, dtype=torch.int32)
    # name, call, buffers it allocates (results and workspace), results among them
    return [
        ("muon_step", lambda s: nso.muon_step([w], [g], [m], lr=0.1, weight_decay=0.0, stream=s), 1, 0),
        ("orthogonalize", lambda s: nso.orthogonalize([w, g], stream=s), 3, 2),
        ("adamw_step", lambda s: nso.adamw_step([w], [g], [m], [v], lr=0.1, weight_decay=0.0, stream=s), 1, 0),
        ("qk_clip", lambda s: nso.qk_clip([w], [g], [torch.zeros(2)], q_heads=2, k_heads=2, stream=s), 1, 0),
        ("grad_norm", lambda s: nso.grad_norm([w], stream=s), 2, 1),
        ("clip_grads", lambda s: nso.clip_grads([w], 1.0, stream=s), 2, 1),
        ("embedding", lambda s: nso.embedding(tok, w, stream=s), 1, 1),
        ("embedding_grad", lambda s: nso.embedding_grad(tok, w, 32, stream=s), 2, 1),
        ("qk_max_logits", lambda s: nso.qk_max_logits(q, q, lengths=lens, stream=s), 2, 1),
    ]


@pytest.mark.parametrize("which", range(9))
@pytest.mark.parametrize("stream,handle", [(FakeStream(22), 22), (33, 33), (0, 0)])
def test_buffers_come_from_the_launch_stream(notes, which, stream, handle):
    """stream: a torch stream, a raw handle, the null stream."""
    made, tied = notes
    name, call, buffers, results = _calls()[which]
    made.clear()
    call(stream)
    # (an unaligned scratch buffer is replaced by a second one)
    assert len(made) in (buffers, buffers + 1) and set(made) == {handle}, (name, made)
    assert tied == [11] * results, (name, tied)     # a result is read on the caller's stream next


@pytest.mark.parametrize("which", range(9))
def test_without_a_stream_the_current_one_is_used(notes, which):
    made, tied = notes
    name, call, _, _ = _calls()[which]
    made.clear()
    call(None)
    assert set(made) == {11} and tied == [], name
