"""Calls on a stream of their own while the caller's stream is still at work:
their buffers come from that stream's memory, and what the caller's stream does
with memory it has given back does not reach them. Exact comparisons: the same
call on an idle GPU gives the reference bits."""

import pytest
import torch

from gpu_util import need_gpu
from workloads import as_dtype, host_normal

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    import newton_schulz_orthogonalized_amd  # noqa: F401  (fails loudly without the library)
    yield


def _stream_of(t):
    """The stream whose memory a tensor lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in the caching allocator's memory")


def _calls():
    import newton_schulz_orthogonalized_amd as nso
    w = as_dtype(host_normal((500, 96), 91000), BF).cuda()
    tok = (torch.arange(20000, device="cuda") * 7919) % 500
    rows = as_dtype(host_normal((20000, 96), 91001), BF).cuda()
    q = as_dtype(host_normal((65, 70, 4, 32), 91002), BF).cuda()
    k = as_dtype(host_normal((65, 70, 2, 32), 91003), BF).cuda()
    lens = (torch.arange(65, device="cuda") % 71).int()
    x = as_dtype(host_normal((160, 96), 91004), FP).cuda()
    outs = [torch.empty_like(rows), torch.empty_like(x)]
    return {
        "grad_norm": lambda **kw: nso.grad_norm([rows, x], **kw),
        "clip_grads": lambda **kw: nso.clip_grads([rows, x], 0.5, outs=outs, **kw),
        "embedding": lambda **kw: nso.embedding(tok, w, scale=2.0, **kw),
        "embedding_grad": lambda **kw: nso.embedding_grad(tok, rows, 500, dtype=FP, **kw),
        "qk_max_logits": lambda **kw: nso.qk_max_logits(q, k, lengths=lens, **kw),
        "orthogonalize": lambda **kw: nso.orthogonalize([x], precision="f32", **kw)[0],
    }


NAMES = ["grad_norm", "clip_grads", "embedding", "embedding_grad", "qk_max_logits", "orthogonalize"]


@pytest.mark.parametrize("name", NAMES)
def test_results_lie_in_the_launch_streams_memory(name):
    call = _calls()[name]
    want = call()
    side, caller = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        got = call(stream=stream)
        torch.cuda.synchronize()
        assert _stream_of(got) == side.cuda_stream and torch.equal(got, want)
    with torch.cuda.stream(caller):    # the null stream, from another one
        got = call(stream=0)
    torch.cuda.synchronize()
    assert _stream_of(got) == 0 and torch.equal(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_callers_stream_still_writes(name):
    """The caller's stream waits, then writes into buffers that have been given
    back to the allocator already, of the sizes of the call's own."""
    call = _calls()[name]
    want = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(20_000_000)
        for n in (512, 1 << 16, 1 << 19, 20000 * 96 * 2):
            bufs = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(4)]
            for b in bufs:
                b.fill_(255)
            del b, bufs
        got = call(stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
