"""Refusals of the operators that feed the optimizer step (gradient norm and
clipping, embedding, attention max logits), on a machine without a GPU: the C
entry points return a status before any HIP call, the Python calls raise."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import feed_oracle as F

A = 0x7f0000000000   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from newton_schulz_orthogonalized_amd import _lib
    return _lib


def _grads(lib, *items):
    d = dict(grad=A, out=None, numel=64, dtype=lib.MU_F32, out_dtype=lib.MU_F32)
    return (lib.MuGrad * max(1, len(items)))(*[lib.MuGrad(**{**d, **kw}) for kw in items])


def _norm(lib, arr, n, max_norm=1.0, eps=1e-6, norm=A + (1 << 30), scale=None, ws=A + (2 << 30), nb=1 << 20, clip=False):
    fn = lib.LIB.mu_clip_grads if clip else lib.LIB.mu_grad_norm
    return fn(ctypes.cast(arr, ctypes.c_void_p), n, max_norm, eps, norm, scale, ws, nb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), 2), (dict(numel=-1), 1), (dict(grad=None), 1), (dict(grad=A + 2), 3),
])
def test_bad_gradient_rejected(lib, kw, code):
    assert _norm(lib, _grads(lib, kw), 1) == code
    assert lib.mu_last_error() != ""


def test_bad_norm_arguments_rejected(lib):
    g = _grads(lib, {})
    assert _norm(lib, g, -1) == lib.MU_ERR_INVALID_ARG
    assert lib.LIB.mu_grad_norm(None, 1, 1.0, 1e-6, A, None, A, 4096, None) == lib.MU_ERR_INVALID_ARG
    for kw in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(eps=-1.0), dict(eps=float("inf")), dict(norm=None)):
        assert _norm(lib, g, 1, **kw) == lib.MU_ERR_INVALID_ARG, kw
    assert _norm(lib, g, 1, norm=A + 2) == lib.MU_ERR_LAYOUT
    for kw in (dict(ws=None), dict(ws=A + 16), dict(nb=8)):
        assert _norm(lib, g, 1, **kw) == lib.MU_ERR_WORKSPACE, kw


def test_bad_clip_outputs_rejected(lib):
    ok = dict(out=A + (1 << 20))
    assert _norm(lib, _grads(lib, dict(out=None)), 1, clip=True) == lib.MU_ERR_INVALID_ARG
    assert _norm(lib, _grads(lib, {**ok, "out_dtype": 9}), 1, clip=True) == lib.MU_ERR_DTYPE
    assert _norm(lib, _grads(lib, dict(out=A + (1 << 20) + 1)), 1, clip=True) == lib.MU_ERR_LAYOUT
    assert _norm(lib, _grads(lib, dict(out=A + 4)), 1, clip=True) == lib.MU_ERR_LAYOUT           # overlaps its input
    assert _norm(lib, _grads(lib, dict(out=A), dict(out=A)), 2, clip=True) == lib.MU_ERR_LAYOUT  # one buffer twice in place
    for kw in (dict(norm=A + 8), dict(scale=A + (1 << 20)), dict(norm=A + (1 << 30), scale=A + (1 << 30))):
        assert _norm(lib, _grads(lib, ok), 1, clip=True, **kw) == lib.MU_ERR_LAYOUT, kw          # results inside buffers
    # the same buffer as another type is not an in-place call
    assert _norm(lib, _grads(lib, dict(out=A, out_dtype=lib.MU_BF16)), 1, clip=True) == lib.MU_ERR_LAYOUT


def test_workspace_query_of_gradients(lib):
    need = ctypes.c_size_t(1)
    g = _grads(lib, dict(numel=0))
    assert lib.LIB.mu_grad_norm_workspace_size(ctypes.cast(g, ctypes.c_void_p), 1, ctypes.byref(need)) == 0
    assert need.value == 0
    assert lib.LIB.mu_grad_norm_workspace_size(ctypes.cast(g, ctypes.c_void_p), 1, None) == lib.MU_ERR_INVALID_ARG
    many = _grads(lib, *[dict(numel=10 ** 9)] * 400)
    assert lib.LIB.mu_grad_norm_workspace_size(ctypes.cast(many, ctypes.c_void_p), 400, ctypes.byref(need)) == 0
    assert 0 < need.value <= 1 << 20


def _lookup(lib, **kw):
    d = dict(tokens=A, weight=A + (1 << 30), out=A + (2 << 30), n_tokens=8, vocab=16, dim=32, token_bits=64,
             dtype=lib.MU_BF16, scale=1.0, pad0=0)
    return lib.LIB.mu_embedding(ctypes.byref(lib.MuLookup(**{**d, **kw})), None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=None), 1), (dict(weight=None), 1), (dict(out=None), 1), (dict(n_tokens=-1), 1), (dict(n_tokens=1 << 31), 1),
    (dict(n_tokens=1 << 29, dim=1 << 20, weight=1 << 52, out=1 << 53), 1),
    (dict(vocab=0), 1), (dict(dim=0), 1), (dict(dim=(1 << 21) + 1), 1), (dict(scale=float("inf")), 1), (dict(token_bits=16), 2),
    (dict(dtype=5), 2), (dict(tokens=A + 4), 3), (dict(weight=A + (1 << 30) + 1), 3), (dict(out=A + (1 << 30) + 64), 3),
    (dict(out=A), 3),
])
def test_bad_lookup_rejected(lib, kw, code):
    assert _lookup(lib, **kw) == code
    assert lib.LIB.mu_embedding(None, None) == lib.MU_ERR_INVALID_ARG


def test_empty_lookup_is_nothing(lib):
    assert _lookup(lib, n_tokens=0, tokens=None, out=None) == lib.MU_OK


def _rowgrad(lib, ws=A + (4 << 30), nb=1 << 30, **kw):
    d = dict(tokens=A, rows=A + (1 << 30), grad=A + (2 << 30), n_tokens=8, vocab=16, dim=32, padding_idx=-1, token_bits=64,
             row_dtype=lib.MU_BF16, grad_dtype=lib.MU_F32, accumulate=0, scale=1.0, pad0=0)
    return lib.LIB.mu_embedding_grad(ctypes.byref(lib.MuRowgrad(**{**d, **kw})), ws, nb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=None), 1), (dict(rows=None), 1), (dict(grad=None), 1), (dict(n_tokens=-1), 1), (dict(vocab=0), 1),
    (dict(n_tokens=(1 << 30) + 1), 1),
    (dict(dim=0), 1), (dict(padding_idx=16), 1), (dict(padding_idx=-2), 1), (dict(accumulate=2), 1),
    (dict(scale=float("nan")), 1), (dict(row_dtype=3), 2), (dict(grad_dtype=3), 2), (dict(token_bits=8), 2),
    (dict(rows=A + (1 << 30) + 1), 3), (dict(grad=A + (2 << 30) + 2), 3), (dict(grad=A + (1 << 30)), 3),
])
def test_bad_rowgrad_rejected(lib, kw, code):
    assert _rowgrad(lib, **kw) == code


def test_rowgrad_workspace_rejected(lib):
    need = ctypes.c_size_t(0)
    e = lib.MuRowgrad(tokens=A, rows=A + (1 << 30), grad=A + (2 << 30), n_tokens=8, vocab=16, dim=32, padding_idx=-1,
                      token_bits=64, row_dtype=lib.MU_BF16, grad_dtype=lib.MU_F32, accumulate=0, scale=1.0, pad0=0)
    assert lib.LIB.mu_embedding_grad_workspace_size(ctypes.byref(e), ctypes.byref(need)) == 0 and need.value > 0
    for kw in (dict(ws=None), dict(ws=A + (4 << 30) + 8), dict(nb=need.value - 1)):
        assert _rowgrad(lib, **kw) == lib.MU_ERR_WORKSPACE, kw
    assert lib.LIB.mu_embedding_grad_workspace_size(ctypes.byref(e), None) == lib.MU_ERR_INVALID_ARG


def test_empty_accumulation_is_nothing(lib):
    assert _rowgrad(lib, n_tokens=0, tokens=None, rows=None, accumulate=1) == lib.MU_OK


def _qk(lib, ws=A + (3 << 30), nb=1 << 20, **kw):
    d = dict(q=A, k=A + (1 << 30), q_stride_b=4096, q_stride_s=256, q_stride_h=64, k_stride_b=4096, k_stride_s=256,
             k_stride_h=64, q_len=16, k_len=16, batch=2, q_heads=4, k_heads=2, dim=64, q_lengths=None, k_lengths=None,
             cu_q=None, cu_k=None, dtype=lib.MU_BF16, causal=1, accumulate=0, scale=0.125, max_logit=A + (2 << 30))
    return lib.LIB.mu_qk_max_logits(ctypes.byref(lib.MuQkLogits(**{**d, **kw})), ws, nb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(max_logit=None), 1), (dict(batch=-1), 1), (dict(q_len=-1), 1),
    (dict(q_heads=0), 1), (dict(k_heads=3), 1), (dict(k_heads=0), 1), (dict(dim=0), 1), (dict(dim=257), 1),
    (dict(causal=2), 1), (dict(accumulate=-1), 1), (dict(scale=float("nan")), 1), (dict(q_stride_s=-1), 1),
    (dict(cu_k=A), 1), (dict(cu_q=A, q_lengths=A), 1), (dict(cu_q=A, k_len=17), 1), (dict(dtype=2), 2),
    (dict(q=A + 1), 3), (dict(max_logit=A + 2), 3), (dict(q_lengths=A + 2), 3),
    # max_logit inside q, at the end of k, among the lengths
    (dict(max_logit=A + 64), 3), (dict(max_logit=A + (1 << 30) + 2 * (4096 + 15 * 256 + 64 + 63) - 2), 3),
    (dict(q_lengths=A + (2 << 30) + 12), 3), (dict(q_stride_b=1 << 62), 1), (dict(k_stride_s=1 << 47), 1),
])
def test_bad_qk_rejected(lib, kw, code):
    assert _qk(lib, **kw) == code


def test_qk_workspace_rejected(lib):
    for kw in (dict(ws=None), dict(ws=A + 8), dict(nb=16)):
        assert _qk(lib, batch=65, q_len=4096, k_len=4096, q_lengths=A, **kw) == lib.MU_ERR_WORKSPACE, kw


def test_empty_accumulating_qk_is_nothing(lib):
    assert _qk(lib, batch=0, accumulate=1) == lib.MU_OK
    assert _qk(lib, q_len=0, q=None, accumulate=1) == lib.MU_OK


def test_python_calls_refuse_what_the_library_cannot_take():
    import newton_schulz_orthogonalized_amd as nso
    x = torch.zeros(4, 8)
    tok = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="on a GPU"):
        nso.grad_norm([x])
    with pytest.raises(ValueError, match="on a GPU"):
        nso.embedding(tok, x)
    with pytest.raises(ValueError, match="on a GPU"):
        nso.embedding_grad(tok, x, 4)
    with pytest.raises(ValueError, match="on a GPU"):
        nso.qk_max_logits(torch.zeros(1, 2, 2, 4), torch.zeros(1, 2, 2, 4))
    with pytest.raises(TypeError):
        nso.grad_norm([x.half()])
    with pytest.raises(ValueError, match="contiguous"):
        nso.grad_norm([x.t()])
    with pytest.raises(ValueError):
        nso.clip_grads([x], 1.0, outs=[])
    with pytest.raises(ValueError):
        nso.clip_grads([x], 1.0, outs=[torch.zeros(8, 4)])
    with pytest.raises(TypeError):
        nso.grad_norm([x], norm_out=torch.zeros((), dtype=torch.float64))
    with pytest.raises(ValueError):
        nso.embedding(tok, x, padding_idx=4)
    with pytest.raises(ValueError):
        nso.embedding(tok, x.requires_grad_(), out=torch.zeros(4, 8))
    with pytest.raises(ValueError):
        nso.embedding_grad(tok, torch.zeros(4, 8), 4, accumulate=True)
    with pytest.raises(ValueError):
        nso.embedding_grad(tok, torch.zeros(4, 8), 4, out=torch.zeros(5, 8))
    with pytest.raises(TypeError):
        nso.embedding_grad(tok, torch.zeros(4, 8), 4, out=torch.zeros(4, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nso.qk_max_logits(torch.zeros(1, 2, 2, 4), torch.zeros(1, 2, 2, 4), accumulate=True)
    w = torch.nn.Parameter(torch.zeros(4, 8))
    with pytest.raises(ValueError):
        nso.MuonAdamW([{"params": [w], "kind": "muon"}], max_grad_norm=-1.0)
    with pytest.raises(ValueError, match="grad_scale"):
        nso.muon_step([x], [x], [x], lr=0.1, weight_decay=0.0, noalloc=True, grad_scale=torch.ones(()))


@pytest.mark.parametrize("requires_grad", [False, True])
def test_embedding_refuses_forward_mode(requires_grad):
    """A tangent would be lost without a word: the lookup works on addresses."""
    import torch.autograd.forward_ad as fw

    import newton_schulz_orthogonalized_amd as nso
    w, tok = torch.ones(4, 8, requires_grad=requires_grad), torch.zeros(3, dtype=torch.int64)
    with fw.dual_level():
        dual = fw.make_dual(w, torch.ones(4, 8))
        with pytest.raises(NotImplementedError, match="forward"):
            nso.embedding(tok, dual)
        with pytest.raises(NotImplementedError, match="forward"), torch.no_grad():
            nso.embedding(tok, dual, out=torch.zeros(3, 8))
        with pytest.raises(ValueError, match="on a GPU"):
            nso.embedding(tok, w)           # no tangent: refused for another reason
    with pytest.raises(ValueError, match="on a GPU"):
        nso.embedding(tok, w)


def test_marshalling_refuses_bad_shapes_and_types(lib):
    """What the binding checks for itself, on CPU tensors (nothing is called)."""
    q = torch.zeros(2, 6, 4, 8)
    out = torch.zeros(4)

    def call(q=q, k=q[:, :, :2], out=out, lengths=None, k_lengths=None, cu=None, cu_k=None):
        return lib.qk_logits(q, k, out, 1.0, True, lengths, k_lengths, cu, cu_k, False)
    call()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    for kw in (dict(q=q[0]), dict(k=q[:1]), dict(k=q[..., :4]), dict(out=torch.zeros(3)), dict(lengths=i32(1)),
               dict(cu_k=i32(0, 1, 2)), dict(cu=i32(0, 6)), dict(q=q.transpose(2, 3), k=q.transpose(2, 3))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(k=q.bfloat16()), dict(lengths=torch.tensor([1, 2]))):
        with pytest.raises(TypeError):
            call(**kw)
    packed = q[0]
    lib.qk_logits(packed, packed, out, 1.0, True, None, None, i32(0, 2, 6), None, False)
    with pytest.raises(ValueError):
        lib.qk_logits(packed, packed, out, 1.0, True, i32(1, 1), None, i32(0, 2, 6), None, False)
    with pytest.raises(ValueError):
        lib.qk_logits(packed, packed, out, 1.0, True, None, None, i32(), None, False)
    w = torch.zeros(5, 8)
    with pytest.raises(TypeError):
        lib.lookup(torch.zeros(3, dtype=torch.int16), w, torch.zeros(3, 8), 1.0)
    with pytest.raises(ValueError):
        lib.lookup(torch.zeros(3, dtype=torch.int64), w, torch.zeros(3, 7), 1.0)
    with pytest.raises(ValueError):
        lib.rowgrad(torch.zeros(3, dtype=torch.int64), torch.zeros(2, 8), w, 1.0, None, False)
    with pytest.raises(ValueError):
        lib.rowgrad(torch.zeros(3, dtype=torch.int64), torch.zeros(3, 8), w, 1.0, 5, False)
    with pytest.raises(TypeError):
        lib.grad_scale_ptr(torch.zeros(2))
    with pytest.raises(ValueError):
        lib.grad_scale_ptr(torch.zeros(()))


def test_scaled_steps_refuse_a_factor_in_their_buffers(lib):
    step = 1 << 30
    mat = (lib.MuMatrix * 1)(lib.MuMatrix(A, A + step, A + 2 * step, 16, 32, lib.MU_F32, 1, 1.0, None, None))
    ten = (lib.MuTensor * 1)(lib.MuTensor(A, A + step, A + 2 * step, A + 3 * step, 512, lib.MU_F32, 0.1, 0.0))
    mh, keep = lib.muon_hparams(0.1, 0.0)
    ah = lib.MuAdamwHparams(0.9, 0.95, 1e-8, 1)
    ws, nb = A + 8 * step, 1 << 28
    for at in (A, A + step + 64, A + 2 * step + 2044):
        assert lib.LIB.mu_muon_step_scaled(mat, 1, ctypes.byref(mh), at, ws, nb, None) == lib.MU_ERR_LAYOUT
        assert lib.LIB.mu_adamw_step_scaled(ten, 1, ctypes.byref(ah), at, ws, nb, None) == lib.MU_ERR_LAYOUT
    assert lib.LIB.mu_muon_step_scaled(mat, 1, ctypes.byref(mh), A - 2, ws, nb, None) == lib.MU_ERR_LAYOUT   # misaligned
    assert lib.LIB.mu_adamw_step_scaled(ten, 1, ctypes.byref(ah), A - 2, ws, nb, None) == lib.MU_ERR_LAYOUT
    del keep


def test_references_by_hand():
    assert F.grad_norm_ref([np.array([3.0]), np.array([[4.0]])]) == 5.0
    assert F.grad_norm_ref([np.array([3e200, 4e200])]) == pytest.approx(5e200, rel=1e-15)
    assert F.grad_norm_ref([]) == 0.0 and math.isnan(F.grad_norm_ref([np.array([np.nan, 1.0])]))
    assert F.clip_scale_ref(4.0, 2.0, 0.0) == 0.5 and F.clip_scale_ref(1.0, 2.0) == 1.0 and F.clip_scale_ref(0.0, 0.0, 0.0) == 1.0
    g, mag, n = F.embedding_grad_ref([1, 3, 1, 9, -1, 0], np.arange(12.0).reshape(6, 2), 4, scale=2.0, padding_idx=0)
    assert np.array_equal(g, [[0, 0], [8, 12], [0, 0], [4, 6]]) and list(n) == [0, 2, 0, 1]
    q = np.array([[[1.0, 0.0]], [[0.0, -3.0]]])
    k = np.array([[[2.0, 0.0]], [[5.0, 4.0]]])
    best, _ = F.qk_max_logits_ref([(q, k)], 1, -0.5, True)
    assert best[0] == 6.0     # |-0.5 * (-3 * 4)|; q0.k1 = 5 is not visible
    assert F.qk_max_logits_ref([(q, k[:1])], 1, 1.0, True)[0][0] == 0.0   # query 0 sees nothing, query 1 sees k0: 0
