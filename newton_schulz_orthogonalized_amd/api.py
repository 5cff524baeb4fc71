"""Tensor-level calls over the C ABI: one Muon step, orthogonalise-only, AdamW,
QK-Clip, and what feeds them (gradient norm and clipping, the embedding and its
gradient, attention max logits).

Each function marshals torch tensors into the library's descriptor lists,
allocates the workspace the library asks for (unless one is passed in) and
enqueues the work on `stream` (default: the current stream). Workspaces and
results allocated here come from `stream`'s share of the caching allocator, so
that neither the work that used their memory before nor the work that gets it
next overlaps the library's kernels; a result is recorded on the current stream
too. The caller orders `stream` behind what made the inputs, and its own use of
the results behind `stream`. Nothing here computes. Of the results only
embedding's carries a gradient.
"""

from __future__ import annotations

import math
from typing import Optional, Sequence

import torch
from torch.autograd import forward_ad

from . import _lib


def muon_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], moms: Sequence[torch.Tensor], *,
              lr: float, weight_decay: float, mu: float = 0.95, nesterov: bool = True,
              heads: Optional[Sequence[int]] = None, scales: Optional[Sequence[float]] = None,
              ns_steps: int = 5, coeffs=None, precision: str = "bf16", norm_eps: float = 1e-7,
              norm_outs: Optional[Sequence[torch.Tensor]] = None,
              ortho_outs: Optional[Sequence[Optional[torch.Tensor]]] = None,
              workspace: Optional[torch.Tensor] = None, stream=None, noalloc: bool = False,
              cautious_wd: bool = False, grad_scale: Optional[torch.Tensor] = None) -> None:
    """In-place Muon step over 2-D params (momentum fp32, grads in the param dtype).

    noalloc=True runs mu_muon_step_noalloc: no workspace is allocated, the
    library's static per-GPU scratch (MU_NOALLOC_SCRATCH_BYTES) is used, and
    calls on one GPU must not overlap in time. cautious_wd=True applies the
    decay only where it agrees in sign with the update (see the header).
    grad_scale (one float32 on the GPU, grad_norm's factor) multiplies every
    gradient as it is read: a clipped step that writes no scaled gradients."""
    mats, n = _lib.matrices(params, grads, moms, heads, scales, norm_outs, ortho_outs)
    hp, keep = _lib.muon_hparams(lr, weight_decay, mu, nesterov, norm_eps, ns_steps, coeffs, precision, cautious_wd)
    if n == 0:
        return
    if noalloc:
        if workspace is not None:
            raise ValueError("noalloc=True takes no workspace")
        if grad_scale is not None:
            raise ValueError("noalloc=True takes no grad_scale")
        _lib.mu_muon_step_noalloc(mats, n, hp, stream)
        del keep
        return
    _same_gpu(grad_scale, params)
    if workspace is None:
        workspace = _lib.workspace(_lib.mu_muon_workspace_size(mats, n, hp), params[0].device, stream)
    _lib.mu_muon_step_scaled(mats, n, hp, grad_scale, workspace, stream)
    del keep


def _same_gpu(grad_scale: Optional[torch.Tensor], params):
    if grad_scale is not None and grad_scale.is_cuda and params[0].is_cuda and grad_scale.device != params[0].device:
        raise ValueError("grad_scale must be on the parameters' GPU")


def muon_workspace_bytes(params, grads, moms, *, heads=None, ns_steps: int = 5, coeffs=None,
                         precision: str = "bf16") -> int:
    mats, n = _lib.matrices(params, grads, moms, heads)
    hp, keep = _lib.muon_hparams(0.0, 0.0, 0.95, True, 1e-7, ns_steps, coeffs, precision)
    return _lib.mu_muon_workspace_size(mats, n, hp)


def orthogonalize(inputs: Sequence[torch.Tensor], *, heads: Optional[Sequence[int]] = None, ns_steps: int = 5,
                  coeffs=None, precision: str = "bf16", norm_eps: float = 1e-7,
                  outputs: Optional[Sequence[torch.Tensor]] = None,
                  norm_outs: Optional[Sequence[torch.Tensor]] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """Frobenius-normalise and Newton-Schulz-orthogonalise each input (per head)."""
    if outputs is None:
        outputs = [_lib.allocate(lambda: torch.empty_like(x), x.device, stream, returned=True) for x in inputs]
    xs, n = _lib.orthos(inputs, outputs, heads, norm_outs)
    hp, keep = _lib.muon_hparams(0.0, 0.0, 0.95, True, norm_eps, ns_steps, coeffs, precision)
    if n == 0:
        return list(outputs)
    if workspace is None:
        workspace = _lib.workspace(_lib.mu_ortho_workspace_size(xs, n, hp), inputs[0].device, stream)
    _lib.mu_muon_orthogonalize(xs, n, hp, workspace, stream)
    del keep
    return list(outputs)


def adamw_step(params, grads, exp_avgs, exp_avg_sqs, *, lr, weight_decay, beta1: float = 0.9,
               beta2: float = 0.95, eps: float = 1e-8, step: int = 1,
               workspace: Optional[torch.Tensor] = None, stream=None,
               grad_scale: Optional[torch.Tensor] = None) -> None:
    """In-place AdamW step over a flat list; lr and weight_decay may be per-tensor lists.
    grad_scale as in muon_step."""
    n = len(params)
    lrs = list(lr) if isinstance(lr, (list, tuple)) else [lr] * n
    wds = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * n
    ts, n = _lib.tensors(params, grads, exp_avgs, exp_avg_sqs, lrs, wds)
    if n == 0:
        return
    _same_gpu(grad_scale, params)
    if workspace is None:
        workspace = _lib.workspace(_lib.mu_adamw_workspace_size(n), params[0].device, stream)
    _lib.mu_adamw_step_scaled(ts, n, beta1, beta2, eps, step, grad_scale, workspace, stream)


def qk_clip(wqs, wks, max_logits, *, q_heads, k_heads, tau: float = 100.0, gamma_outs=None,
            workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """QK-Clip over attention layers (one (wq, wk, max_logit) per layer): heads
    whose max |logit| exceeds tau get their query and key rows scaled by
    tau / max_logit, in place. q_heads / k_heads are per layer (or one int)."""
    n = len(wqs)
    qh = list(q_heads) if isinstance(q_heads, (list, tuple)) else [q_heads] * n
    kh = list(k_heads) if isinstance(k_heads, (list, tuple)) else [k_heads] * n
    pairs, n = _lib.qk_pairs(wqs, wks, max_logits, qh, kh, gamma_outs)
    if n == 0:
        return
    if workspace is None:
        workspace = _lib.workspace(_lib.mu_qk_clip_workspace_size(pairs, n), wqs[0].device, stream)
    _lib.mu_qk_clip(pairs, n, tau, workspace, stream)


def _on(device: int, stream, call, *args):
    """call(stream, *args) with GPU `device` current; the stream is the caller's
    or the device's current one (as its handle: a torch.cuda.Stream object costs
    more to make than a small kernel to run)."""
    if device != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _on(device, stream, call, *args)
    return call(torch._C._cuda_getCurrentRawStream(device) if stream is None else stream, *args)


def _new(shape, dtype, device: int, stream) -> torch.Tensor:
    return _lib.allocate(lambda: torch.empty(shape, dtype=dtype, device=torch.device("cuda", device)), device, stream,
                         returned=True)


def grad_norm(grads: Sequence[torch.Tensor], *, max_norm: float = math.inf, eps: float = 1e-6,
              norm_out: Optional[torch.Tensor] = None, scale_out: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The global 2-norm of a list of float32 and bfloat16 tensors, as a float32
    scalar on the GPU (no synchronisation). scale_out receives the factor
    min(1, max_norm / (norm + eps)), which muon_step and adamw_step take as
    grad_scale; without a bound (the default) 1 unless the norm is NaN."""
    return _norm(grads, None, max_norm, eps, norm_out, scale_out, workspace, stream)


def clip_grads(grads: Sequence[torch.Tensor], max_norm: float, *, outs: Optional[Sequence[torch.Tensor]] = None,
               eps: float = 1e-6, norm_out: Optional[torch.Tensor] = None, scale_out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Scale gradients to a global norm of at most max_norm: in place, or into
    `outs` (of either type, e.g. float32 accumulation buffers into the bfloat16
    gradients the steps take). Returns the norm before scaling, as grad_norm."""
    return _norm(grads, grads if outs is None else outs, max_norm, eps, norm_out, scale_out, workspace, stream)


def _norm(grads, outs, max_norm, eps, norm_out, scale_out, workspace, stream):
    if not isinstance(grads, (list, tuple)):
        raise TypeError("grads must be a list or tuple of tensors")
    gs, n = _lib.gradients(grads, outs)
    for t in (norm_out, scale_out):
        if t is not None and (t.dtype != torch.float32 or t.numel() != 1):
            raise TypeError("norm_out and scale_out must be one float32 element")
    others = () if outs is None or outs is grads else outs
    device = _lib.device_of((*grads, *others, norm_out, scale_out, workspace), "gradients and outputs")

    def call(st):
        out = _new((), torch.float32, device, stream) if norm_out is None else norm_out
        ws = _lib.scratch(_lib.mu_grad_norm_workspace_size(gs, n), device, stream) if workspace is None else workspace
        run = _lib.mu_grad_norm if outs is None else _lib.mu_clip_grads
        run(gs, n, max_norm, eps, out, scale_out, ws, st)
        return out
    return _on(device, stream, call)


def embedding(tokens: torch.Tensor, weight: torch.Tensor, *, scale: float = 1.0, padding_idx: Optional[int] = None,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """scale * weight[tokens] for int32 or int64 tokens of any shape. A token
    outside the table reads nothing and gives a row of NaN. Differentiable in
    weight (embedding_grad; the row padding_idx gets no gradient) unless `out`
    is given; forward mode is refused. A captured backward pass needs what torch
    asks of any: no eager graph of the same leaf alive meanwhile."""
    if padding_idx is not None and not 0 <= padding_idx < weight.shape[0]:
        raise ValueError("padding_idx must name a row of the weight")
    if forward_ad._current_level >= 0 and forward_ad.unpack_dual(weight).tangent is not None:
        raise NotImplementedError("embedding has no forward-mode derivative")
    if torch.is_grad_enabled() and weight.requires_grad:
        if out is not None:
            raise ValueError("out takes no gradient: call under torch.no_grad()")
        return _Embedding.apply(tokens, weight, float(scale), padding_idx, stream)
    return _lookup(tokens, weight, scale, out, stream)


def _lookup(tokens, weight, scale, out, stream):
    device = _lib.device_of((tokens, weight, out), "tokens, weight and out")

    def call(st):
        o = _new(tokens.shape + weight.shape[1:], weight.dtype, device, stream) if out is None else out
        _lib.mu_embedding(_lib.lookup(tokens, weight, o, scale), st)
        return o
    return _on(device, stream, call)


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, weight, scale, padding_idx, stream):
        ctx.save_for_backward(tokens)
        ctx.spec = (weight.shape[0], weight.dtype, scale, padding_idx)
        return _lookup(tokens, weight, scale, None, stream)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, rows):
        (tokens,) = ctx.saved_tensors
        vocab, dtype, scale, padding_idx = ctx.spec
        # autograd hands in expanded or transposed gradients too
        grad = embedding_grad(tokens, rows.contiguous(), vocab, scale=scale, padding_idx=padding_idx, dtype=dtype)
        return None, grad, None, None, None


def embedding_grad(tokens: torch.Tensor, rows: torch.Tensor, num_embeddings: int, *, scale: float = 1.0,
                   padding_idx: Optional[int] = None, dtype: Optional[torch.dtype] = None,
                   out: Optional[torch.Tensor] = None, accumulate: bool = False,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The dense gradient [num_embeddings, dim] of an embedding from its rows'
    gradients: row v is scale times the float32 sum of rows[t] over tokens[t] ==
    v, in a fixed order. Tokens outside the table and padding_idx add nothing.
    `out` receives it (accumulate=True: added to it); dtype is that of a new
    one (default: the rows')."""
    if accumulate and out is None:
        raise ValueError("accumulate=True needs out")
    if out is not None and (out.dim() != 2 or out.shape[0] != num_embeddings):
        raise ValueError("out must be [num_embeddings, dim]")
    if out is not None and dtype is not None and out.dtype != dtype:
        raise TypeError("dtype differs from out's")
    device = _lib.device_of((tokens, rows, out, workspace), "tokens, rows and out")

    def call(st):
        g = out
        if g is None:
            g = _new((num_embeddings, rows.shape[-1]), rows.dtype if dtype is None else dtype, device, stream)
        e = _lib.rowgrad(tokens, rows, g, scale, padding_idx, accumulate)
        ws = _lib.scratch(_lib.mu_embedding_grad_workspace_size(e), device, stream) if workspace is None else workspace
        _lib.mu_embedding_grad(e, ws, st)
        return g
    return _on(device, stream, call)


def qk_max_logits(q: torch.Tensor, k: torch.Tensor, *, scale: Optional[float] = None, causal: bool = True,
                  lengths: Optional[torch.Tensor] = None, k_lengths: Optional[torch.Tensor] = None,
                  cu_seqlens: Optional[torch.Tensor] = None, cu_seqlens_k: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, accumulate: bool = False,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The largest |scale * q.k| of each query head over the visible pairs of a
    batch, float32 [q_heads]: the max_logits that qk_clip takes.

    q [batch, length, q_heads, dim] and k [batch, length, k_heads, dim] may be
    strided views (of a fused projection) with a contiguous last dimension;
    `lengths` and `k_lengths` (int32 [batch]; k_lengths defaults to lengths) cut
    padded rows short. With cu_seqlens (int32 [sequences + 1]; cu_seqlens_k
    defaults to it) they are packed, [rows, heads, dim]. scale defaults to
    dim ** -0.5. causal: query i of a sequence sees keys j <= i + (keys -
    queries). A head without a visible pair gets 0. accumulate=True keeps what
    is larger in `out`, over the micro-batches of a step."""
    if accumulate and out is None:
        raise ValueError("accumulate=True needs out")
    if scale is None:
        scale = q.shape[-1] ** -0.5
    if k_lengths is None:
        k_lengths = lengths
    device = _lib.device_of((q, k, lengths, k_lengths, cu_seqlens, cu_seqlens_k, out, workspace), "q, k, lengths and out")

    def call(st):
        o = _new(q.shape[-2:-1], torch.float32, device, stream) if out is None else out
        a = _lib.qk_logits(q, k, o, scale, causal, lengths, k_lengths, cu_seqlens, cu_seqlens_k, accumulate)
        ws = _lib.scratch(_lib.mu_qk_max_logits_workspace_size(a), device, stream) if workspace is None else workspace
        _lib.mu_qk_max_logits(a, ws, st)
        return o
    return _on(device, stream, call)
