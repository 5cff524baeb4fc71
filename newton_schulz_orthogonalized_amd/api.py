"""Tensor-level calls over the C ABI: one Muon step, orthogonalise-only, AdamW,
QK-Clip, and what feeds them (gradient norm and clipping, the embedding and its
gradient, attention max logits, and the parts of a block between its products:
rotary positions, the norms around the block, the gated feed-forward product).

Each function marshals torch tensors into the library's descriptor lists,
allocates the workspace the library asks for (unless one is passed in) and
enqueues the work on `stream` (default: the current stream). Workspaces and
results allocated here come from `stream`'s share of the caching allocator, so
that neither the work that used their memory before nor the work that gets it
next overlaps the library's kernels; a result is recorded on the current stream
too. The caller orders `stream` behind what made the inputs, and its own use of
the results behind `stream`. Nothing here computes. Of the results those of
embedding, rotary, residual_norm, rms_norm and gated_mlp carry gradients (not in
forward mode, which they refuse, and once: a gradient of a gradient is refused).
Buffers of the caller's that rotary, the norms and the gated product write count
as changed in place: a backward pass that saved one of them raises.
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
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _lib.allocate(lambda: torch.empty(shape, dtype=dtype, device=torch.device("cuda", device)), device, stream,
                         returned=True)


def _no_tangents(what: str, *tensors):
    if forward_ad._current_level >= 0 and any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise NotImplementedError(f"{what} has no forward-mode derivative")


def _differentiable(what: str, tensors, *outs) -> bool:
    """Whether a call needs autograd; then it writes no buffers of the caller's."""
    _no_tangents(what, *tensors)
    if not (torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)):
        return False
    if any(o is not None for o in outs):
        raise ValueError("outputs of the caller's take no gradient: call under torch.no_grad()")
    return True


def _wrote(*outs):
    """Count the caller's buffers that a call wrote as changed in place, as torch's
    own operations do: a backward pass that saved one of them then refuses."""
    for o in outs:
        if o is not None:
            torch.autograd.graph.increment_version(o)


def _once(backward):
    """torch's once_differentiable, whose own work is a good part of a small
    call's, only where a graph of the gradient is asked for."""
    guarded = torch.autograd.function.once_differentiable(backward)

    def call(ctx, *grads):
        return guarded(ctx, *grads) if torch.is_grad_enabled() else backward(ctx, *grads)
    return call


def _dense(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    return None if t is None else t.contiguous()   # autograd hands in expanded or transposed gradients too


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
    _no_tangents("embedding", weight)
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


def rotary_frequencies(part: int, *, base: float = 10000.0, factor: float = 1.0, original_length: Optional[float] = None,
                       low: float = 1.0, high: float = 32.0, device=None) -> torch.Tensor:
    """The frequencies f_i = base ** (-2 i / part), i < part / 2, that rotary
    takes: radians a position, float64, on `device` (default: the current GPU).

    For contexts `factor` times as long as those a model was trained on: without
    original_length every frequency is divided by factor; with it, by parts. A
    frequency that makes r = original_length f / 2 pi turns over the original
    length is divided by factor where r <= low, kept where r >= high, and
    between them f (y + (1 - y) / factor) with y = (r - low) / (high - low)."""
    if part < 2 or part % 2:
        raise ValueError("part must be even and at least 2")
    if not base > 0 or not factor > 0 or math.isinf(base) or math.isinf(factor):
        raise ValueError("base and factor must be > 0 and finite")
    f = float(base) ** (-torch.arange(0, part, 2, dtype=torch.float64) / part)
    if original_length is None:
        f = f / factor
    else:
        if not original_length > 0 or not high > low:
            raise ValueError("original_length must be > 0 and high above low")
        y = ((original_length * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f * (y + (1 - y) / factor)
    return f.to("cuda" if device is None else device)


def rotary(q: torch.Tensor, k: Optional[torch.Tensor] = None, *, freqs: torch.Tensor,
           positions: Optional[torch.Tensor] = None, offset: int = 0, interleaved: bool = False, scale: float = 1.0,
           inverse: bool = False, out=None, stream=None):
    """Rotary positions: the first 2 * len(freqs) elements of every head of q
    (and k) turn by position * freqs, pair by pair, times scale; the rest of the
    head is copied. Returns the turned q, or (q, k).

    q [batch, length, heads, dim] and k [batch, length, k_heads, dim], or packed
    [rows, heads, dim], may be strided views (of a fused projection) with a
    contiguous last dimension. Pairs are (i, i + half) of that part, or (2 i,
    2 i + 1) with interleaved. positions (int32 or int64, [batch, length], [length]
    or [rows]) default to 0, 1, ..; offset is added to them. inverse turns back.
    freqs: float64 (rotary_frequencies). `out` (q's, or a pair) may be the inputs
    themselves. Differentiable in q and k unless `out` is given; freqs that ask for
    a gradient are refused."""
    xs = (q,) if k is None else (q, k)
    if out is not None:
        out = (out,) if isinstance(out, torch.Tensor) else tuple(out)
        if len(out) != len(xs):
            raise ValueError("out must have one tensor for each of q and k")
    _no_tangents("rotary", freqs)
    if freqs.requires_grad and torch.is_grad_enabled():
        raise NotImplementedError("rotary has no gradient of freqs")
    if _differentiable("rotary", xs, out):
        res = _Rotary.apply(q, k, freqs, positions, offset, interleaved, scale, inverse, stream)
    else:
        res = _rotary(xs, freqs, positions, offset, interleaved, scale, inverse, out, stream)[0]
    return res[0] if k is None else res


def _rotary(xs, freqs, positions, offset, interleaved, scale, inverse, out, stream):
    device = _lib.device_of((*xs, *(out or ()), freqs, positions), "q, k, freqs, positions and out")

    def call(st):
        outs = out if out is not None else tuple([_new(x.shape, x.dtype, device, stream) for x in xs])
        a = _lib.rotary_args(xs, outs, freqs, positions, offset, interleaved, inverse, scale)
        _lib.mu_rotary(a, st)
        _wrote(*(out or ()))
        return outs, a
    return _on(device, stream, call)


# The backward passes below run on a thread of autograd's, where every Python
# object that the forward call touched on its own thread costs a transfer between
# cores: they start from the structs that the forward calls filled and set
# addresses alone (the saved tensors', as they may have been moved meanwhile). A
# struct holds no tensor: what it points at, dense copies of gradients among it,
# keeps a name here until the launch has been made, or the workspace that is
# allocated before the launch may get its memory.
class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, freqs, positions, offset, interleaved, scale, inverse, stream):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(freqs, positions)
        outs, a = _rotary((q,) if k is None else (q, k), freqs, positions, offset, interleaved, scale, inverse, None, stream)
        a.inverse ^= 1
        ctx.args = a
        return outs

    @staticmethod
    @_once
    def backward(ctx, gq, gk=None):
        freqs, positions = ctx.saved_tensors
        a = _lib.MuRotaryArgs.from_buffer_copy(ctx.args)
        a.freqs = freqs.data_ptr()
        if positions is not None:
            a.positions = positions.data_ptr()
        dq = dk = None
        n = 0
        if gq is not None and ctx.needs_input_grad[0]:
            gq, dq = _lib.rotary_grad(a.x[0], gq)
            n = 1
        if gk is not None and ctx.needs_input_grad[1]:
            gk, dk = _lib.rotary_grad(a.x[1], gk)
            if n == 0:
                a.x[0] = a.x[1]
            n += 1
        if n:
            a.n = n
            _on(freqs.get_device(), None, _lib.rotary_call, a)
        return dq, dk, None, None, None, None, None, None, None


def residual_norm(residual: torch.Tensor, update: torch.Tensor, *, gate: Optional[torch.Tensor] = None,
                  post_norm: bool = False, post_weight: Optional[torch.Tensor] = None,
                  pre_weight: Optional[torch.Tensor] = None, residual_scale: float = 1.0, eps: float = 1e-6,
                  out: Optional[torch.Tensor] = None, normed_out: Optional[torch.Tensor] = None, stream=None):
    """What stands between two blocks, in one pass, with N(v; w) = v /
    sqrt(mean(v ** 2) + eps) * w over the last dimension:

        new_residual = residual_scale * residual + gate * N(update; post_weight)
        normed       = N(new_residual; pre_weight)          (the next block's input)

    Returns (new_residual, normed). The norm of the update is taken with
    post_norm=True or a post_weight; absent weights are 1. gate is [dim], or
    [groups, dim] whose rows apply to equal runs of the rows in turn (a gate for
    each sequence of a batch, or for each token). normed has the update's dtype;
    residual is of the same or float32 beside a bfloat16 update; weights and gate
    share either dtype. `out` may be the residual itself, normed_out the update.
    Differentiable in all tensors unless buffers are given."""
    if update is None:
        raise TypeError("update must be a tensor (rms_norm normalises without one)")
    post_norm = bool(post_norm) or post_weight is not None
    tensors = (residual, update, gate, post_weight, pre_weight)
    if _differentiable("residual_norm", tensors, out, normed_out):
        return _ResidualNorm.apply(*tensors, post_norm, residual_scale, eps, None, stream)
    return _residual_norm(*tensors, post_norm, residual_scale, eps, None, out, normed_out, stream)[:2]


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
             dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x / sqrt(mean(x ** 2) + eps) * weight over the last dimension: the norm
    before the first block. dtype is the result's (default: x's; bfloat16 beside a
    float32 x). Differentiable in x and weight unless `out` is given."""
    if out is not None and dtype is not None and out.dtype != dtype:
        raise TypeError("dtype differs from out's")
    dtype = out.dtype if out is not None else x.dtype if dtype is None else dtype
    if _differentiable("rms_norm", (x, weight), out):
        return _ResidualNorm.apply(x, None, None, None, weight, False, 1.0, eps, dtype, stream)
    return _residual_norm(x, None, None, None, weight, False, 1.0, eps, dtype, None, out, stream)[1]


def _residual_norm(residual, update, gate, post_weight, pre_weight, post_norm, residual_scale, eps, dtype, out, normed_out,
                   stream):
    device = _lib.device_of((residual, update, gate, post_weight, pre_weight, out, normed_out),
                            "residual, update, weights, gate and outputs")

    def call(st):
        r = out
        if r is None and update is not None:
            r = _new(residual.shape, residual.dtype, device, stream)
        n = normed_out
        if n is None:
            n = _new(residual.shape, dtype if update is None else update.dtype, device, stream)
        a = _lib.resnorm(residual, update, gate, post_weight, pre_weight, r, n, post_norm, residual_scale, eps)
        _lib.mu_residual_norm(a, st)
        _wrote(out, normed_out)
        return r, n, a
    return _on(device, stream, call)


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, residual, update, gate, post_weight, pre_weight, post_norm, residual_scale, eps, dtype, stream):
        ctx.set_materialize_grads(False)
        r, n, ctx.args = _residual_norm(residual, update, gate, post_weight, pre_weight, post_norm, residual_scale, eps, dtype,
                                        None, None, stream)
        ctx.save_for_backward(residual if update is None else r, update, gate, post_weight, pre_weight)
        return n if update is None else (r, n)

    @staticmethod
    @_once
    def backward(ctx, dr, dn=None):
        saved, need = ctx.saved_tensors, ctx.needs_input_grad
        if saved[1] is None:
            dr, dn = None, dr
        res = (None,) * 5
        if dr is not None or dn is not None:
            dr, dn = _dense(dr), _dense(dn)
            a, res = _lib.resnorm_backward(ctx.args, saved, need, dr, dn)
            _on(saved[0].get_device(), None, _lib.resnorm_grad_call, a, saved[0])
        return (*res, None, None, None, None, None)


def residual_norm_grad(grad_residual: Optional[torch.Tensor], grad_normed: Optional[torch.Tensor],
                       new_residual: torch.Tensor, update: Optional[torch.Tensor], *, gate: Optional[torch.Tensor] = None,
                       post_norm: bool = False, post_weight: Optional[torch.Tensor] = None,
                       pre_weight: Optional[torch.Tensor] = None, residual_scale: float = 1.0, eps: float = 1e-6,
                       workspace: Optional[torch.Tensor] = None, stream=None):
    """The gradients (residual, update, gate, post_weight, pre_weight) of
    residual_norm from those of its results (None: zero) and the new_residual it
    returned; None where there is no such tensor. Of rms_norm: update None and x
    in the place of new_residual. Sums over rows are float32 in a fixed order."""
    return _residual_norm_grad(grad_residual, grad_normed, new_residual, update, gate, post_weight, pre_weight,
                               bool(post_norm) or post_weight is not None, residual_scale, eps, (True,) * 5, workspace, stream)


def _residual_norm_grad(dr, dn, r, update, gate, post_weight, pre_weight, post_norm, residual_scale, eps, need, workspace,
                        stream):
    device = _lib.device_of((dr, dn, r, update, gate, post_weight, pre_weight, workspace), "gradients, inputs and weights")

    def call(st):
        res = tuple(_new(t.shape, t.dtype, device, stream) if t is not None and wanted else None
                    for t, wanted in zip((r, update, gate, post_weight, pre_weight), need))
        a = _lib.resnorm_grad(dr, dn, r, update, gate, post_weight, pre_weight, post_norm, residual_scale, eps, res)
        ws = _lib.scratch(_lib.mu_residual_norm_grad_workspace_size(a), device, stream) if workspace is None else workspace
        _lib.mu_residual_norm_grad(a, ws, st)
        return res
    return _on(device, stream, call)


def gated_mlp(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, *, activation: str = "silu",
              save_gates=torch.float32, out: Optional[torch.Tensor] = None, gates_out: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """act(x @ w_gate.T) * (x @ w_up.T), the input of a gated feed-forward
    block's last projection, in one kernel: x [..., dim], weights [hidden, dim],
    result [..., hidden], of one dtype. activation: "silu", "gelu", "gelu_tanh" or
    "relu". gates_out [2, ..., hidden], of x's dtype or float32, receives both
    products, which gated_mlp_grad reads. Differentiable in x and the weights unless
    buffers are given. save_gates is what is kept of the products for that: float32,
    as they are; True, rounded to x's dtype (half the memory beside a bfloat16 x, and
    less exact gradients); False, nothing, they are computed again."""
    keep = _kept_gates(save_gates, x)
    if _differentiable("gated_mlp", (x, w_gate, w_up), out, gates_out):
        return _GatedMlp.apply(x, w_gate, w_up, activation, keep, workspace, stream)
    return _gated_mlp(x, w_gate, w_up, activation, out, gates_out, workspace, stream)[0]


def _kept_gates(save_gates, x) -> Optional[torch.dtype]:
    if not isinstance(save_gates, torch.dtype):
        return x.dtype if save_gates else None
    if save_gates not in (x.dtype, torch.float32):
        raise TypeError("save_gates must be True, False, float32 or x's dtype")
    return save_gates


def _gated_mlp(x, w_gate, w_up, activation, out, gates_out, workspace, stream, keep=None):
    device = _lib.device_of((x, w_gate, w_up, out, gates_out, workspace), "x, weights and outputs")

    def call(st):
        shape = x.shape[:-1] + w_gate.shape[:1]
        h = _new(shape, x.dtype, device, stream) if out is None else out
        gates = gates_out if keep is None else _new((2, *shape), keep, device, stream)
        a = _lib.gated(x, w_gate, w_up, h, gates, activation)
        ws = _lib.scratch(_lib.mu_gated_mlp_workspace_size(a), device, stream) if workspace is None else workspace
        _lib.mu_gated_mlp(a, ws, st)
        _wrote(out, gates_out)
        return h, gates, a
    return _on(device, stream, call)


class _GatedMlp(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, activation, keep, workspace, stream):
        h, gates, a = _gated_mlp(x, w_gate, w_up, activation, None, None, workspace, stream, keep)
        ctx.args = _lib.MuGatedGrad(tokens=a.tokens, dim=a.dim, hidden=a.hidden, dtype=a.dtype, grad_dtype=a.dtype,
                                    activation=a.activation)
        ctx.save_for_backward(x, w_gate, w_up, gates)
        return h

    @staticmethod
    @_once
    def backward(ctx, grad):
        saved, grad = ctx.saved_tensors, _dense(grad)
        a, res = _lib.gated_backward(ctx.args, saved, ctx.needs_input_grad, grad)
        _on(saved[0].get_device(), None, _lib.gated_grad_call, a, saved[0])
        return (*res[:3], None, None, None, None)


def gated_mlp_grad(grad: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                   gates: Optional[torch.Tensor] = None, *, activation: str = "silu", need_x: bool = True,
                   need_weights: bool = True, d_gate: Optional[torch.Tensor] = None, d_up: Optional[torch.Tensor] = None,
                   dtype: Optional[torch.dtype] = None, accumulate: bool = False,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """The gradients (dx, d_gate, d_up) of gated_mlp from its result's. gates is
    the forward call's gates_out, of x's dtype or float32 (None: both products are
    computed again). d_gate
    and d_up receive the weights' gradients, of x's dtype or float32
    (accumulate=True: added to them, over the micro-batches of a step); dtype is
    that of new ones (default: x's). The same call gives the same bits."""
    if (d_gate is None) != (d_up is None):
        raise ValueError("d_gate and d_up go together")
    if d_gate is not None and not need_weights:
        raise ValueError("d_gate and d_up without need_weights")
    if accumulate and d_gate is None:
        raise ValueError("accumulate=True needs d_gate and d_up")
    if d_gate is not None and dtype is not None and d_gate.dtype != dtype:
        raise TypeError("dtype differs from d_gate's")
    device = _lib.device_of((grad, x, w_gate, w_up, gates, d_gate, d_up, workspace), "grad, x, weights and results")

    def call(st):
        dx = _new(x.shape, x.dtype, device, stream) if need_x else None
        dg, du = d_gate, d_up
        if dg is None and need_weights:
            dg, du = (_new(w_gate.shape, x.dtype if dtype is None else dtype, device, stream) for _ in range(2))
        a = _lib.gated_grad(grad, x, w_gate, w_up, gates, dx, dg, du, accumulate, activation)
        ws = _lib.scratch(_lib.mu_gated_mlp_grad_workspace_size(a), device, stream) if workspace is None else workspace
        _lib.mu_gated_mlp_grad(a, ws, st)
        _wrote(d_gate, d_up)
        return dx, dg, du
    return _on(device, stream, call)
