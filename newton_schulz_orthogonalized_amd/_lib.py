"""ctypes binding of libmuon_mi355x.so: argument marshalling only.

Every entry point of ``include/muon_mi355x.h`` has a function of the same name
here that takes torch tensors, fills the C structs with their device pointers
and calls the library on the current HIP stream. All arithmetic runs in the
library's kernels; there is no fallback path, and importing this module fails
loudly when the shared library is missing.
"""

from __future__ import annotations

import ctypes
import operator
import os
import struct
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmuon_mi355x.so")

MU_F32 = 0
MU_BF16 = 1
MU_NS_F32 = 0
MU_NS_BF16 = 1

MU_OK = 0
MU_ERR_INVALID_ARG = 1
MU_ERR_DTYPE = 2
MU_ERR_LAYOUT = 3
MU_ERR_WORKSPACE = 4
MU_ERR_HIP = 5

(MU_K_PREP, MU_K_NORM, MU_K_GRAM, MU_K_GRAM2, MU_K_APPLY, MU_K_FINISH, MU_K_ADAMW, MU_K_QKCLIP, MU_K_FUSED,
 MU_K_RESCALE, MU_K_TILEMAP, MU_K_GRADNORM, MU_K_CLIP, MU_K_LOOKUP, MU_K_ROWGRAD, MU_K_QKMAX, MU_K_ROTARY,
 MU_K_RESNORM, MU_K_RESNORM_GRAD, MU_K_GATED, MU_K_GATED_GRAD) = range(21)
MU_K_COUNT = 21

EXPORTED = (
    "mu_muon_workspace_size", "mu_muon_step", "mu_muon_step_noalloc", "mu_ortho_workspace_size",
    "mu_muon_orthogonalize",
    "mu_adamw_workspace_size", "mu_adamw_step", "mu_qk_clip_workspace_size", "mu_qk_clip",
    "mu_muon_step_scaled", "mu_adamw_step_scaled", "mu_grad_norm_workspace_size", "mu_grad_norm", "mu_clip_grads",
    "mu_embedding", "mu_embedding_grad_workspace_size", "mu_embedding_grad", "mu_qk_max_logits_workspace_size",
    "mu_qk_max_logits", "mu_rotary", "mu_residual_norm", "mu_residual_norm_grad_workspace_size", "mu_residual_norm_grad",
    "mu_gated_mlp_workspace_size", "mu_gated_mlp", "mu_gated_mlp_grad_workspace_size", "mu_gated_mlp_grad",
    "mu_status_string", "mu_last_error", "mu_version", "mu_profile_enable", "mu_profile_read", "mu_kernel_name",
)


class MuMatrix(ctypes.Structure):
    _fields_ = [
        ("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("momentum", ctypes.c_void_p),
        ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("dtype", ctypes.c_int32),
        ("num_heads", ctypes.c_int32), ("scale", ctypes.c_float), ("norm_out", ctypes.c_void_p),
        ("ortho_out", ctypes.c_void_p),
    ]


class MuMuonHparams(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_float), ("weight_decay", ctypes.c_float), ("mu", ctypes.c_float),
        ("nesterov", ctypes.c_int32), ("norm_eps", ctypes.c_float), ("ns_steps", ctypes.c_int32),
        ("coeffs", ctypes.POINTER(ctypes.c_float)), ("ns_precision", ctypes.c_int32),
        ("cautious_wd", ctypes.c_int32),
    ]


class MuOrtho(ctypes.Structure):
    _fields_ = [
        ("input", ctypes.c_void_p), ("output", ctypes.c_void_p), ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64), ("dtype", ctypes.c_int32), ("num_heads", ctypes.c_int32),
        ("norm_out", ctypes.c_void_p),
    ]


class MuTensor(ctypes.Structure):
    _fields_ = [
        ("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
        ("exp_avg_sq", ctypes.c_void_p), ("numel", ctypes.c_int64), ("dtype", ctypes.c_int32),
        ("lr", ctypes.c_float), ("weight_decay", ctypes.c_float),
    ]


class MuAdamwHparams(ctypes.Structure):
    _fields_ = [("beta1", ctypes.c_float), ("beta2", ctypes.c_float), ("eps", ctypes.c_float),
                ("step", ctypes.c_int64)]


class MuQkPair(ctypes.Structure):
    _fields_ = [
        ("wq", ctypes.c_void_p), ("wk", ctypes.c_void_p), ("q_rows", ctypes.c_int64), ("k_rows", ctypes.c_int64),
        ("cols", ctypes.c_int64), ("q_heads", ctypes.c_int32), ("k_heads", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("pad0", ctypes.c_int32), ("max_logit", ctypes.c_void_p),
        ("gamma_out", ctypes.c_void_p),
    ]


class MuGrad(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


class MuLookup(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("n_tokens", ctypes.c_int64), ("vocab", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("token_bits", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("pad0", ctypes.c_int32)]


class MuRowgrad(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_void_p), ("rows", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("n_tokens", ctypes.c_int64), ("vocab", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("padding_idx", ctypes.c_int64), ("token_bits", ctypes.c_int32), ("row_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("accumulate", ctypes.c_int32), ("scale", ctypes.c_float),
                ("pad0", ctypes.c_int32)]


class MuQkLogits(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("q_stride_b", ctypes.c_int64), ("q_stride_s", ctypes.c_int64), ("q_stride_h", ctypes.c_int64),
                ("k_stride_b", ctypes.c_int64), ("k_stride_s", ctypes.c_int64), ("k_stride_h", ctypes.c_int64),
                ("q_len", ctypes.c_int64), ("k_len", ctypes.c_int64), ("batch", ctypes.c_int32),
                ("q_heads", ctypes.c_int32), ("k_heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("q_lengths", ctypes.c_void_p), ("k_lengths", ctypes.c_void_p), ("cu_q", ctypes.c_void_p),
                ("cu_k", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("causal", ctypes.c_int32),
                ("accumulate", ctypes.c_int32), ("scale", ctypes.c_float), ("max_logit", ctypes.c_void_p)]


class MuRotaryTensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("x_stride_b", ctypes.c_int64), ("x_stride_s", ctypes.c_int64), ("x_stride_h", ctypes.c_int64),
                ("out_stride_b", ctypes.c_int64), ("out_stride_s", ctypes.c_int64), ("out_stride_h", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("pad0", ctypes.c_int32)]


class MuRotaryArgs(ctypes.Structure):
    _fields_ = [("x", MuRotaryTensor * 2), ("freqs", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("offset", ctypes.c_int64), ("batch", ctypes.c_int64), ("len", ctypes.c_int64), ("n", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("part", ctypes.c_int32), ("position_bits", ctypes.c_int32),
                ("shared_positions", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("inverse", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("pad0", ctypes.c_int32)]


class MuResnorm(ctypes.Structure):
    _fields_ = [("residual", ctypes.c_void_p), ("update", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("post_weight", ctypes.c_void_p), ("pre_weight", ctypes.c_void_p), ("new_residual", ctypes.c_void_p),
                ("normed", ctypes.c_void_p), ("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("groups", ctypes.c_int64),
                ("residual_dtype", ctypes.c_int32), ("dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32),
                ("post_norm", ctypes.c_int32), ("residual_scale", ctypes.c_float), ("eps", ctypes.c_float)]


class MuResnormGrad(ctypes.Structure):
    _fields_ = [("fwd", MuResnorm), ("grad_residual", ctypes.c_void_p), ("grad_normed", ctypes.c_void_p),
                ("d_residual", ctypes.c_void_p), ("d_update", ctypes.c_void_p), ("d_gate", ctypes.c_void_p),
                ("d_post", ctypes.c_void_p), ("d_pre", ctypes.c_void_p)]


class MuGated(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("h", ctypes.c_void_p),
                ("gate_out", ctypes.c_void_p), ("up_out", ctypes.c_void_p), ("tokens", ctypes.c_int64),
                ("dim", ctypes.c_int64), ("hidden", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("activation", ctypes.c_int32)]


class MuGatedGrad(ctypes.Structure):
    _fields_ = [("grad_h", ctypes.c_void_p), ("x", ctypes.c_void_p), ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("up", ctypes.c_void_p), ("dx", ctypes.c_void_p), ("d_gate", ctypes.c_void_p),
                ("d_up", ctypes.c_void_p), ("tokens", ctypes.c_int64), ("dim", ctypes.c_int64), ("hidden", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32), ("accumulate", ctypes.c_int32),
                ("activation", ctypes.c_int32)]


class MuonError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{_status_text(status)} (status {status}): {detail}")
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m newton_schulz_orthogonalized_amd.build` "
            "(there is no fallback path)")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER
    sz = ctypes.c_size_t
    lib.mu_muon_workspace_size.argtypes = [P(MuMatrix), ctypes.c_int32, P(MuMuonHparams), P(sz)]
    lib.mu_muon_step.argtypes = [P(MuMatrix), ctypes.c_int32, P(MuMuonHparams), ctypes.c_void_p, sz, ctypes.c_void_p]
    lib.mu_muon_step_noalloc.argtypes = [P(MuMatrix), ctypes.c_int32, P(MuMuonHparams), ctypes.c_void_p]
    lib.mu_ortho_workspace_size.argtypes = [P(MuOrtho), ctypes.c_int32, P(MuMuonHparams), P(sz)]
    lib.mu_muon_orthogonalize.argtypes = [P(MuOrtho), ctypes.c_int32, P(MuMuonHparams), ctypes.c_void_p, sz,
                                          ctypes.c_void_p]
    lib.mu_adamw_workspace_size.argtypes = [ctypes.c_int32, P(sz)]
    lib.mu_adamw_step.argtypes = [P(MuTensor), ctypes.c_int32, P(MuAdamwHparams), ctypes.c_void_p, sz,
                                  ctypes.c_void_p]
    lib.mu_qk_clip_workspace_size.argtypes = [P(MuQkPair), ctypes.c_int32, P(sz)]
    lib.mu_qk_clip.argtypes = [P(MuQkPair), ctypes.c_int32, ctypes.c_float, ctypes.c_void_p, sz, ctypes.c_void_p]
    vp = ctypes.c_void_p
    lib.mu_muon_step_scaled.argtypes = [P(MuMatrix), ctypes.c_int32, P(MuMuonHparams), vp, vp, sz, vp]
    lib.mu_adamw_step_scaled.argtypes = [P(MuTensor), ctypes.c_int32, P(MuAdamwHparams), vp, vp, sz, vp]
    lib.mu_grad_norm_workspace_size.argtypes = [vp, ctypes.c_int32, P(sz)]   # mu_grad lists are packed bytes (gradients())
    for name in ("mu_grad_norm", "mu_clip_grads"):
        getattr(lib, name).argtypes = [vp, ctypes.c_int32, ctypes.c_float, ctypes.c_float, vp, vp, vp, sz, vp]
    lib.mu_embedding.argtypes = [P(MuLookup), vp]
    lib.mu_embedding_grad_workspace_size.argtypes = [P(MuRowgrad), P(sz)]
    lib.mu_embedding_grad.argtypes = [P(MuRowgrad), vp, sz, vp]
    lib.mu_qk_max_logits_workspace_size.argtypes = [P(MuQkLogits), P(sz)]
    lib.mu_qk_max_logits.argtypes = [P(MuQkLogits), vp, sz, vp]
    lib.mu_rotary.argtypes = [P(MuRotaryArgs), vp]
    lib.mu_residual_norm.argtypes = [P(MuResnorm), vp]
    for name, args in (("mu_residual_norm_grad", MuResnormGrad), ("mu_gated_mlp", MuGated), ("mu_gated_mlp_grad", MuGatedGrad)):
        getattr(lib, name + "_workspace_size").argtypes = [P(args), P(sz)]
        getattr(lib, name).argtypes = [P(args), vp, sz, vp]
    lib.mu_status_string.argtypes = [ctypes.c_int]
    lib.mu_status_string.restype = ctypes.c_char_p
    lib.mu_last_error.argtypes = []
    lib.mu_last_error.restype = ctypes.c_char_p
    lib.mu_version.restype = ctypes.c_int
    lib.mu_profile_enable.argtypes = [ctypes.c_int]
    lib.mu_profile_read.argtypes = [ctypes.c_int, P(ctypes.c_double), P(ctypes.c_int64), P(ctypes.c_double),
                                    P(ctypes.c_double)]
    lib.mu_kernel_name.argtypes = [ctypes.c_int]
    lib.mu_kernel_name.restype = ctypes.c_char_p
    for name in ("mu_muon_workspace_size", "mu_muon_step", "mu_muon_step_noalloc", "mu_ortho_workspace_size",
                 "mu_muon_orthogonalize",
                 "mu_adamw_workspace_size", "mu_adamw_step", "mu_profile_enable", "mu_profile_read",
                 "mu_muon_step_scaled", "mu_adamw_step_scaled", "mu_grad_norm_workspace_size", "mu_grad_norm",
                 "mu_clip_grads", "mu_embedding", "mu_embedding_grad_workspace_size", "mu_embedding_grad",
                 "mu_qk_max_logits_workspace_size", "mu_qk_max_logits", "mu_rotary", "mu_residual_norm",
                 "mu_residual_norm_grad_workspace_size", "mu_residual_norm_grad", "mu_gated_mlp_workspace_size",
                 "mu_gated_mlp", "mu_gated_mlp_grad_workspace_size", "mu_gated_mlp_grad"):
        getattr(lib, name).restype = ctypes.c_int
    return lib


LIB = _load()


def _status_text(status: int) -> str:
    return LIB.mu_status_string(status).decode()


def _check(status: int) -> None:
    if status != MU_OK:
        raise MuonError(status, LIB.mu_last_error().decode())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MU_BF16
    if t.dtype == torch.float32:
        return MU_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _require(t: torch.Tensor, what: str) -> None:
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous (the library takes dense row-major buffers)")


def muon_hparams(lr: float, weight_decay: float, mu: float = 0.95, nesterov: bool = True, norm_eps: float = 1e-7,
                 ns_steps: int = 5, coeffs: Optional[Sequence[Sequence[float]]] = None,
                 precision: str = "bf16", cautious_wd: bool = False):
    """Build mu_muon_hparams. Returns (struct, keepalive) - keep both alive for the call."""
    buf = None
    if coeffs is not None:
        flat = []
        for c in coeffs:
            c = list(c)
            if len(c) == 2:
                c.append(0.0)
            flat.extend(float(v) for v in c)
        if len(flat) != 3 * ns_steps:
            raise ValueError("coeffs must give (a, b[, c]) for each of ns_steps steps")
        buf = (ctypes.c_float * len(flat))(*flat)
    hp = MuMuonHparams(lr, weight_decay, mu, 1 if nesterov else 0, norm_eps, ns_steps,
                       ctypes.cast(buf, ctypes.POINTER(ctypes.c_float)) if buf is not None else None,
                       MU_NS_BF16 if precision == "bf16" else MU_NS_F32, 1 if cautious_wd else 0)
    return hp, buf


def matrices(params, grads, moms, heads=None, scales=None, norm_outs=None, ortho_outs=None):
    """Array of mu_matrix for lists of 2-D tensors."""
    n = len(params)
    arr = (MuMatrix * max(n, 1))()
    for i in range(n):
        p, g, m = params[i], grads[i], moms[i]
        for t, what in ((p, "param"), (g, "grad"), (m, "momentum")):
            _require(t, what)
        if p.dim() != 2 or g.shape != p.shape or m.shape != p.shape:
            raise ValueError("param, grad and momentum must be 2-D and of one shape")
        if m.dtype != torch.float32 or g.dtype != p.dtype:
            raise TypeError("momentum must be float32 and grad must share the param dtype")
        no = None if norm_outs is None else norm_outs[i]
        oo = None if ortho_outs is None else ortho_outs[i]
        if oo is not None and (oo.dtype != torch.float32 or oo.shape != p.shape or not oo.is_contiguous()):
            raise ValueError("ortho_out must be a contiguous float32 tensor of the param's shape")
        arr[i] = MuMatrix(_ptr(p), _ptr(g), _ptr(m), p.shape[0], p.shape[1], _dtype_code(p),
                          1 if heads is None else int(heads[i]), 1.0 if scales is None else float(scales[i]),
                          _ptr(no), _ptr(oo))
    return arr, n


def mu_muon_workspace_size(mats, n, hp) -> int:
    out = ctypes.c_size_t(0)
    _check(LIB.mu_muon_workspace_size(mats, n, ctypes.byref(hp), ctypes.byref(out)))
    return out.value


def mu_muon_step(mats, n, hp, workspace: Optional[torch.Tensor], stream=None) -> None:
    ws = 0 if workspace is None else workspace.data_ptr()
    nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(LIB.mu_muon_step(mats, n, ctypes.byref(hp), ws, nb, _stream(stream)))


def grad_scale_ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    """Address of a clip factor: one float32 on the GPU (None: the plain step)."""
    if t is None:
        return None
    if t.dtype != torch.float32 or t.numel() != 1:
        raise TypeError("grad_scale must be one float32 element")
    if not t.is_cuda:
        raise ValueError("grad_scale must be a GPU tensor (it is read when the kernels run)")
    return t.data_ptr()


def mu_muon_step_scaled(mats, n, hp, grad_scale: Optional[torch.Tensor], workspace: Optional[torch.Tensor],
                        stream=None) -> None:
    ws = 0 if workspace is None else workspace.data_ptr()
    nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(LIB.mu_muon_step_scaled(mats, n, ctypes.byref(hp), grad_scale_ptr(grad_scale), ws, nb, _stream(stream)))


MU_NOALLOC_SCRATCH_BYTES = 64 << 20


def mu_muon_step_noalloc(mats, n, hp, stream=None) -> None:
    """mu_muon_step with the library's static per-GPU scratch as workspace."""
    _check(LIB.mu_muon_step_noalloc(mats, n, ctypes.byref(hp), _stream(stream)))


def orthos(inputs, outputs, heads=None, norm_outs=None):
    n = len(inputs)
    arr = (MuOrtho * max(n, 1))()
    for i in range(n):
        x, o = inputs[i], outputs[i]
        _require(x, "input")
        _require(o, "output")
        if x.dim() != 2 or o.shape != x.shape or o.dtype != x.dtype:
            raise ValueError("input and output must be 2-D, of one shape and dtype")
        no = None if norm_outs is None else norm_outs[i]
        arr[i] = MuOrtho(_ptr(x), _ptr(o), x.shape[0], x.shape[1], _dtype_code(x),
                         1 if heads is None else int(heads[i]), _ptr(no))
    return arr, n


def mu_ortho_workspace_size(xs, n, hp) -> int:
    out = ctypes.c_size_t(0)
    _check(LIB.mu_ortho_workspace_size(xs, n, ctypes.byref(hp), ctypes.byref(out)))
    return out.value


def mu_muon_orthogonalize(xs, n, hp, workspace: Optional[torch.Tensor], stream=None) -> None:
    ws = 0 if workspace is None else workspace.data_ptr()
    nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(LIB.mu_muon_orthogonalize(xs, n, ctypes.byref(hp), ws, nb, _stream(stream)))


def tensors(params, grads, exp_avgs, exp_avg_sqs, lrs, wds):
    n = len(params)
    arr = (MuTensor * max(n, 1))()
    for i in range(n):
        p, g, m, v = params[i], grads[i], exp_avgs[i], exp_avg_sqs[i]
        for t, what in ((p, "param"), (g, "grad"), (m, "exp_avg"), (v, "exp_avg_sq")):
            _require(t, what)
        if g.shape != p.shape or m.shape != p.shape or v.shape != p.shape:
            raise ValueError("param, grad and states must share a shape")
        if m.dtype != torch.float32 or v.dtype != torch.float32 or g.dtype != p.dtype:
            raise TypeError("states must be float32 and grad must share the param dtype")
        arr[i] = MuTensor(_ptr(p), _ptr(g), _ptr(m), _ptr(v), p.numel(), _dtype_code(p), float(lrs[i]),
                          float(wds[i]))
    return arr, n


def mu_adamw_workspace_size(n: int) -> int:
    out = ctypes.c_size_t(0)
    _check(LIB.mu_adamw_workspace_size(n, ctypes.byref(out)))
    return out.value


def mu_adamw_step(ts, n, beta1: float, beta2: float, eps: float, step: int,
                  workspace: Optional[torch.Tensor], stream=None) -> None:
    hp = MuAdamwHparams(beta1, beta2, eps, step)
    ws = 0 if workspace is None else workspace.data_ptr()
    nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(LIB.mu_adamw_step(ts, n, ctypes.byref(hp), ws, nb, _stream(stream)))


def mu_adamw_step_scaled(ts, n, beta1: float, beta2: float, eps: float, step: int,
                         grad_scale: Optional[torch.Tensor], workspace: Optional[torch.Tensor], stream=None) -> None:
    hp = MuAdamwHparams(beta1, beta2, eps, step)
    ws = 0 if workspace is None else workspace.data_ptr()
    nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(LIB.mu_adamw_step_scaled(ts, n, ctypes.byref(hp), grad_scale_ptr(grad_scale), ws, nb, _stream(stream)))


def device_of(tensors, what: str) -> int:
    """The index of the one GPU that all of `tensors` (None entries aside) live
    on; the current one where there is none."""
    devs = set(map(_Tensor.get_device, [t for t in tensors if t is not None]))
    if not devs:
        return torch.cuda.current_device()
    if min(devs) < 0:
        raise ValueError(f"{what} must be on a GPU")
    if len(devs) > 1:
        raise ValueError(f"{what} must share one device (got GPUs {sorted(devs)})")
    return devs.pop()


def scratch(nbytes: int, device: int, stream=None) -> Optional[torch.Tensor]:
    """workspace() without the slice where the allocator's address will do."""
    if nbytes == 0:
        return None
    buf = allocate(lambda: torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", device)), device, stream)
    return buf if buf.data_ptr() % 256 == 0 else workspace(nbytes, buf.device, stream)


_CODES = {torch.float32: MU_F32, torch.bfloat16: MU_BF16}
_Tensor = torch._C.TensorBase
_SHAPE = operator.attrgetter("shape")
_DTYPE = operator.attrgetter("dtype")


def _list_of(tensors, what: str):
    """Addresses, sizes and type codes of a list, in a few passes of C speed (a
    list may hold hundreds of tensors)."""
    try:
        codes = list(map(_CODES.__getitem__, map(_DTYPE, tensors)))
    except KeyError as e:
        raise TypeError(f"unsupported dtype {e.args[0]}") from None
    if not all(map(_Tensor.is_contiguous, tensors)):
        raise ValueError(f"{what} must be contiguous (the library takes dense row-major buffers)")
    return list(map(_Tensor.data_ptr, tensors)), list(map(_Tensor.numel, tensors)), codes


def gradients(grads, outs=None):
    """(mu_grad list as packed bytes, n)."""
    n = len(grads)
    ptrs, sizes, codes = _list_of(grads, "gradient")
    if outs is None:
        optrs, ocodes = [0] * n, codes
    else:
        if len(outs) != n:
            raise ValueError("outs must have one tensor for each gradient")
        optrs, _, ocodes = _list_of(outs, "output")
        if outs is not grads and list(map(_SHAPE, outs)) != list(map(_SHAPE, grads)):
            raise ValueError("each output must have its gradient's shape")
    flat = [0] * (5 * n)
    flat[0::5], flat[1::5], flat[2::5], flat[3::5], flat[4::5] = ptrs, optrs, sizes, codes, ocodes
    return struct.pack("=" + "QQqii" * n, *flat), n


def mu_grad_norm_workspace_size(gs, n) -> int:
    out = ctypes.c_size_t(0)
    _check(LIB.mu_grad_norm_workspace_size(gs, n, ctypes.byref(out)))
    return out.value


def mu_grad_norm(gs, n, max_norm: float, eps: float, norm_out, scale_out, workspace, stream=None) -> None:
    ws = 0 if workspace is None else workspace.data_ptr()
    nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(LIB.mu_grad_norm(gs, n, max_norm, eps, _ptr(norm_out), _ptr(scale_out), ws, nb, _stream(stream)))


def mu_clip_grads(gs, n, max_norm: float, eps: float, norm_out, scale_out, workspace, stream=None) -> None:
    ws = 0 if workspace is None else workspace.data_ptr()
    nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(LIB.mu_clip_grads(gs, n, max_norm, eps, _ptr(norm_out), _ptr(scale_out), ws, nb, _stream(stream)))


def _token_bits(t: torch.Tensor, what: str = "tokens") -> int:
    if t.dtype == torch.int64:
        return 64
    if t.dtype == torch.int32:
        return 32
    raise TypeError(f"{what} must be int32 or int64 (got {t.dtype})")


def lookup(tokens, weight, out, scale: float) -> MuLookup:
    for t, what in ((tokens, "tokens"), (weight, "weight"), (out, "out")):
        _require(t, what)
    if weight.dim() != 2:
        raise ValueError("weight must be 2-D")
    if out.shape != tokens.shape + weight.shape[1:]:
        raise ValueError("out must have the tokens' shape and the weight's row length")
    if out.dtype != weight.dtype:
        raise TypeError("out must share the weight's dtype")
    return MuLookup(_ptr(tokens), _ptr(weight), _ptr(out), tokens.numel(), weight.shape[0], weight.shape[1],
                    _token_bits(tokens), _dtype_code(weight), float(scale), 0)


def mu_embedding(e: MuLookup, stream=None) -> None:
    _check(LIB.mu_embedding(ctypes.byref(e), _stream(stream)))


def rowgrad(tokens, rows, grad, scale: float, padding_idx: Optional[int], accumulate: bool) -> MuRowgrad:
    for t, what in ((tokens, "tokens"), (rows, "rows"), (grad, "grad")):
        _require(t, what)
    if grad.dim() != 2:
        raise ValueError("grad must be 2-D")
    if rows.shape != tokens.shape + grad.shape[1:]:
        raise ValueError("rows must have the tokens' shape and the gradient's row length")
    if padding_idx is not None and not 0 <= padding_idx < grad.shape[0]:
        raise ValueError("padding_idx must name a row of the gradient")
    return MuRowgrad(_ptr(tokens), _ptr(rows), _ptr(grad), tokens.numel(), grad.shape[0], grad.shape[1],
                     -1 if padding_idx is None else int(padding_idx), _token_bits(tokens), _dtype_code(rows),
                     _dtype_code(grad), 1 if accumulate else 0, float(scale), 0)


def mu_embedding_grad_workspace_size(e: MuRowgrad) -> int:
    out = ctypes.c_size_t(0)
    _check(LIB.mu_embedding_grad_workspace_size(ctypes.byref(e), ctypes.byref(out)))
    return out.value


def mu_embedding_grad(e: MuRowgrad, workspace: Optional[torch.Tensor], stream=None) -> None:
    ws = 0 if workspace is None else workspace.data_ptr()
    nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(LIB.mu_embedding_grad(ctypes.byref(e), ws, nb, _stream(stream)))


def qk_logits(q, k, out, scale: float, causal: bool, lengths, k_lengths, cu_seqlens, cu_seqlens_k,
              accumulate: bool) -> MuQkLogits:
    packed = cu_seqlens is not None
    q_shape, k_shape, q_stride, k_stride = q.shape, k.shape, q.stride(), k.stride()
    nd = 3 if packed else 4
    if len(q_shape) != nd or len(k_shape) != nd:
        raise ValueError("q and k must be [batch, length, heads, dim], or [rows, heads, dim] with cu_seqlens")
    if k.dtype != q.dtype:
        raise TypeError("k must share q's dtype")
    dim = q_shape[-1]
    if dim != k_shape[-1] or (not packed and q_shape[0] != k_shape[0]):
        raise ValueError("q and k must agree in dim and batch")
    if dim > 1 and (q_stride[-1] != 1 or k_stride[-1] != 1):
        raise ValueError("the last dimension of q and k must be contiguous")
    if out.dtype != torch.float32 or out.shape != q_shape[-2:-1]:
        raise ValueError("out must be float32 with one element for each query head")
    _require(out, "out")
    if packed:
        if lengths is not None or k_lengths is not None:
            raise ValueError("packed sequences (cu_seqlens) take no lengths")
        batch = cu_seqlens.numel() - 1
        if batch < 0:
            raise ValueError("cu_seqlens must have at least one element")
        q_stride, k_stride = (0, *q_stride), (0, *k_stride)
    else:
        if cu_seqlens_k is not None:
            raise ValueError("cu_seqlens_k needs cu_seqlens")
        batch = q_shape[0]
    for t, what, size in ((lengths, "lengths", batch), (k_lengths, "k_lengths", batch),
                          (cu_seqlens, "cu_seqlens", batch + 1), (cu_seqlens_k, "cu_seqlens_k", batch + 1)):
        if t is None:
            continue
        if t.dtype != torch.int32:
            raise TypeError(f"{what} must be int32")
        if t.dim() != 1 or t.numel() != size:
            raise ValueError(f"{what} must have {size} elements")
        _require(t, what)
    return MuQkLogits(q.data_ptr(), k.data_ptr(), *q_stride[:3], *k_stride[:3], q_shape[-3], k_shape[-3], batch,
                      q_shape[-2], k_shape[-2], dim, _ptr(lengths), _ptr(k_lengths), _ptr(cu_seqlens),
                      _ptr(cu_seqlens_k), _dtype_code(q), 1 if causal else 0, 1 if accumulate else 0, float(scale),
                      out.data_ptr())


def mu_qk_max_logits_workspace_size(a: MuQkLogits) -> int:
    out = ctypes.c_size_t(0)
    _check(LIB.mu_qk_max_logits_workspace_size(ctypes.byref(a), ctypes.byref(out)))
    return out.value


def mu_qk_max_logits(a: MuQkLogits, workspace: Optional[torch.Tensor], stream=None) -> None:
    ws = 0 if workspace is None else workspace.data_ptr()
    nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(LIB.mu_qk_max_logits(ctypes.byref(a), ws, nb, _stream(stream)))


def rotary_args(xs, outs, freqs, positions, offset: int, interleaved: bool, inverse: bool, scale: float) -> MuRotaryArgs:
    first = xs[0]
    a = MuRotaryArgs()
    shape = first.shape
    packed = len(shape) == 3   # [rows, heads, dim]: one sequence
    if len(shape) not in (3, 4):
        raise ValueError("q and k must be [batch, length, heads, dim] or [rows, heads, dim]")
    for i, (x, o) in enumerate(zip(xs, outs)):
        if x.dtype != first.dtype or o.dtype != first.dtype:
            raise TypeError("q, k and their outputs must share a dtype")
        if x.shape[:-2] != shape[:-2] or x.shape[-1] != shape[-1]:
            raise ValueError("q and k must agree in batch, length and dim")
        if o.shape != x.shape:
            raise ValueError("an output must have its input's shape")
        sx, so = x.stride(), o.stride()
        if shape[-1] > 1 and (sx[-1] != 1 or so[-1] != 1):
            raise ValueError("the last dimension of q, k and their outputs must be contiguous")
        if packed:
            sx, so = (0, *sx), (0, *so)
        a.x[i] = MuRotaryTensor(x.data_ptr(), o.data_ptr(), *sx[:3], *so[:3], x.shape[-2], 0)
    if freqs.dtype != torch.float64 or freqs.dim() != 1:
        raise TypeError("freqs must be a float64 vector (rotary_frequencies)")
    _require(freqs, "freqs")
    if not -1 << 52 <= offset <= 1 << 52:   # (the field would take its low 64 bits)
        raise ValueError("offset is too large")
    a.batch, a.len = (1, shape[0]) if packed else shape[:2]
    if positions is not None:
        rows = shape[:-2]
        if positions.shape != rows and positions.shape != rows[-1:]:
            raise ValueError(f"positions must be {list(rows)} or {list(rows[-1:])}")
        a.position_bits = _token_bits(positions, "positions")
        a.shared_positions = 1 if positions.shape != rows else 0
        _require(positions, "positions")
        a.positions = positions.data_ptr()
    a.freqs, a.offset, a.n, a.dim, a.part = freqs.data_ptr(), int(offset), len(xs), shape[-1], 2 * freqs.numel()
    a.interleaved, a.inverse, a.dtype, a.scale = 1 if interleaved else 0, 1 if inverse else 0, _dtype_code(first), float(scale)
    return a


def mu_rotary(a: MuRotaryArgs, stream=None) -> None:
    _check(LIB.mu_rotary(ctypes.byref(a), _stream(stream)))


def rotary_call(stream, a: MuRotaryArgs) -> None:
    status = LIB.mu_rotary(ctypes.byref(a), stream)
    if status:
        _check(status)


def rotary_grad(t: MuRotaryTensor, g):
    """Point one tensor of a backward call at its result's gradient and at a new
    tensor for its own: (the gradient as it is read, the new tensor). Both have the
    layout of the forward call's result, which t's out_stride_* are, if the
    gradient is dense."""
    if not g.is_contiguous():
        if g.shape[-1] > 1 and g.stride(-1) != 1:
            g = g.contiguous()
    d = torch.empty_like(g, memory_format=torch.contiguous_format)
    if g.is_contiguous():
        t.x_stride_b, t.x_stride_s, t.x_stride_h = t.out_stride_b, t.out_stride_s, t.out_stride_h
    else:
        s = g.stride()
        t.x_stride_b, t.x_stride_s, t.x_stride_h = s[:3] if len(s) == 4 else (0, *s[:2])
    t.x, t.out = g.data_ptr(), d.data_ptr()
    return g, d


def resnorm(residual, update, gate, post_weight, pre_weight, new_residual, normed, post_norm: bool, residual_scale: float,
            eps: float) -> MuResnorm:
    """residual [..., dim] is the residual, or in a gradient call the shape and
    type of it (new_residual then)."""
    base = residual if residual is not None else new_residual
    dim = base.shape[-1]
    rows = base.numel() // dim if dim else 0
    for t, what in ((residual, "residual"), (update, "update"), (new_residual, "new_residual"), (normed, "normed")):
        if t is None:
            continue
        _require(t, what)
        if t.shape != base.shape:
            raise ValueError(f"{what} must have the residual's shape")
    if new_residual is not None and new_residual.dtype != base.dtype:
        raise TypeError("new_residual must share the residual's dtype")
    kind = update if update is not None else normed if normed is not None else base
    if normed is not None and normed.dtype != kind.dtype:
        raise TypeError("normed must share the update's dtype")
    first = None   # of the weights and the gate
    for t, what in ((post_weight, "post_weight"), (pre_weight, "pre_weight"), (gate, "gate")):
        if t is None:
            continue
        _require(t, what)
        if first is not None and t.dtype != first.dtype:
            raise TypeError("the weights and the gate must share a dtype")
        first = t
        if t is not gate and t.shape != (dim,):
            raise ValueError(f"{what} must be [{dim}]")
    groups = 1
    if gate is not None:
        if gate.dim() not in (1, 2) or gate.shape[-1] != dim:
            raise ValueError(f"gate must be [{dim}] or [groups, {dim}]")
        groups = gate.numel() // dim if dim else 0
    return MuResnorm(_ptr(residual), _ptr(update), _ptr(gate), _ptr(post_weight), _ptr(pre_weight), _ptr(new_residual),
                     _ptr(normed), rows, dim, groups, _dtype_code(base), _dtype_code(kind),
                     MU_F32 if first is None else _dtype_code(first),
                     1 if post_norm else 0, float(residual_scale), float(eps))


def mu_residual_norm(a: MuResnorm, stream=None) -> None:
    _check(LIB.mu_residual_norm(ctypes.byref(a), _stream(stream)))


def resnorm_grad(grad_residual, grad_normed, r, update, gate, post_weight, pre_weight, post_norm: bool, residual_scale: float,
                 eps: float, results) -> MuResnormGrad:
    """r is new_residual, or x without an update; results (d_residual, d_update,
    d_gate, d_post, d_pre) are new tensors of their inputs' shapes and types."""
    for t, what in ((grad_residual, "grad_residual"), (grad_normed, "grad_normed")):
        if t is not None:
            _require(t, what)
            if t.shape != r.shape:
                raise ValueError(f"{what} must have the residual's shape")
    if grad_residual is not None and grad_residual.dtype != r.dtype:
        raise TypeError("grad_residual must share the residual's dtype")
    if update is None:
        f = resnorm(r, None, gate, post_weight, pre_weight, None, None, post_norm, residual_scale, eps)
        if grad_normed is not None:
            f.dtype = _dtype_code(grad_normed)
    else:
        f = resnorm(None, update, gate, post_weight, pre_weight, r, None, post_norm, residual_scale, eps)
        if grad_normed is not None and grad_normed.dtype != update.dtype:
            raise TypeError("grad_normed must share the update's dtype")
    return MuResnormGrad(f, _ptr(grad_residual), _ptr(grad_normed), *map(_ptr, results))


def resnorm_backward(args: MuResnorm, saved, need, dr, dn):
    """(MuResnormGrad, gradients) of a forward call's struct: saved (r, update,
    gate, post_weight, pre_weight), need which of their gradients, dr and dn those
    of the results, dense."""
    r, update, gate, post, pre = saved
    f = MuResnorm.from_buffer_copy(args)
    f.residual = f.new_residual = f.normed = None
    if update is None:
        f.residual = r.data_ptr()
    else:
        f.new_residual, f.update = r.data_ptr(), update.data_ptr()
    if gate is not None:
        f.gate = gate.data_ptr()
    if post is not None:
        f.post_weight = post.data_ptr()
    if pre is not None:
        f.pre_weight = pre.data_ptr()
    res = [torch.empty_like(t) if t is not None and w else None for t, w in zip(saved, need)]
    return MuResnormGrad(f, dr.data_ptr() if dr is not None else None, dn.data_ptr() if dn is not None else None,
                         *[None if t is None else t.data_ptr() for t in res]), res


def resnorm_grad_call(stream, a: MuResnormGrad, like) -> None:
    need = ctypes.c_size_t(0)
    ref = ctypes.byref(a)
    _check(LIB.mu_residual_norm_grad_workspace_size(ref, ctypes.byref(need)))
    ws = scratch(need.value, like.get_device())
    _check(LIB.mu_residual_norm_grad(ref, _ptr(ws), need.value, stream))


def mu_residual_norm_grad_workspace_size(a: MuResnormGrad) -> int:
    out = ctypes.c_size_t(0)
    _check(LIB.mu_residual_norm_grad_workspace_size(ctypes.byref(a), ctypes.byref(out)))
    return out.value


def mu_residual_norm_grad(a: MuResnormGrad, workspace: Optional[torch.Tensor], stream=None) -> None:
    ws = 0 if workspace is None else workspace.data_ptr()
    nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(LIB.mu_residual_norm_grad(ctypes.byref(a), ws, nb, _stream(stream)))


ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}
MU_GATES_F32 = 0x100


def _activation(name: str, gates: Optional[torch.Tensor]) -> int:
    """The activation's code, with the flag of float32 gates."""
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)} (got {name!r})")
    return ACTIVATIONS[name] | (MU_GATES_F32 if gates is not None and gates.dtype == torch.float32 else 0)


def _gated_sizes(x, w_gate, w_up):
    for t, what in ((x, "x"), (w_gate, "w_gate"), (w_up, "w_up")):
        _require(t, what)
        if t.dtype != x.dtype:
            raise TypeError("x, w_gate and w_up must share a dtype")
    if w_gate.dim() != 2 or w_up.shape != w_gate.shape:
        raise ValueError("w_gate and w_up must be 2-D and of one shape")
    if x.dim() < 1 or x.shape[-1] != w_gate.shape[1]:
        raise ValueError("x must be [..., dim] with the weights' row length")
    hidden, dim = w_gate.shape
    return x.numel() // dim if dim else 0, dim, hidden


def gated(x, w_gate, w_up, h, gates, activation: str) -> MuGated:
    tokens, dim, hidden = _gated_sizes(x, w_gate, w_up)
    _require(h, "out")
    if h.shape != x.shape[:-1] + (hidden,) or h.dtype != x.dtype:
        raise ValueError("out must have x's dtype and shape with hidden in the last place")
    if gates is not None:
        _require(gates, "gates")
        if gates.shape != (2,) + h.shape or gates.dtype not in (x.dtype, torch.float32):
            raise ValueError("gates must be [2, *out's shape] of x's dtype or float32")
    half = 0 if gates is None else tokens * hidden * gates.element_size()
    base = _ptr(gates)
    return MuGated(_ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(h), base, base + half if base else None, tokens, dim, hidden,
                   _dtype_code(x), _activation(activation, gates))


def mu_gated_mlp_workspace_size(a: MuGated) -> int:
    out = ctypes.c_size_t(0)
    _check(LIB.mu_gated_mlp_workspace_size(ctypes.byref(a), ctypes.byref(out)))
    return out.value


def mu_gated_mlp(a: MuGated, workspace: Optional[torch.Tensor], stream=None) -> None:
    ws = 0 if workspace is None else workspace.data_ptr()
    nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(LIB.mu_gated_mlp(ctypes.byref(a), ws, nb, _stream(stream)))


def gated_grad(grad, x, w_gate, w_up, gates, dx, d_gate, d_up, accumulate: bool, activation: str) -> MuGatedGrad:
    tokens, dim, hidden = _gated_sizes(x, w_gate, w_up)
    _require(grad, "grad")
    if grad.shape != x.shape[:-1] + (hidden,) or grad.dtype != x.dtype:
        raise ValueError("grad must have x's dtype and shape with hidden in the last place")
    if gates is not None:
        _require(gates, "gates")
        if gates.shape != (2,) + grad.shape or gates.dtype not in (x.dtype, torch.float32):
            raise ValueError("gates must be [2, *grad's shape] of x's dtype or float32")
    if dx is not None:
        _require(dx, "dx")
        if dx.shape != x.shape or dx.dtype != x.dtype:
            raise ValueError("dx must have x's shape and dtype")
    for t, what in ((d_gate, "d_gate"), (d_up, "d_up")):
        if t is not None:
            _require(t, what)
            if t.shape != w_gate.shape:
                raise ValueError(f"{what} must have the weights' shape")
    if d_gate is not None and d_up is not None and d_gate.dtype != d_up.dtype:
        raise TypeError("d_gate and d_up must share a dtype")
    half = 0 if gates is None else tokens * hidden * gates.element_size()
    base = _ptr(gates)
    return MuGatedGrad(_ptr(grad), _ptr(x), _ptr(w_gate), _ptr(w_up), base, base + half if base else None, _ptr(dx),
                       _ptr(d_gate), _ptr(d_up), tokens, dim, hidden, _dtype_code(x),
                       _dtype_code(x if d_gate is None else d_gate), 1 if accumulate else 0, _activation(activation, gates))


def gated_backward(args: MuGatedGrad, saved, need, grad):
    """(MuGatedGrad, gradients of x and the weights) with a forward call's sizes:
    saved (x, w_gate, w_up, gates or None), need which gradients, grad dense."""
    x, w_gate, w_up, gates = saved
    a = MuGatedGrad.from_buffer_copy(args)
    a.grad_h, a.x, a.w_gate, a.w_up = grad.data_ptr(), x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr()
    if gates is not None:
        a.gate = gates.data_ptr()
        a.up = a.gate + grad.numel() * gates.element_size() if a.gate else None
    dx = dg = du = None
    if need[0]:
        dx = torch.empty_like(x)
        a.dx = dx.data_ptr()
    if need[1] or need[2]:
        dg, du = torch.empty_like(w_gate), torch.empty_like(w_up)
        a.d_gate, a.d_up = dg.data_ptr(), du.data_ptr()
    return a, (dx, dg if need[1] else None, du if need[2] else None, dg, du)


def gated_grad_call(stream, a: MuGatedGrad, like) -> None:
    need = ctypes.c_size_t(0)
    ref = ctypes.byref(a)
    _check(LIB.mu_gated_mlp_grad_workspace_size(ref, ctypes.byref(need)))
    ws = scratch(need.value, like.get_device())
    _check(LIB.mu_gated_mlp_grad(ref, _ptr(ws), need.value, stream))


def mu_gated_mlp_grad_workspace_size(a: MuGatedGrad) -> int:
    out = ctypes.c_size_t(0)
    _check(LIB.mu_gated_mlp_grad_workspace_size(ctypes.byref(a), ctypes.byref(out)))
    return out.value


def mu_gated_mlp_grad(a: MuGatedGrad, workspace: Optional[torch.Tensor], stream=None) -> None:
    ws = 0 if workspace is None else workspace.data_ptr()
    nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(LIB.mu_gated_mlp_grad(ctypes.byref(a), ws, nb, _stream(stream)))


def qk_pairs(wqs, wks, max_logits, q_heads, k_heads, gamma_outs=None):
    n = len(wqs)
    arr = (MuQkPair * max(n, 1))()
    for i in range(n):
        wq, wk, ml = wqs[i], wks[i], max_logits[i]
        for t, what in ((wq, "wq"), (wk, "wk"), (ml, "max_logit")):
            _require(t, what)
        if wq.dim() != 2 or wk.dim() != 2 or wq.shape[1] != wk.shape[1]:
            raise ValueError("wq and wk must be 2-D with the same number of columns")
        if wk.dtype != wq.dtype or ml.dtype != torch.float32:
            raise TypeError("wk must share wq's dtype and max_logit must be float32")
        go = None if gamma_outs is None else gamma_outs[i]
        if go is not None:
            _require(go, "gamma_out")
        arr[i] = MuQkPair(_ptr(wq), _ptr(wk), wq.shape[0], wk.shape[0], wq.shape[1], int(q_heads[i]),
                          int(k_heads[i]), _dtype_code(wq), 0, _ptr(ml), _ptr(go))
    return arr, n


def mu_qk_clip_workspace_size(pairs, n) -> int:
    out = ctypes.c_size_t(0)
    _check(LIB.mu_qk_clip_workspace_size(pairs, n, ctypes.byref(out)))
    return out.value


def mu_qk_clip(pairs, n, tau: float, workspace: Optional[torch.Tensor], stream=None) -> None:
    ws = 0 if workspace is None else workspace.data_ptr()
    nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(LIB.mu_qk_clip(pairs, n, float(tau), ws, nb, _stream(stream)))


def mu_version() -> int:
    return LIB.mu_version()


def mu_status_string(status: int) -> str:
    return _status_text(status)


def mu_last_error() -> str:
    return LIB.mu_last_error().decode()


def mu_profile_enable(on: bool) -> None:
    _check(LIB.mu_profile_enable(1 if on else 0))


def mu_profile_read(kernel: int) -> dict:
    ms = ctypes.c_double(0)
    n = ctypes.c_int64(0)
    fl = ctypes.c_double(0)
    by = ctypes.c_double(0)
    _check(LIB.mu_profile_read(kernel, ctypes.byref(ms), ctypes.byref(n), ctypes.byref(fl), ctypes.byref(by)))
    return {"kernel": LIB.mu_kernel_name(kernel).decode(), "ms": ms.value, "launches": n.value,
            "flops": fl.value, "bytes": by.value}


def mu_kernel_name(kernel: int) -> str:
    return LIB.mu_kernel_name(kernel).decode()


def workspace(nbytes: int, device, stream=None) -> Optional[torch.Tensor]:
    """A 256-byte aligned uint8 device buffer of at least nbytes (None for 0)
    for work on `stream` (default: the current one)."""
    if nbytes == 0:
        return None
    buf = allocate(lambda: torch.empty(nbytes + 256, dtype=torch.uint8, device=device), device, stream)
    off = (-buf.data_ptr()) % 256
    return buf[off:off + nbytes]


def torch_stream(stream, device) -> torch.cuda.Stream:
    """A torch stream object as it is, or one for a raw hipStream_t value."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    if int(stream) == 0:   # ExternalStream takes 0 for "any stream"
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(int(stream), device=device)


def allocate(make, device, stream, returned: bool = False):
    """make() with `stream` current. The caching allocator hands out memory as
    soon as its last owner has dropped it, when kernels queued on the stream of
    that allocation may still use it: only work on the same stream comes behind
    them. So a buffer of work on `stream` is allocated there, wherever the caller
    works. One that is `returned` to the caller is also recorded on the caller's
    stream, where it is read next."""
    if stream is None:
        return make()
    caller = torch.cuda.current_stream(device)
    with torch.cuda.stream(torch_stream(stream, device)):
        buf = make()
        if returned:
            tie_to_stream(buf, caller)
    return buf


def tie_to_stream(buf: Optional[torch.Tensor], stream, current=None) -> None:
    """Keep a buffer allocated on the current stream alive for work queued on
    `stream` (a torch stream or a raw hipStream_t value): the caching
    allocator may otherwise hand its memory to the next allocation on the
    current stream as soon as the caller drops it, while kernels on `stream`
    still use it. No-op for None or for the current stream."""
    if buf is None or stream is None:
        return
    stream = torch_stream(stream, buf.device)
    cur = torch.cuda.current_stream(buf.device) if current is None else current
    if stream.cuda_stream != cur.cuda_stream:
        buf.record_stream(stream)
