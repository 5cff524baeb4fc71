"""MI355X-native Muon optimizer step (momentum, Frobenius normalisation,
Newton-Schulz orthogonalisation, decoupled-weight-decay update) and fused
AdamW, on hand-written gfx950 HIP kernels behind a C ABI, with what a training
loop computes to feed the step: gradient norm and clipping, the embedding and
its gradient, and the attention max logits of QK-Clip.

The HIP library is loaded on first use of any compute entry point; a missing
library raises ImportError (there is no CPU fallback).
"""

_CALLS = ("muon_step", "orthogonalize", "adamw_step", "qk_clip", "muon_workspace_bytes", "grad_norm", "clip_grads",
          "embedding", "embedding_grad", "qk_max_logits")
__all__ = [*_CALLS, "MuonAdamW", "split_params"]


def __getattr__(name):
    if name in _CALLS:
        from . import api as mod
    elif name in ("MuonAdamW", "split_params"):
        from . import optim as mod
    else:
        raise AttributeError(name)
    globals()[name] = value = getattr(mod, name)   # found without this function from now on
    return value
