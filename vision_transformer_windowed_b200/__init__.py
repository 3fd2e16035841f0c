"""B200-native FlashSwin windowed-RoPE attention (forward and backward), and the operators of a Swin layer around it:
attention with a learned relative position bias, the residual step with its norms, the gated feed-forward block.

The compute lives in ``libfswin.so`` (hand-written CUDA for sm_100a, C ABI in
``include/fswin.h``); this package only marshals arguments to it.
"""
from ._lib import FswinError, MlpShape, ResnormShape, Shape, load, make_shape, status_string  # noqa: F401
from .ops import (WindowAttentionRoPE, alloc_relbias_workspace, alloc_workspace, bwd_workspace_bytes,  # noqa: F401
                  gated_mlp, gated_mlp_bwd, gated_mlp_fwd, log_distance_buckets, residual_norm, residual_norm_bwd,
                  residual_norm_fwd, window_attention, window_attention_relbias, winattn_bwd, winattn_fwd,
                  winattn_relbias_bwd, winattn_relbias_fwd)

__all__ = ["FswinError", "MlpShape", "ResnormShape", "Shape", "load", "make_shape", "status_string",
           "WindowAttentionRoPE", "alloc_relbias_workspace", "alloc_workspace", "bwd_workspace_bytes", "gated_mlp",
           "gated_mlp_bwd", "gated_mlp_fwd", "log_distance_buckets", "residual_norm", "residual_norm_bwd",
           "residual_norm_fwd", "window_attention", "window_attention_relbias", "winattn_bwd", "winattn_fwd",
           "winattn_relbias_bwd", "winattn_relbias_fwd"]
