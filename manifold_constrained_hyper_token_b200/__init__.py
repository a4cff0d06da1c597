"""mHC (manifold-constrained hyper-connections) layer hot path for NVIDIA B200.

The computation lives in ``libmhc.so`` (CUDA, sm_100a; C ABI in
``include/mhc.h``).  This package holds the build script, a ctypes binding
with the C entry points' names (``api``) and the seeded synthetic input
recipes (``synth``), the depth-stack driver with block recompute (``depth``) and
the feed-forward layer function it can wrap (``feedforward``).
"""
from .api import (MhcError, mhc_backward, mhc_backward_apply, mhc_backward_map,
                  mhc_backward_noalloc, mhc_backward_workspace_size, mhc_depth_amax, mhc_ffn,
                  mhc_ffn_backward, mhc_ffn_backward_workspace_size, mhc_ffn_workspace_size,
                  mhc_layer_norm, mhc_layer_norm_backward,
                  mhc_layer_norm_backward_workspace_size, mhc_post, mhc_layer_input, mhc_post_backward, mhc_post_fused, mhc_pre,
                  mhc_pre_backward, mhc_pre_workspace_size, mhc_recompute_plan,
                  mhc_sinkhorn_knopp, mhc_status_string, mhc_version, params)

__all__ = ["MhcError", "mhc_backward", "mhc_backward_apply", "mhc_backward_map",
           "mhc_backward_noalloc", "mhc_backward_workspace_size", "mhc_depth_amax", "mhc_ffn",
           "mhc_ffn_backward", "mhc_ffn_backward_workspace_size", "mhc_ffn_workspace_size",
           "mhc_layer_norm", "mhc_layer_norm_backward",
           "mhc_layer_norm_backward_workspace_size", "mhc_post",
           "mhc_layer_input", "mhc_post_backward", "mhc_post_fused", "mhc_pre",
           "mhc_pre_backward", "mhc_pre_workspace_size", "mhc_recompute_plan",
           "mhc_sinkhorn_knopp", "mhc_status_string", "mhc_version", "params"]
