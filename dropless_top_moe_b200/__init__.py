"""B200-native dropless top-k Mixture-of-Experts layer (sm_100a CUDA kernels
behind a C ABI, include/moe.h).  Python here only marshals arguments."""
from ._lib import LIB_PATH, MOE_LAYER_GATHER_ROWS, MoEError, load
from .ops import (MoEDecodeLayer, MoELayer, clip_workspace, device_status, moe_add_rms_norm, moe_add_rms_norm_bwd, moe_aux_loss,
                  moe_clip_grad_norm, moe_combine, moe_combine_bwd, moe_dispatch_meta,
                  moe_grouped_swiglu, moe_grouped_swiglu_bwd, moe_permute, moe_route,
                  moe_unpermute_router_bwd, padded_rows_max, selftest_handover_timeout, selftest_wait_timeout,
                  tile_rows, workspace)

__all__ = ["LIB_PATH", "MOE_LAYER_GATHER_ROWS", "MoEError", "load", "MoELayer", "MoEDecodeLayer", "device_status", "moe_aux_loss", "moe_combine",
           "moe_combine_bwd", "moe_dispatch_meta", "moe_grouped_swiglu", "moe_grouped_swiglu_bwd",
           "moe_permute", "moe_route", "moe_unpermute_router_bwd", "padded_rows_max", "selftest_wait_timeout",
           "selftest_handover_timeout",
           "tile_rows",
           "clip_workspace", "moe_add_rms_norm", "moe_add_rms_norm_bwd", "moe_clip_grad_norm",
           "workspace"]
