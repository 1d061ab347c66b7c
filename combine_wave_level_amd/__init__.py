"""MI355X-native (gfx950) share of a fine-grained expert-parallel MoE layer.

The compute path is the HIP library ``libmoe.so`` (C ABI: include/moe.h);
``combine_wave_level_amd.moe`` is its thin Python binding.
"""
from . import moe  # noqa: F401
from .moe import (  # noqa: F401
    MOE_ACT_RELU2, MOE_ACT_SWIGLU, MOE_BF16, MOE_F32, MOE_FLAG_SERIAL, MoEError, Problem, backward, combine,
    dequantize_mxfp4, dispatch, ffn_mxfp4, ffn_waved, ffn_waved_fp8, forward, forward_few, forward_mxfp4,
    pack_weights, pack_weights_bwd, pack_weights_mxfp4, problem, quantize_fp8, quantize_mxfp4, route,
    unpack_weights_mxfp4, wgrad, workspace, workspace_size,
)
