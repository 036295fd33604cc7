"""MI355X (gfx950) fused SwiGLU GEMM: Y = SiLU(A.W1) (.) (A.W2).

The computation lives in the HIP library ``libswiglu.so`` (C ABI in
``include/swiglu.h``); ``gated_mlp_gemm_amd.swiglu`` is its ctypes binding.
Importing the package does not load the library; the first call does, and
fails loudly if it is not built (``python -m gated_mlp_gemm_amd.build``).
"""
from .swiglu import (  # noqa: F401
    SWIGLU_AUTO, SWIGLU_VARIANT_I, SWIGLU_VARIANT_S, SwigluError, SwigluLora, load_library,
    make_lora_workspace, make_workspace, swiglu_dequantize_mx4, swiglu_describe_backward,
    swiglu_describe_launch,
    swiglu_down_proj, swiglu_down_proj_backward, swiglu_down_proj_lora, swiglu_down_proj_mx4,
    swiglu_fp8_scale_exp, swiglu_fused_gemm, swiglu_fused_gemm_backward, swiglu_fused_gemm_fp8,
    swiglu_fused_gemm_lora, swiglu_fused_gemm_mx4, swiglu_fused_gemm_noalloc,
    swiglu_fused_gemm_strided, swiglu_fused_gemm_train, swiglu_gated_mlp,
    swiglu_gated_mlp_backward, swiglu_gated_mlp_lora, swiglu_gated_mlp_mx4,
    swiglu_gated_mlp_train, swiglu_last_error, swiglu_lora_workspace_size, swiglu_m_switch,
    swiglu_pack_weights, swiglu_pack_weights_nk, swiglu_quantize_fp8, swiglu_quantize_mx4,
    swiglu_route, swiglu_route_backward,
    swiglu_route_workspace_size, swiglu_select_variant, swiglu_silu_mul, swiglu_status_string,
    swiglu_unfused_ablation, swiglu_workspace_size,
)
