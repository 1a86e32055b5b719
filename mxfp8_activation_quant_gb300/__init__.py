"""GB300 (sm_103a) MXFP8 activation chain: standalone quantizer, the fused `_o_proj` pair
(wo_a einsum writing MXFP8 z, wo_b MXFP8 GEMM consuming it), the RMSNorm dual-output producer,
the mixture-of-experts half of the layer (residual RMSNorm, router, experts' products), and the
paged MXFP8 key-value cache with the attention that reads it, behind the C ABI in include/mxq.h,
include/mxq_moe.h and include/mxq_kv.h. The Python layer only marshals arguments."""
from ._lib import (  # noqa: F401
    MXFP8,
    SF_PACKED_I32_MN,
    SF_ROWMAJOR_U8,
    SF_TILED_128X4,
    MxqError,
    abi_version,
    check_status,
    empty_sf,
    gemm_mxfp8_bf16,
    load,
    mxfp8_quantize,
    new_status,
    o_proj_mxfp8,
    o_proj_mxfp8_from_bf16,
    o_proj_mxfp8_noalloc,
    quantize,
    rmsnorm_dual_out,
    selftest_hold_sms,
    selftest_wait_timeout,
    sf_bytes,
    status_bytes,
    wo_a_einsum_mxfp8,
    workspace_bytes,
    workspace_for,
)
from .moe import (  # noqa: F401
    add_rmsnorm_dual_out,
    interleave_gate_up,
    moe_experts_mxfp8,
    moe_route,
    moe_workspace_bytes,
)
from .kv import (  # noqa: F401
    MXFP8Cache,
    kv_read_bf16,
    kv_write_mxfp8,
    paged_attention_mxfp8,
    paged_attention_workspace_bytes,
)
