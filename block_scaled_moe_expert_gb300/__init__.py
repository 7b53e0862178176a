"""Block-scaled MoE experts forward for GB300 (sm_103a).

The compute path is the CUDA library built from csrc/ (libbsmoe.so, C ABI in
include/moe_experts.h); `binding` marshals torch tensors into it. The operators
around the forward (tokens sorted by expert and back, norms around the block,
4-bit products) are in include/moe_block.h, routing, the FP4 format and its
products in include/moe_route_fp4.h, the Python functions of both in `block`.
"""
from .binding import (MoeError, PreparedWeights, device_status, experts_forward, prepare_weights,  # noqa: F401
                      workspace_bytes, workspace_layout)
from .block import (PreparedMatmulFp4, PreparedMatvec, SortPlan, dequantize_fp4, matmul_fp4, matvec,  # noqa: F401
                    norm_after, norm_after_backward, norm_before, norm_before_backward, permute_tokens,
                    permute_tokens_backward, prepare_matmul_fp4, prepare_matvec, quantize_fp4, route_tokens,
                    route_tokens_backward, sort_tokens, unpermute_tokens, unpermute_tokens_backward)
