"""MI355X (gfx950) AWQ activation-aware scale search and INT4 group quantization.

The computation lives in the HIP library libawq_mi355x.so behind the C ABI of
include/awq.h and include/awq_moe.h; `binding` and `moe` expose its entry points to Python with the
same names.
"""
from . import binding, moe  # noqa: F401
from .binding import (AwqError, awq_act_stats, awq_candidate_scales, awq_error_sse, awq_error_tiles,
                      awq_layer, awq_loss_argmin, awq_quant_delta, awq_quantize_pack, awq_search_scales,
                      load_library)
from .moe import (awq_block_norm, awq_block_norm_backward, awq_moe_combine, awq_moe_combine_backward, awq_moe_gather,
                  awq_moe_gather_backward, awq_moe_sort, awq_w4a16_grouped_gemm, awq_w4a16_grouped_gemm_backward)

__all__ = ["AwqError", "awq_act_stats", "awq_candidate_scales", "awq_error_sse", "awq_error_tiles",
           "awq_layer", "awq_loss_argmin", "awq_quant_delta", "awq_quantize_pack", "awq_search_scales",
           "awq_block_norm", "awq_block_norm_backward", "awq_moe_combine", "awq_moe_combine_backward",
           "awq_moe_gather", "awq_moe_gather_backward", "awq_moe_sort", "awq_w4a16_grouped_gemm",
           "awq_w4a16_grouped_gemm_backward", "load_library", "binding", "moe"]
