"""MI355X-native TACO FP8 compression operator for tensor-parallel intermediate tensors.

Python face of libtaco (include/taco.h): ``compress``, ``decompress`` and
``decompress_sum`` over bf16 [tokens, hidden] GPU tensors, and the operators of
an 8-bit linear layer (include/taco_linear.h): block-scaled FP8 quantisation,
norm, matrix product, gradients and gated unit.  The library is loaded on first
use and the calls raise if it is missing; there is no CPU path.
"""
from ._binding import (  # noqa: F401
    TACO_AMAX_FLOATS,
    TACO_AMAX_SLOTS,
    TACO_MAX_PARTS,
    TacoError,
    compress,
    compress_blockscale,
    compress_delayed,
    compress_int8,
    compress_noalloc,
    TACO_DEFAULT_BARRIER_POLLS,
    TACO_FLAG_TWO_PASS,
    is_single_pass,
    two_shot_allreduce,
    decompress,
    decompress_blockscale,
    decompress_int8,
    decompress_sum,
    decompress_sum_compress,
    library_path,
    load,
    num_scales,
    version,
    workspace_bytes,
    workspace_timed_out,
)
from ._linear import (  # noqa: F401
    fp8_cols,
    fp8_scale_cols,
    matmul_fp8,
    matmul_fp8_workspace_bytes,
    quantize_rows,
    quantize_weight,
    rmsnorm_backward,
    rmsnorm_backward_workspace_bytes,
    rmsnorm_quantize,
    swiglu_backward,
    swiglu_quantize,
    wgrad_fp8,
    wgrad_fp8_workspace_bytes,
)

__all__ = [
    "TACO_AMAX_FLOATS", "TACO_AMAX_SLOTS", "TACO_DEFAULT_BARRIER_POLLS", "TACO_FLAG_TWO_PASS", "TACO_MAX_PARTS",
    "TacoError", "compress", "compress_blockscale", "compress_delayed", "compress_int8", "compress_noalloc", "decompress",
    "decompress_blockscale", "decompress_int8", "decompress_sum", "decompress_sum_compress", "fp8_cols",
    "fp8_scale_cols", "is_single_pass", "library_path", "load", "matmul_fp8", "matmul_fp8_workspace_bytes",
    "num_scales", "quantize_rows", "quantize_weight", "rmsnorm_backward", "rmsnorm_backward_workspace_bytes",
    "rmsnorm_quantize", "swiglu_backward", "swiglu_quantize", "two_shot_allreduce", "version", "wgrad_fp8",
    "wgrad_fp8_workspace_bytes", "workspace_bytes", "workspace_timed_out",
]
