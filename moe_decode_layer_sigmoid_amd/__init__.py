"""MI355X (gfx950) decode-step MoE layer with a sigmoid router, and the
operators beside it: the block-scaled fp8 product with its activation
quantiser, and attention over an 8-bit paged cache with append and eviction.

The layer runs in hand-written HIP kernels behind the C ABI declared in
include/moe_decode.h (libmoe_decode.so, built in-tree by
``python -m moe_decode_layer_sigmoid_amd.build``).  This package is its thin
Python binding; PyTorch only provides device memory and streams.
"""

from .binding import (  # noqa: F401
    Args,
    Desc,
    MoeDecodeError,
    Plan,
    EXPORTED,
    LIB_PATH,
    OK,
    ERR_HIP,
    ERR_INVALID_ARG,
    ERR_NO_MEMORY,
    ERR_SCRATCH,
    STATIC_SCRATCH_BYTES,
    ERR_UNSUPPORTED,
    PATH_AUTO,
    PATH_GEMV,
    PATH_GROUPED,
    PATH_GEMV_SPLIT,
    SCALE_E8M0,
    SCALE_FP32,
    args_check,
    desc_check,
    lib,
    make_desc,
    read_probe,
    run_static,
    strerror,
    PROBE_STEP,
)
from .ops import (  # noqa: F401
    AppendArgs,
    AttendArgs,
    Cache,
    CacheDesc,
    CachePlan,
    EvictArgs,
    OUT_BF16,
    OUT_FP32,
    PAGE_TOKENS,
    ProductArgs,
    ProductDesc,
    ProductPlan,
    append_check,
    attend_check,
    cache_desc_check,
    evict_check,
    make_cache_desc,
    make_product_desc,
    product_args_check,
    product_desc_check,
    quant,
)
