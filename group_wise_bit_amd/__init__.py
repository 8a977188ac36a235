"""qlin on MI355X: fused dequantize-matmul over group-wise affine low-bit weights.

The computation lives in libqlin.so (HIP kernels for gfx950 behind the C ABI in
include/qlin.h, qlin_rows.h, qlin_kv.h and qlin_sample.h); this package is its Python binding.
"""
from .qlin import (  # noqa: F401
    FMT_FP16_MASTER, FMT_PACKED, EXPORTS, KV_EXPORTS, LIB_PATH, ROWS_EXPORTS, SAMPLE_EXPORTS,
    Adapters, KVCache, QExperts, QWeight, QlinError, Router, Sampling, embed_rows, gemm, gemm_lora,
    gemm_multi, gemv, gemv_multi, gemv_swiglu, kv_attention, kv_cache, kv_page_bytes, kv_read,
    kv_write, library, master_weight, meta_entries, moe_mlp, packed_bytes, quantize, quantize_batch,
    quantize_experts, route, sample, workspace,
)
