"""B200-native PagedAttention over a block-table KV cache.

The hot path lives in libtv.so (CUDA kernels for sm_100a behind the C ABI of
include/tv.h); this package is its thin Python binding plus the seeded
synthetic workloads used by the tests and the benchmark.
"""
from ._lib import (TVError, load, tv_kv_append,  # noqa: F401
                   tv_kv_append_mrope, tv_page_copy, tv_paged_chunk,
                   tv_paged_cross_attention, tv_paged_decode,
                   tv_paged_decode_append, tv_paged_decode_split,
                   tv_paged_decode_split_static, tv_paged_prefill,
                   tv_pool_compact, tv_pool_truncate, tv_split_merge)

__all__ = ["TVError", "load", "tv_kv_append", "tv_paged_decode",
           "tv_paged_decode_append", "tv_paged_decode_split",
           "tv_split_merge", "tv_paged_prefill",
           "tv_paged_decode_split_static", "tv_kv_append_mrope",
           "tv_paged_chunk", "tv_paged_cross_attention", "tv_pool_truncate",
           "tv_pool_compact", "tv_page_copy"]
