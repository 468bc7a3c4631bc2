"""GB300-native KV residency path for index-based sparse attention (single-GPU DP mode).

``ula`` is the ctypes binding of the C ABI (include/ula.h) implemented by the
CUDA library ``_build/libula.so``; ``cache.UlaCache`` adds the PyTorch pools
and streams; ``rows`` holds the operators on the cache's FP8 rows (rotary positions,
packing, norms with either, attention, also of trees of drafted tokens, joining partial results, accumulated
weights, eviction).  Build with ``serving_step_sparse_gb300.build.build()``.
"""
__all__ = ["ula", "cache", "rows"]
