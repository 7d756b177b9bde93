// attn_cache_rows.cuh's kernels for int8 caches.
#include "attn_cache_rows.cuh"

namespace ta {

cudaError_t launch_attn_cache_rows_i8(bool bf16, int D, int mt, const CacheArgs& c, const CacheAttnArgs& a,
                                      cudaStream_t s) {
  return bf16 ? run_d<__nv_bfloat16, kCacheI8>(D, mt, c, a, s) : run_d<__half, kCacheI8>(D, mt, c, a, s);
}

}  // namespace ta

TA_GUARD_ACCESSOR(attn_cache_i8)
