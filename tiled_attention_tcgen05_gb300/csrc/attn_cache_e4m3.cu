// attn_cache_rows.cuh's kernels for e4m3 caches.
#include "attn_cache_rows.cuh"

namespace ta {

cudaError_t launch_attn_cache_rows_e4m3(bool bf16, int D, int mt, const CacheArgs& c, const CacheAttnArgs& a,
                                        cudaStream_t s) {
  return bf16 ? run_d<__nv_bfloat16, kCacheE4m3>(D, mt, c, a, s) : run_d<__half, kCacheE4m3>(D, mt, c, a, s);
}

}  // namespace ta

TA_GUARD_ACCESSOR(attn_cache_e4m3)
