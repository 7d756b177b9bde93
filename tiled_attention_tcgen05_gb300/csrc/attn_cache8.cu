// attn_cache_rows.cuh's kernels for 8-bit caches.
#include "attn_cache_rows.cuh"

namespace ta {

cudaError_t launch_attn_cache_rows8(bool bf16, int ct, int D, int mt, const CacheArgs& c, const CacheAttnArgs& a,
                                    cudaStream_t s) {
  if (ct == kCacheE4m3)
    return bf16 ? run_d<__nv_bfloat16, kCacheE4m3>(D, mt, c, a, s) : run_d<__half, kCacheE4m3>(D, mt, c, a, s);
  return bf16 ? run_d<__nv_bfloat16, kCacheI8>(D, mt, c, a, s) : run_d<__half, kCacheI8>(D, mt, c, a, s);
}

}  // namespace ta

TA_GUARD_ACCESSOR(attn_cache8)
