// attn_cache_tc.cuh's kernels for 8-bit caches.
#include "attn_cache_tc.cuh"

namespace ta {

size_t attn_cache_tc8_ws_bytes(int D) { return tc_ws_bytes<kCacheE4m3>(D); }

template <int CT>
static cudaError_t run_ct(bool bf16, int D, const PageMaps& m, const CacheArgs& c, const CacheAttnArgs& a, cudaStream_t s) {
  if (D <= 64) return bf16 ? run_tc<__nv_bfloat16, CT, 64>(D, m, c, a, s) : run_tc<__half, CT, 64>(D, m, c, a, s);
  return bf16 ? run_tc<__nv_bfloat16, CT, 128>(D, m, c, a, s) : run_tc<__half, CT, 128>(D, m, c, a, s);
}

cudaError_t launch_attn_cache_tc8(bool bf16, int ct, int D, const PageMaps& m, const CacheArgs& c,
                                  const CacheAttnArgs& a, cudaStream_t s) {
  return ct == kCacheE4m3 ? run_ct<kCacheE4m3>(bf16, D, m, c, a, s) : run_ct<kCacheI8>(bf16, D, m, c, a, s);
}

}  // namespace ta

TA_GUARD_ACCESSOR(attn_cache_tc8)
