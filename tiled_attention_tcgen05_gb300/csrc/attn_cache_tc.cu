// attn_cache_tc.cuh's kernels for 16-bit caches.
#include "attn_cache_tc.cuh"

namespace ta {

size_t attn_cache_tc16_ws_bytes(int D) { return tc_ws_bytes<kCache16>(D); }

cudaError_t launch_attn_cache_tc16(bool bf16, int D, const PageMaps& m, const CacheArgs& c, const CacheAttnArgs& a, cudaStream_t s) {
  if (D <= 64)
    return bf16 ? run_tc<__nv_bfloat16, kCache16, 64>(D, m, c, a, s) : run_tc<__half, kCache16, 64>(D, m, c, a, s);
  return bf16 ? run_tc<__nv_bfloat16, kCache16, 128>(D, m, c, a, s) : run_tc<__half, kCache16, 128>(D, m, c, a, s);
}

}  // namespace ta

TA_GUARD_ACCESSOR(attn_cache_tc)
