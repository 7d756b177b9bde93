// attn_cache_rows.cuh's kernels for 16-bit caches, and the choice between the
// kernels of the attention over a cache.
#include <algorithm>

#include "attn_cache_rows.cuh"

namespace ta {

cudaError_t launch_attn_cache_rows_e4m3(bool bf16, int D, int mt, const CacheArgs& c, const CacheAttnArgs& a,
                                        cudaStream_t s);
cudaError_t launch_attn_cache_rows_i8(bool bf16, int D, int mt, const CacheArgs& c, const CacheAttnArgs& a,
                                      cudaStream_t s);

// Row tiles (of 16) per unit: as many as the accumulators leave registers for.
static int row_tiles(int D, long long rows) {
  const long long most = D <= 32 ? 4 : D <= 64 ? 3 : 2;
  return static_cast<int>(std::min((rows + 15) / 16, most));
}

size_t attn_cache_ws_bytes(int D, long long rows) {
  const int mt = row_tiles(D, rows);
  const size_t blocks = mt == 1 ? Cfg<kCache16, 64, 1>::BLOCKS : Cfg<kCache16, 64, 2>::BLOCKS;
  return blocks * (2 * (16 * mt) * (D + 2) * sizeof(float) + sizeof(CutUnit));
}

cudaError_t launch_attn_cache(bool bf16, int ct, int D, const CacheArgs& c, const CacheAttnArgs& a, cudaStream_t s) {
  const int mt = row_tiles(D, static_cast<long long>(a.G) * c.T);
  if (ct == kCacheE4m3) return launch_attn_cache_rows_e4m3(bf16, D, mt, c, a, s);
  if (ct == kCacheI8) return launch_attn_cache_rows_i8(bf16, D, mt, c, a, s);
  return bf16 ? run_d<__nv_bfloat16, kCache16>(D, mt, c, a, s) : run_d<__half, kCache16>(D, mt, c, a, s);
}

}  // namespace ta

TA_GUARD_ACCESSOR(attn_cache)
