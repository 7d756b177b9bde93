// The rotary kernels (rotary_kernels.cuh) on fp16 rows.
#include "rotary_kernels.cuh"

namespace ta {
cudaError_t launch_rotary_f16(int mode, int ct, int D, const RotArgs& a, const CacheArgs& c, cudaStream_t s) {
  return run_rotary_t<__half>(mode, ct, D, a, c, s);
}
}  // namespace ta

TA_GUARD_ACCESSOR(rotary_f16)
