// The rotary kernels (rotary_kernels.cuh) on bf16 rows.
#include "rotary_kernels.cuh"

namespace ta {
cudaError_t launch_rotary_bf16(int mode, int ct, int D, const RotArgs& a, const CacheArgs& c, cudaStream_t s) {
  return run_rotary_t<__nv_bfloat16>(mode, ct, D, a, c, s);
}
}  // namespace ta

TA_GUARD_ACCESSOR(rotary_bf16)
