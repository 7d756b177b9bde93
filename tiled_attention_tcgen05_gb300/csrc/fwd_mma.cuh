// The two matrix products of a forward attention step on 128-row tiles.
#pragma once
#include "common.cuh"

namespace ta {

// 32 consecutive registers of an array, as the TMEM loads take them.
#define TA_CHUNK(arr, c) (*reinterpret_cast<uint32_t(*)[32]>(&(arr)[32 * (c)]))

// d = A B^T over the head dimension: A, B are 128 x D K-major swizzled tiles.
// The descriptors are built once; each K-step adds its byte offset / 16 to
// the 14-bit start-address field (shared addresses stay below 256 KB, so the
// add never carries out of the field).
template <int D>
__device__ __forceinline__ void mma_qk(uint32_t d_tmem, uint32_t a_smem, uint32_t b_smem, uint32_t idesc,
                                       bool accumulate) {
  const uint64_t da0 = sdesc_sw128(a_smem, 16, 1024);
  const uint64_t db0 = sdesc_sw128(b_smem, 16, 1024);
  uint64_t da[D / 16], db[D / 16];
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint64_t off = static_cast<uint64_t>(((kk >> 2) * (kBM * 128) + (kk & 3) * 32) >> 4);
    da[kk] = da0 + off;
    db[kk] = db0 + off;
  }
  mma_ss_n<D / 16>(d_tmem, da, db, idesc, accumulate ? 1u : 0u);
}

// d (+)= P V: P is 128 x 128 (16-bit, TMEM), V is 128 keys x D stored with D
// contiguous (MN-major B operand; 64-column blocks kBM*128 bytes apart).
template <int D>
__device__ __forceinline__ void mma_pv(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_smem, uint32_t idesc,
                                       bool accumulate) {
  const uint64_t dv = sdesc_sw128(v_smem, kBM * 128, 1024);
  uint32_t a[kBN / 16];
  uint64_t b[kBN / 16];
#pragma unroll
  for (int kk = 0; kk < kBN / 16; ++kk) {
    a[kk] = p_tmem + kk * 8;
    b[kk] = dv + static_cast<uint64_t>((kk * 16 * 128) >> 4);
  }
  mma_ts_n<kBN / 16>(d_tmem, a, b, idesc, accumulate ? 1u : 0u);
}

}  // namespace ta
