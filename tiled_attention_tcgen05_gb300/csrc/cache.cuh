// The paged key/value cache as the kernels see it: arguments, the page look-up
// and the checks of what the caller's device arrays hold.
//
// Position n of sequence b is row n % page of page table[b][n / page]; a row
// of head h there is row (id * Hkv + h) * page + n % page of k, v (D elements
// each) and of the scales (one float).
#pragma once
#include <cstdint>

#include "common.cuh"

namespace ta {

// Bit of the device error word (ptx.cuh): a length, page or token index outside
// the cache.
constexpr uint32_t kErrIndex = 1u << 6;

enum CacheType : int { kCache16 = 0, kCacheE4m3 = 1, kCacheI8 = 2 };

// The scale of a row is amax / kQmax, at least this (a row of zeros, or of
// values too small for it, gets codes that round toward zero).
constexpr float kMinScale = 8.673617379884035e-19f;  // 2^-60

// n / d for 0 <= n < 2^31 by one multiplication: m = floor(2^(31+s) / d) + 1
// with 2^s >= d, so that m d - 2^(31+s) <= d <= 2^s and the error n (m d -
// 2^(31+s)) / (d 2^(31+s)) stays under 1 / d.
struct FastDiv {
  uint32_t d, m, s;
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return static_cast<uint32_t>((static_cast<uint64_t>(n) * m) >> s);
  }
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  FastDiv f;
  f.d = d;
  f.m = static_cast<uint32_t>((1ull << (31 + s)) / d + 1);
  f.s = 31 + s;
  return f;
}

struct CacheArgs {
  void *k, *v;        // [num_pages, Hkv, page, D]
  float *ks, *vs;     // [num_pages, Hkv, page], 8-bit types only
  const int* table;   // [B, max_pages]
  const int* kv_lens; // [B]: tokens with the new ones
  const int* q_lens;  // [B]: new tokens; null: T each
  int num_pages, Hkv, max_pages, B, T;
  int capacity;       // min(max_pages * page, 2^31 - 1): positions a sequence can have
  FastDiv page;
  uint32_t* err;
};

__device__ __forceinline__ void cache_error(uint32_t* err) {
  if (err) atomicOr(err, kErrIndex);
}

// Tokens (kv) and new tokens (q) of sequence b.  Lengths that cannot be
// (q outside [0, T], kv < q, kv past the page table) are recorded in the error
// word and read as an empty sequence.
struct SeqLens {
  int kv, q;
};
__device__ __forceinline__ SeqLens cache_lens(const CacheArgs& c, int b) {
  SeqLens s;
  s.kv = __ldg(c.kv_lens + b);
  s.q = c.q_lens ? __ldg(c.q_lens + b) : c.T;
  if (s.q < 0 || s.q > c.T || s.kv < s.q || s.kv > c.capacity) {
    cache_error(c.err);
    s.kv = s.q = 0;
  }
  return s;
}

// Page of position n < kv: its table entry and the row in it.
__device__ __forceinline__ int cache_page_id(const CacheArgs& c, int b, int n, int* r) {
  const uint32_t col = c.page.div(static_cast<uint32_t>(n));
  *r = n - static_cast<int>(col * c.page.d);
  return __ldg(c.table + static_cast<long long>(b) * c.max_pages + col);
}

// Row (of D elements) of head h at row r of page id; -1, recorded, for a page
// the cache does not have.
__device__ __forceinline__ int cache_row(const CacheArgs& c, int h, int id, int r) {
  if (static_cast<unsigned>(id) >= static_cast<unsigned>(c.num_pages)) {
    cache_error(c.err);
    return -1;
  }
  return (id * c.Hkv + h) * static_cast<int>(c.page.d) + r;
}

// ------------------------------------------------------ 8-bit conversions
// Four e4m3 codes -> four fp16 (exact: e4m3's range lies inside fp16's).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// Four signed bytes -> four fp16 (exact): with the sign bit flipped a byte is
// the code + 128, and 0x64 above it makes it the fp16 1024 + code + 128.
__device__ __forceinline__ void i8x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
  __half2 x = __hsub2(reinterpret_cast<const __half2&>(a), off);
  __half2 y = __hsub2(reinterpret_cast<const __half2&>(b), off);
  lo = reinterpret_cast<uint32_t&>(x);
  hi = reinterpret_cast<uint32_t&>(y);
}
template <int CT>
__device__ __forceinline__ void code4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (CT == kCacheE4m3) e4m3x4_to_f16(w, lo, hi);
  else i8x4_to_f16(w, lo, hi);
}

// Four values -> four codes, lowest byte first; inv = 1 / scale.
template <int CT>
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d, float inv) {
  if constexpr (CT == kCacheE4m3) {
    uint32_t r;
    asm("{\n .reg .b16 x, y;\n cvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n"
        " mov.b32 %0, {x, y};\n}\n"
        : "=r"(r)
        : "f"(__fmul_rn(a, inv)), "f"(__fmul_rn(b, inv)), "f"(__fmul_rn(c, inv)), "f"(__fmul_rn(d, inv)));
    return r;
  } else {
    // 1.5 * 2^23 + x * inv in one fma rounds the exact product to an integer
    // (ties to even) in the low bits of the sum: one rounding, not two
    constexpr float kMagic = 12582912.f;
    const uint32_t x = __float_as_uint(__fmaf_rn(a, inv, kMagic)), y = __float_as_uint(__fmaf_rn(b, inv, kMagic));
    const uint32_t z = __float_as_uint(__fmaf_rn(c, inv, kMagic)), w = __float_as_uint(__fmaf_rn(d, inv, kMagic));
    return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
  }
}
template <int CT>
constexpr float kQmax = CT == kCacheE4m3 ? 448.f : 127.f;

// ---------------------------------------------------------- 16-byte copies
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace ta
