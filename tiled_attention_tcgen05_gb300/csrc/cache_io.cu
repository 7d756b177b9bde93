// Writing to, reading from and compacting a paged key/value cache.
//
// All three are bound by memory traffic (or, for a token a sequence, by
// latency).  Rows are spread over groups of lanes, 8 or 16 elements a lane: a
// lane's accesses are 16 bytes and a warp's cover whole 128-byte lines; consecutive groups take consecutive tokens of one head,
// which lie side by side in a page.
#include "cache.cuh"
#include "launch.h"

namespace ta {

__device__ __forceinline__ uint4 ldg_stream(const void* p) { return __ldcs(static_cast<const uint4*>(p)); }

// Largest magnitudes of two packed pairs, NaN kept.
template <typename T>
__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b) {
  if constexpr (DT<T>::bf16) {
    __nv_bfloat162 r = __hmax2_nan(__habs2(reinterpret_cast<const __nv_bfloat162&>(a)),
                                   __habs2(reinterpret_cast<const __nv_bfloat162&>(b)));
    return reinterpret_cast<uint32_t&>(r);
  } else {
    __half2 r = __hmax2_nan(__habs2(reinterpret_cast<const __half2&>(a)), __habs2(reinterpret_cast<const __half2&>(b)));
    return reinterpret_cast<uint32_t&>(r);
  }
}

// One lane's 16 elements of a row -> codes; the row's G lanes (a power of two,
// aligned) must all call it.  Writes the scale from the group's first lane.
template <typename T, int CT, int G>
__device__ __forceinline__ uint4 quantise16(const uint4 (&u)[2], float* scale_out, bool write) {
  const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
  uint32_t top = absmax2<T>(absmax2<T>(absmax2<T>(w[0], w[1]), absmax2<T>(w[2], w[3])),
                            absmax2<T>(absmax2<T>(w[4], w[5]), absmax2<T>(w[6], w[7])));
#pragma unroll
  for (int s = G / 2; s > 0; s >>= 1) top = absmax2<T>(top, __shfl_xor_sync(0xffffffffu, top, s));
  top = absmax2<T>(top, __byte_perm(top, top, 0x1032));
  const float amax = static_cast<float>(reinterpret_cast<const T*>(&top)[0]);
  const bool finite = amax < INFINITY;  // false for NaN too
  const float scale = fmaxf(__fdiv_rn(amax, kQmax<CT>), kMinScale);
  const float inv = __frcp_rn(scale);
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const T* h = reinterpret_cast<const T*>(&w[2 * i]);
    r[i] = code4<CT>(static_cast<float>(h[0]), static_cast<float>(h[1]), static_cast<float>(h[2]),
                     static_cast<float>(h[3]), inv);
    if (!finite) r[i] = 0u;
  }
  if (write) *scale_out = finite ? scale : __uint_as_float(0x7fc00000u);
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// cache_append.  Row i of B * Hkv * T is (b, h, t), t fastest.  8-bit caches: 16
// elements a lane, so that a row's maximum, division and reciprocal are
// shared by twice as many (with 8 the instructions, not the memory, set the
// time of a prompt's rows).
template <typename T, int CT, int D>
__global__ void __launch_bounds__(256) append_kernel(CacheArgs c, CacheAppendArgs a) {
  constexpr int E = CT == kCache16 ? 8 : 16;  // elements per lane
  constexpr int G = D / E;
  constexpr int U = 2;  // rows of K and of V in flight per lane
  const int g = threadIdx.x % G;
  const int rpb = 256 / G;
  const int base = blockIdx.x * (rpb * U) + threadIdx.x / G;
  int row[U];
  uint4 xk[U][E / 8], xv[U][E / 8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = base + u * rpb;
    row[u] = -1;
#pragma unroll
    for (int e = 0; e < E / 8; ++e) xk[u][e] = xv[u][e] = make_uint4(0u, 0u, 0u, 0u);
    if (i < a.rows) {
      const int bh = static_cast<int>(a.t_div.div(i)), t = i - bh * c.T;
      const int b = static_cast<int>(a.h_div.div(bh)), h = bh - b * c.Hkv;
      const SeqLens s = cache_lens(c, b);
      if (t < s.q) {
        const T* pk = static_cast<const T*>(a.k) + b * a.ks[0] + h * a.ks[1] + t * a.ks[2] + g * E;
        const T* pv = static_cast<const T*>(a.v) + b * a.vs[0] + h * a.vs[1] + t * a.vs[2] + g * E;
#pragma unroll
        for (int e = 0; e < E / 8; ++e) {
          xk[u][e] = ldg_stream(pk + 8 * e);
          xv[u][e] = ldg_stream(pv + 8 * e);
        }
        int r;
        const int id = cache_page_id(c, b, s.kv - s.q + t, &r);
        row[u] = cache_row(c, h, id, r);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool act = row[u] >= 0;
    const size_t at = static_cast<size_t>(act ? row[u] : 0);
    if constexpr (CT == kCache16) {
      if (act) {
        *reinterpret_cast<uint4*>(static_cast<T*>(c.k) + at * D + g * 8) = xk[u][0];
        *reinterpret_cast<uint4*>(static_cast<T*>(c.v) + at * D + g * 8) = xv[u][0];
      }
    } else {
      const uint4 yk = quantise16<T, CT, G>(xk[u], c.ks + at, act && g == 0);
      const uint4 yv = quantise16<T, CT, G>(xv[u], c.vs + at, act && g == 0);
      if (act) {
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(c.k) + at * D + g * 16) = yk;
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(c.v) + at * D + g * 16) = yv;
      }
    }
  }
}

// 8 codes x scale -> 8 values rounded once to T.
template <typename T, int CT>
__device__ __forceinline__ uint4 dequantise8(const uint2& w, float scale) {
  constexpr bool BF = DT<T>::bf16;
  uint32_t h[4];
  code4_to_f16<CT>(w.x, h[0], h[1]);
  code4_to_f16<CT>(w.y, h[2], h[3]);
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(reinterpret_cast<const __half2&>(h[i]));
    o[i] = pack2<BF>(f.x * scale, f.y * scale);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// cache_read.  Row i of B * Hkv * N is (b, h, n), n fastest; rows at and
// behind a sequence's end are zeros.
template <typename T, int CT, int D>
__global__ void __launch_bounds__(256) read_kernel(CacheArgs c, CacheReadArgs a) {
  constexpr int G = D / 8;
  constexpr int U = 2;
  const int g = threadIdx.x % G;
  const int rpb = 256 / G;
  const int base = blockIdx.x * (rpb * U) + threadIdx.x / G;
  int row[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = base + u * rpb;
    row[u] = -1;
    if (i < a.rows) {
      const int bh = static_cast<int>(a.n_div.div(i)), n = i - bh * static_cast<int>(a.n_div.d);
      const int b = static_cast<int>(a.h_div.div(bh)), h = bh - b * c.Hkv;
      const int kv = __ldg(c.kv_lens + b);
      if (kv < 0 || kv > c.capacity) {
        cache_error(c.err);
      } else if (n < kv) {
        int r;
        const int id = cache_page_id(c, b, n, &r);
        row[u] = cache_row(c, h, id, r);
      }
    }
  }
  if constexpr (CT == kCache16) {
    uint4 k[U], v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      k[u] = v[u] = make_uint4(0u, 0u, 0u, 0u);
      if (row[u] >= 0) {
        const size_t at = static_cast<size_t>(row[u]) * D + g * 8;
        k[u] = ldg_stream(static_cast<const T*>(c.k) + at);
        v[u] = ldg_stream(static_cast<const T*>(c.v) + at);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = base + u * rpb;
      if (i < a.rows) {
        const size_t at = static_cast<size_t>(i) * D + g * 8;
        *reinterpret_cast<uint4*>(static_cast<T*>(a.k) + at) = k[u];
        *reinterpret_cast<uint4*>(static_cast<T*>(a.v) + at) = v[u];
      }
    }
  } else {
    uint2 k[U], v[U];
    float sk[U], sv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      k[u] = v[u] = make_uint2(0u, 0u);
      sk[u] = sv[u] = 0.f;
      if (row[u] >= 0) {
        const size_t at = static_cast<size_t>(row[u]);
        k[u] = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.k) + at * D + g * 8));
        v[u] = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.v) + at * D + g * 8));
        sk[u] = __ldg(c.ks + at);
        sv[u] = __ldg(c.vs + at);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = base + u * rpb;
      if (i < a.rows) {
        const size_t at = static_cast<size_t>(i) * D + g * 8;
        *reinterpret_cast<uint4*>(static_cast<T*>(a.k) + at) = dequantise8<T, CT>(k[u], sk[u]);
        *reinterpret_cast<uint4*>(static_cast<T*>(a.v) + at) = dequantise8<T, CT>(v[u], sv[u]);
      }
    }
  }
}

// cache_keep: one block per (sequence, head).  keep is ascending, so token i's
// new place never lies behind its old one (keep[i] >= i) and never on the old
// place of a later token: rows move in rounds, each read into registers whole
// before it is written.
template <int RB>  // bytes of a row
__global__ void __launch_bounds__(128) keep_kernel(CacheArgs c, CacheKeepArgs a, bool scaled) {
  constexpr int L = RB / 16;          // lanes per row and tensor
  constexpr int U = 4;                // rows in flight per lane
  constexpr int RPR = 128 / (2 * L);  // rows of K and V per step
  const int b = blockIdx.x / c.Hkv, h = blockIdx.x % c.Hkv;
  const SeqLens s = cache_lens(c, b);
  const int n = __ldg(a.keep_lens + b);
  const int first = s.kv - s.q;
  const int* keep = a.keep + static_cast<long long>(b) * c.T;
  // the list must be ascending inside the draft
  bool bad = false;
  if (n < 0 || n > s.q) {
    bad = true;
  } else {
    for (int i = threadIdx.x; i < n; i += 128) {
      const int j = __ldg(keep + i);
      const int before = i ? __ldg(keep + i - 1) : -1;
      if (j <= before || j >= s.q) bad = true;
    }
  }
  bad = __syncthreads_or(bad);
  if (bad) cache_error(c.err);
  if (h == 0 && threadIdx.x == 0) a.new_lens[b] = bad ? first : first + n;
  if (bad) return;
  const int which = (threadIdx.x / L) & 1;  // K or V
  const int lane = threadIdx.x % L, sub = threadIdx.x / (2 * L);
  char* const x = static_cast<char*>(which ? c.v : c.k);
  float* const xs = which ? c.vs : c.ks;
  for (int i0 = 0; i0 < n; i0 += RPR * U) {
    uint4 d[U];
    float ds[U];
    int to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * RPR + sub;
      to[u] = -1;
      if (i < n) {
        const int j = __ldg(keep + i);
        if (j != i) {
          int r;
          int id = cache_page_id(c, b, first + j, &r);
          const int src = cache_row(c, h, id, r);
          id = cache_page_id(c, b, first + i, &r);
          to[u] = cache_row(c, h, id, r);
          if (src < 0) to[u] = -1;
          if (to[u] >= 0) {
            d[u] = *reinterpret_cast<const uint4*>(x + static_cast<size_t>(src) * RB + lane * 16);
            if (scaled && lane == 0) ds[u] = xs[src];
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (to[u] >= 0) {
        *reinterpret_cast<uint4*>(x + static_cast<size_t>(to[u]) * RB + lane * 16) = d[u];
        if (scaled && lane == 0) xs[to[u]] = ds[u];
      }
    }
    __syncthreads();
  }
}

template <typename T, int CT, int D>
static cudaError_t append_t(const CacheArgs& c, const CacheAppendArgs& a, cudaStream_t s) {
  constexpr int rows = 2 * (256 / (D / (CT == kCache16 ? 8 : 16)));
  append_kernel<T, CT, D><<<(a.rows + rows - 1) / rows, 256, 0, s>>>(c, a);
  return cudaGetLastError();
}
template <typename T, int CT, int D>
static cudaError_t read_t(const CacheArgs& c, const CacheReadArgs& a, cudaStream_t s) {
  constexpr int rows = 2 * (256 / (D / 8));
  read_kernel<T, CT, D><<<(a.rows + rows - 1) / rows, 256, 0, s>>>(c, a);
  return cudaGetLastError();
}

#define TA_CACHE_DISPATCH(FN, ARGS)                                          \
  template <typename T, int CT>                                              \
  static cudaError_t FN##_d(int D, const CacheArgs& c, const ARGS& a, cudaStream_t s) { \
    switch (D) {                                                             \
      case 16: return FN##_t<T, CT, 16>(c, a, s);                            \
      case 32: return FN##_t<T, CT, 32>(c, a, s);                            \
      case 64: return FN##_t<T, CT, 64>(c, a, s);                            \
      case 128: return FN##_t<T, CT, 128>(c, a, s);                          \
      default: return cudaErrorInvalidValue;                                 \
    }                                                                        \
  }                                                                          \
  template <typename T>                                                      \
  static cudaError_t FN##_c(int ct, int D, const CacheArgs& c, const ARGS& a, cudaStream_t s) { \
    if (ct == kCache16) return FN##_d<T, kCache16>(D, c, a, s);              \
    if (ct == kCacheE4m3) return FN##_d<T, kCacheE4m3>(D, c, a, s);          \
    return FN##_d<T, kCacheI8>(D, c, a, s);                                  \
  }
TA_CACHE_DISPATCH(append, CacheAppendArgs)
TA_CACHE_DISPATCH(read, CacheReadArgs)
#undef TA_CACHE_DISPATCH

cudaError_t launch_cache_append(bool bf16, int ct, int D, const CacheArgs& c, const CacheAppendArgs& a,
                                cudaStream_t s) {
  return bf16 ? append_c<__nv_bfloat16>(ct, D, c, a, s) : append_c<__half>(ct, D, c, a, s);
}

cudaError_t launch_cache_read(bool bf16, int ct, int D, const CacheArgs& c, const CacheReadArgs& a, cudaStream_t s) {
  return bf16 ? read_c<__nv_bfloat16>(ct, D, c, a, s) : read_c<__half>(ct, D, c, a, s);
}

cudaError_t launch_cache_keep(int ct, int D, const CacheArgs& c, const CacheKeepArgs& a, cudaStream_t s) {
  const int rb = D * (ct == kCache16 ? 2 : 1);
  const int blocks = c.B * c.Hkv;
  const bool scaled = ct != kCache16;
  switch (rb) {
    case 16: keep_kernel<16><<<blocks, 128, 0, s>>>(c, a, scaled); break;
    case 32: keep_kernel<32><<<blocks, 128, 0, s>>>(c, a, scaled); break;
    case 64: keep_kernel<64><<<blocks, 128, 0, s>>>(c, a, scaled); break;
    case 128: keep_kernel<128><<<blocks, 128, 0, s>>>(c, a, scaled); break;
    case 256: keep_kernel<256><<<blocks, 128, 0, s>>>(c, a, scaled); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace ta

TA_GUARD_ACCESSOR(cache_io)
