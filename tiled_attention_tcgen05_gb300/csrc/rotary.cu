// Rotary positions of queries and keys, alone, behind a norm of each head's
// row, and on the way into a paged cache.
//
//   y_i = scale (x_i cos a_p - x_j sin a_p),  y_j = scale (x_j cos a_p + x_i sin a_p)
//
// for the pairs (i, j) of the first `rot` elements of a row: (p, p + rot / 2),
// or (2p, 2p + 1) interleaved; the rest of the row passes through.  With the norm, x = u r w
// elementwise, r = 1 / sqrt(mean u^2 + eps).  The backward of the rotation is the
// rotation by -a; of the norm, with g the gradient rotated back and h = u r,
//   du = r (g w - h mean(g w h)),   dw = sum over rows of g h.
//
// Angles.  a = position * f in fp32 loses 2^-24 of a (0.06 at position 10^6); here f is
// a fraction of a turn in 64-bit fixed point, so that the product modulo 2^64 is
// the exact fraction of the last turn at any position, and only its 32 upper
// bits are turned into a float for sinpi and cospi.
//
// Bound by memory: a row is read once and written once (backward of the norm:
// two reads).  A warp takes one token's rows (or a slice of them where tokens are
// few), D / 8 lanes a row with 16 bytes each, and keeps the token's angles times
// the norm's weights in registers for all of its heads.
#include "launch.h"
#include "pdl.cuh"
#include "rotary.cuh"

namespace ta {

namespace {

constexpr int kWarps = 8;
constexpr int kMaxPairs = 64;

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const T* h = reinterpret_cast<const T*>(&u);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = static_cast<float>(h[e]);
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  constexpr bool BF = DT<T>::bf16;
  return make_uint4(pack2<BF>(f[0], f[1]), pack2<BF>(f[2], f[3]), pack2<BF>(f[4], f[5]), pack2<BF>(f[6], f[7]));
}

template <int L>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int s = L / 2; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// How the lane that holds elements [8 l, 8 l + 8) of a row finds their partners.
struct Place {
  int l;
  bool swap;     // interleaved: the partner is the neighbour
  bool reload;   // halves that are no multiple of 8: partners are read again
  int from;      // lane that holds the partners (halves of whole lanes)
};

// The partners of the lane's elements, 0 beyond the rotated part (whose
// factor is 0: a pass-through element's infinity must not meet it).  Warp-collective.
template <typename T>
__device__ __forceinline__ void partners(const Place& w, int rot, const uint4& raw, const float (&f)[8], const T* row,
                                         bool act, float (&xp)[8]) {
  if (w.swap) {
#pragma unroll
    for (int e = 0; e < 8; ++e) xp[e] = 8 * w.l + e < rot ? f[e ^ 1] : 0.f;
  } else if (!w.reload) {
    uint4 o;
    o.x = __shfl_sync(0xffffffffu, raw.x, w.from);
    o.y = __shfl_sync(0xffffffffu, raw.y, w.from);
    o.z = __shfl_sync(0xffffffffu, raw.z, w.from);
    o.w = __shfl_sync(0xffffffffu, raw.w, w.from);
    if (8 * w.l >= rot) o = make_uint4(0u, 0u, 0u, 0u);
    unpack8<T>(o, xp);
  } else {
    const int half = rot >> 1;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = 8 * w.l + e;
      xp[e] = (act && i < rot) ? static_cast<float>(row[i < half ? i + half : i - half]) : 0.f;
    }
    __syncwarp();  // the row may be written over from here on
  }
}

// Factors of an element and of its partner: y = x ca + xp cb.
struct Coef {
  float ca[8], cb[8];
};

// w: the norm's weights (null: ones).  back: of the transposed rotation (weights not included).
template <typename T>
__device__ __forceinline__ void coefs(const RotArgs& a, const Place& w, const float* cs, const float* sn, const void* wt,
                                      Coef& c) {
  auto weight = [&](int i) {
    return !wt ? 1.f : a.w32 ? __ldg(static_cast<const float*>(wt) + i) : static_cast<float>(static_cast<const T*>(wt)[i]);
  };
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = 8 * w.l + e;
    c.ca[e] = weight(i);
    c.cb[e] = 0.f;
    if (i < a.rot) {
      const bool first = a.interleaved ? !(i & 1) : i < a.pairs;
      const int p = a.interleaved ? i >> 1 : first ? i : i - a.pairs;
      const int j = a.interleaved ? i ^ 1 : first ? i + a.pairs : i - a.pairs;
      c.ca[e] *= cs[p];
      c.cb[e] = (first ? -sn[p] : sn[p]) * weight(j);
    }
  }
}

// 1 / sqrt(mean f^2 + eps) over the row; where the squares pass fp32's range
// f and xp are scaled by *down first (the result is that of the scaled row).
// Warp-collective.
template <int D>
__device__ __forceinline__ float row_norm(float (&f)[8], float (&xp)[8], float eps, float* down) {
  constexpr int L = D / 8;
  auto squares = [&] {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
    return row_sum<L>(ss);
  };
  float ss = squares();
  const bool big = !(ss < INFINITY);
  float tiny = 1.f;
  if (__any_sync(0xffffffffu, big)) {
    tiny = big ? 5.421010862427522e-20f : 1.f;  // 2^-64
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[e] *= tiny;
      xp[e] *= tiny;
    }
    ss = squares();
  }
  *down = tiny;
  return rsqrtf(fmaf(ss, 1.f / D, eps * tiny * tiny));
}

// A row's eight fp32 elements a lane -> codes of a cache type; returns the scale.
template <int CT, int L>
__device__ __forceinline__ uint2 quantise8(const float (&y)[8], float* scale_out) {
  uint32_t top = 0;  // magnitudes as integers: a NaN is larger than infinity
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(y[e]) & 0x7fffffffu);
#pragma unroll
  for (int s = L / 2; s > 0; s >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, s));
  const bool finite = top < 0x7f800000u;
  const float scale = fmaxf(__fdiv_rn(__uint_as_float(top), kQmax<CT>), kMinScale);
  const float inv = __frcp_rn(scale);
  uint2 r = make_uint2(code4<CT>(y[0], y[1], y[2], y[3], inv), code4<CT>(y[4], y[5], y[6], y[7], inv));
  if (!finite) r = make_uint2(0u, 0u);
  *scale_out = finite ? scale : __uint_as_float(0x7fc00000u);
  return r;
}

// cos and sin (times scale, and sign) of the token's pairs into the warp's
// shared arrays.
__device__ __forceinline__ void token_angles(const RotArgs& a, int pos, int lane, float* cs, float* sn) {
  __syncwarp();  // the token before it has been read
  for (int p = lane; p < a.pairs; p += 32) {
    const uint64_t ph = static_cast<uint64_t>(static_cast<int64_t>(pos)) * __ldg(a.turns + p);
    const float x = static_cast<float>(static_cast<int32_t>(ph >> 32)) * 4.656612873077393e-10f;  // half turns, [-1, 1)
    float s, c;
    sincospif(x, &s, &c);
    cs[p] = c * a.scale;
    sn[p] = s * a.scale * a.sign;
  }
  __syncwarp();
}

template <int D>
__device__ __forceinline__ Place place_of(const RotArgs& a, int lane) {
  constexpr int L = D / 8;
  Place w;
  w.l = lane % L;
  w.swap = a.interleaved != 0;
  w.reload = !w.swap && (a.pairs & 7) != 0;
  const int step = a.pairs >> 3;
  w.from = lane;
  if (!w.swap && !w.reload && 8 * w.l < a.rot) w.from = lane + (8 * w.l < a.pairs ? step : -step);
  return w;
}

}  // namespace

// kRotPlain, kRotNorm and kRotAppend (CT: the cache's type).
template <typename T, int D, int MODE, int CT>
__global__ void __launch_bounds__(kWarps * 32) rotary_kernel(const RotArgs a, const CacheArgs c) {
  constexpr int L = D / 8, RPW = 32 / L;  // lanes a row, rows a warp holds at once
  constexpr int U = 4;                    // such groups of rows in flight
  __shared__ float angles[kWarps][2][kMaxPairs];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x * kWarps + warp;
  if (unit >= a.units) return;
  const int token = static_cast<int>(a.slice_div.div(unit)), slice = unit - token * static_cast<int>(a.slice_div.d);
  const int b = static_cast<int>(a.t_div.div(token)), t = token - b * a.T;
  float *cs = angles[warp][0], *sn = angles[warp][1];
  token_angles(a, __ldg(a.pos + b * a.pos_b + t * a.pos_t), lane, cs, sn);
  const Place w = place_of<D>(a, lane);
  const int sub = lane / L;
  const int r0 = slice * a.slice_rows, r1 = r0 + a.slice_rows;  // rows of the token: q, k (, v) heads

  long long slot_row = -1;  // append: row of head 0 in the cache
  if constexpr (MODE == kRotAppend) {
    const int slot = __ldg(a.slots + token);
    if (slot >= 0) {
      const uint32_t id = c.page.div(slot);
      if (id < static_cast<uint32_t>(c.num_pages))
        slot_row = static_cast<long long>(id) * c.Hkv * c.page.d + (slot - id * c.page.d);
      else if (lane == 0)
        cache_error(c.err);
    }
  }

  // one tensor's heads [n0, n1); kind 0: q, 1: k, 2: v
  auto rows_of = [&](const RotRows& in, const RotRows& out, const void* wt, int kind, int n0, int n1) {
    if (n0 >= n1) return;
    const bool cached = MODE == kRotAppend && kind > 0;
    if (cached && slot_row < 0) return;
    Coef co;
    if (kind < 2) coefs<T>(a, w, cs, sn, wt, co);
    const T* src = static_cast<const T*>(in.p) + b * in.sb + t * in.st;
    T* dst = static_cast<T*>(out.p) + b * out.sb + t * out.st;
    for (int h0 = n0; h0 < n1; h0 += RPW * U) {
      uint4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * RPW + sub;
        raw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (h < n1) raw[u] = __ldcs(reinterpret_cast<const uint4*>(src + h * in.sh + 8 * w.l));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h0 + u * RPW >= n1) break;
        const int h = h0 + u * RPW + sub;
        const bool act = h < n1;
        float f[8], y[8];
        unpack8<T>(raw[u], f);
        if (kind < 2) {
          float xp[8];
          partners<T>(w, a.rot, raw[u], f, src + h * in.sh, act, xp);
          float r = 1.f, down;
          if (MODE == kRotNorm || (MODE == kRotAppend && a.wq)) r = row_norm<D>(f, xp, a.eps, &down);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = r * fmaf(f[e], co.ca[e], xp[e] * co.cb[e]);
        }
        if (!cached) {
          if (act) *reinterpret_cast<uint4*>(dst + h * out.sh + 8 * w.l) = pack8<T>(y);
          continue;
        }
        if constexpr (MODE == kRotAppend) {
          if (kind == 2) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = f[e];
          }
          const long long row = slot_row + static_cast<long long>(h) * c.page.d;
          if constexpr (CT == kCache16) {
            const uint4 o = kind == 2 ? raw[u] : pack8<T>(y);
            if (act) *reinterpret_cast<uint4*>(static_cast<T*>(kind == 2 ? c.v : c.k) + row * D + 8 * w.l) = o;
          } else {
            float scale;
            const uint2 o = quantise8<CT, L>(y, &scale);
            if (act) {
              *reinterpret_cast<uint2*>(static_cast<uint8_t*>(kind == 2 ? c.v : c.k) + row * D + 8 * w.l) = o;
              if (w.l == 0) (kind == 2 ? c.vs : c.ks)[row] = scale;
            }
          }
        }
      }
    }
  };
  rows_of(a.q, a.qo, a.wq, 0, min(r0, a.Hq), min(r1, a.Hq));
  auto part = [&](int r, int first) { return min(max(r - first, 0), a.Hkv); };
  rows_of(a.k, a.ko, a.wk, 1, part(r0, a.Hq), part(r1, a.Hq));
  if constexpr (MODE == kRotAppend) rows_of(a.v, a.ko, nullptr, 2, part(r0, a.Hq + a.Hkv), part(r1, a.Hq + a.Hkv));
}

// Backward of the norm and the rotation.  A block sums its rows' part of dw in
// registers, then over its lanes in a fixed order; the join adds the blocks'.
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) rotary_norm_bwd_kernel(const RotArgs a) {
  constexpr int L = D / 8, RPW = 32 / L;
  constexpr int U = 2;
  __shared__ float angles[kWarps][2][kMaxPairs];
  __shared__ float sums[kWarps][2][D];
  pdl_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Place w = place_of<D>(a, lane);
  const int sub = lane / L;
  float *cs = angles[warp][0], *sn = angles[warp][1];
  float dw[2][8] = {};
  for (int unit = blockIdx.x * kWarps + warp; unit < a.units; unit += gridDim.x * kWarps) {
    const int token = static_cast<int>(a.slice_div.div(unit)), slice = unit - token * static_cast<int>(a.slice_div.d);
    const int b = static_cast<int>(a.t_div.div(token)), t = token - b * a.T;
    token_angles(a, __ldg(a.pos + b * a.pos_b + t * a.pos_t), lane, cs, sn);
    const int r0 = slice * a.slice_rows, r1 = r0 + a.slice_rows;
    Coef co;
    coefs<T>(a, w, cs, sn, nullptr, co);  // of the negative angle: the same for queries and keys
    auto rows_of = [&](const RotRows& in, const RotRows& grad, const RotRows& out, const void* wt, float (&acc)[8], int n0,
                       int n1) {
      if (n0 >= n1) return;
      float wv[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        wv[e] = a.w32 ? __ldg(static_cast<const float*>(wt) + 8 * w.l + e)
                      : static_cast<float>(static_cast<const T*>(wt)[8 * w.l + e]);
      const T* px = static_cast<const T*>(in.p) + b * in.sb + t * in.st;
      const T* pg = static_cast<const T*>(grad.p) + b * grad.sb + t * grad.st;
      T* po = static_cast<T*>(out.p) + b * out.sb + t * out.st;
      for (int h0 = n0; h0 < n1; h0 += RPW * U) {
        uint4 rx[U], rg[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = h0 + u * RPW + sub;
          rx[u] = rg[u] = make_uint4(0u, 0u, 0u, 0u);
          if (h < n1) {
            rx[u] = __ldcs(reinterpret_cast<const uint4*>(px + h * in.sh + 8 * w.l));
            rg[u] = __ldcs(reinterpret_cast<const uint4*>(pg + h * grad.sh + 8 * w.l));
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (h0 + u * RPW >= n1) break;
          const int h = h0 + u * RPW + sub;
          const bool act = h < n1;
          float f[8], g[8], gp[8];
          unpack8<T>(rx[u], f);
          unpack8<T>(rg[u], g);
          partners<T>(w, a.rot, rg[u], g, pg + h * grad.sh, act, gp);
          float none[8] = {}, down;
          const float r = row_norm<D>(f, none, a.eps, &down);
          float dot = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            g[e] = fmaf(g[e], co.ca[e], gp[e] * co.cb[e]);
            f[e] *= r;  // h = u r
            if (act) acc[e] = fmaf(g[e], f[e], acc[e]);
            g[e] *= wv[e];
            dot = fmaf(g[e], f[e], dot);
          }
          dot = row_sum<L>(dot) * (1.f / D);
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = r * down * fmaf(-f[e], dot, g[e]);
          if (act) *reinterpret_cast<uint4*>(po + h * out.sh + 8 * w.l) = pack8<T>(g);
        }
      }
    };
    rows_of(a.q, a.dq, a.qo, a.wq, dw[0], min(r0, a.Hq), min(r1, a.Hq));
    auto part = [&](int r) { return min(max(r - a.Hq, 0), a.Hkv); };
    rows_of(a.k, a.dk, a.ko, a.wk, dw[1], part(r0), part(r1));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float v = dw[i][e];
#pragma unroll
      for (int s = 16; s >= L; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
      if (sub == 0) sums[warp][i][8 * w.l + e] = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kWarps * 32) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) v += sums[k][i / D][i % D];
    a.part[static_cast<size_t>(blockIdx.x) * 2 * D + i] = v;
  }
}

// dw[i] = sum of the blocks' partial sums, each of a block's 8 warps over every
// eighth block, in a fixed order.
template <int D>
__global__ void __launch_bounds__(256) rotary_dw_kernel(const float* part, int blocks, float* dwq, float* dwk) {
  __shared__ float sums[8][32];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), warp = threadIdx.x >> 5;
  pdl_wait();
  float v[4] = {};
  int i = warp;
  for (; i + 24 < blocks; i += 32)
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] += part[static_cast<size_t>(i + 8 * u) * 2 * D + col];
  for (; i < blocks; i += 8) v[0] += part[static_cast<size_t>(i) * 2 * D + col];
  sums[warp][threadIdx.x & 31] = (v[0] + v[1]) + (v[2] + v[3]);
  __syncthreads();
  if (warp == 0) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) t += sums[k][threadIdx.x];
    float* out = col < D ? dwq : dwk;
    if (out) out[col % D] = t;
  }
}

template <typename T, int D>
static cudaError_t run_rotary(int mode, int ct, const RotArgs& a, const CacheArgs& c, cudaStream_t s) {
  const unsigned blocks = static_cast<unsigned>((static_cast<long long>(a.units) + kWarps - 1) / kWarps);
  constexpr int threads = kWarps * 32;
  if (mode == kRotPlain) {
    rotary_kernel<T, D, kRotPlain, kCache16><<<blocks, threads, 0, s>>>(a, c);
  } else if (mode == kRotNorm) {
    rotary_kernel<T, D, kRotNorm, kCache16><<<blocks, threads, 0, s>>>(a, c);
  } else if (mode == kRotAppend) {
    if (ct == kCache16) rotary_kernel<T, D, kRotAppend, kCache16><<<blocks, threads, 0, s>>>(a, c);
    else if (ct == kCacheE4m3) rotary_kernel<T, D, kRotAppend, kCacheE4m3><<<blocks, threads, 0, s>>>(a, c);
    else rotary_kernel<T, D, kRotAppend, kCacheI8><<<blocks, threads, 0, s>>>(a, c);
  } else {
    rotary_norm_bwd_kernel<T, D><<<a.blocks, threads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return pdl_launch(rotary_dw_kernel<D>, dim3(2 * D / 32), 256, 0, s, static_cast<const float*>(a.part), a.blocks,
                      a.dwq, a.dwk);
  }
  return cudaGetLastError();
}

template <typename T>
static cudaError_t rotary_d(int mode, int ct, int D, const RotArgs& a, const CacheArgs& c, cudaStream_t s) {
  switch (D) {
    case 16: return run_rotary<T, 16>(mode, ct, a, c, s);
    case 32: return run_rotary<T, 32>(mode, ct, a, c, s);
    case 64: return run_rotary<T, 64>(mode, ct, a, c, s);
    case 128: return run_rotary<T, 128>(mode, ct, a, c, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_rotary(int mode, bool bf16, int ct, int D, const RotArgs& a, const CacheArgs& c, cudaStream_t s) {
  return bf16 ? rotary_d<__nv_bfloat16>(mode, ct, D, a, c, s) : rotary_d<__half>(mode, ct, D, a, c, s);
}

}  // namespace ta

TA_GUARD_ACCESSOR(rotary)
