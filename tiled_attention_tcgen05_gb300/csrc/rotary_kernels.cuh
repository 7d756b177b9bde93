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
// few), D / 16 lanes a row.  A lane holds two 16-byte chunks: where the halves of
// the rotated part are whole chunks, one of each half, so that both elements of
// its pairs are its own; else chunks l and l + D / 16, partners found in the chunk
// (interleaved) or read again.  The token's cosines and sines, times the norm's
// weights, stay in registers for all of its heads.  All of a slice's rows are copied to
// shared memory (cp.async) before the warp works on the first: loads that wait in registers
// were too few to fill the memory's latency.  Replayed calls:
//   rotation of 8192 tokens, 32 / 8 heads of 128, bf16: 32 us, 5.3 TB/s (16384: 52 us, 6.4 TB/s);
//   norm and rotation of 16383 tokens of these: 64 us, 5.3 TB/s, and of 64: 2.5 us in a row of calls;
//   its backward for 8192 tokens, 32 / 4 heads of 64, fp16: 31 us, 3.7 TB/s (issue: half of all slots);
//   8191 tokens of the first kind into a cache: 41 us, 4.9 TB/s.
// A plain copy reaches 6.8 TB/s; at these sizes launch, first loads and last stores are some 5 us.
#pragma once
#include <atomic>
#include <type_traits>

#include "launch.h"
#include "pdl.cuh"
#include "rotary.cuh"

namespace ta {

namespace {

constexpr int kWarps = 8;
constexpr int kMaxPairs = 64;

// How a lane's elements find their partners.
enum RotPath : int {
  kHalves = 0,   // the whole row turns, partner of chunk 0's element e: chunk 1's
  kNeighbours = 1,  // the whole row turns, interleaved
  kAny = 2       // anything else
};

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& u, float2 (&f)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (DT<T>::bf16) f[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
    else f[e] = __half22float2(reinterpret_cast<const __half2&>(w[e]));
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
  constexpr bool BF = DT<T>::bf16;
  return make_uint4(pack2<BF>(f[0].x, f[0].y), pack2<BF>(f[1].x, f[1].y), pack2<BF>(f[2].x, f[2].y),
                    pack2<BF>(f[3].x, f[3].y));
}

template <int L>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int s = L / 2; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// Where a lane's two chunks of a row start, and which path its row takes.
struct Place {
  int at[2];
  int path;
  bool reload;  // kAny: partners are read again
};
template <int D>
__device__ __forceinline__ Place place_of(const RotArgs& a, int lane) {
  constexpr int L = D / 16;
  const int l = lane % L;
  Place w;
  w.at[0] = 8 * l;
  w.at[1] = D / 2 + 8 * l;
  w.reload = false;
  if (a.interleaved) {
    w.path = a.rot == D ? kNeighbours : kAny;
  } else if ((a.pairs & 7) == 0) {
    w.path = a.rot == D ? kHalves : kAny;
    if (8 * l < a.pairs) {
      w.at[1] = a.pairs + 8 * l;
    } else {  // two chunks that pass through
      w.at[0] = a.rot + 16 * (l - a.pairs / 8);
      w.at[1] = w.at[0] + 8;
    }
  } else {
    w.path = kAny;
    w.reload = true;
  }
  return w;
}

// Partners of the lane's elements.  kAny: zeros beyond the rotated part, whose
// factor is 0 (a pass-through element's infinity must not meet it).  Warp-collective.
template <typename T, int PATH>
__device__ __forceinline__ void partners(const RotArgs& a, const Place& w, const float2 (&f)[2][4], const T* row, bool act,
                                         float2 (&xp)[2][4]) {
  if constexpr (PATH == kHalves) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      xp[0][e] = f[1][e];
      xp[1][e] = f[0][e];
    }
  } else if constexpr (PATH == kNeighbours) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) xp[c][e] = make_float2(f[c][e].y, f[c][e].x);
  } else {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = w.at[c] + 2 * e;
        float2 p;
        if (w.reload) {
          auto get = [&](int k) {
            return act && k < a.rot ? static_cast<float>(row[k < a.pairs ? k + a.pairs : k - a.pairs]) : 0.f;
          };
          p = make_float2(get(i), get(i + 1));
        } else {
          p = a.interleaved ? make_float2(f[c][e].y, f[c][e].x) : f[c ^ 1][e];
          if (i >= a.rot) p = make_float2(0.f, 0.f);
        }
        xp[c][e] = p;
      }
    if (w.reload) __syncwarp();  // the row may be written over from here on
  }
}

// Factors of an element and of its partner: y = x ca + xp cb.
struct Coef {
  float2 ca[2][4], cb[2][4];
};
// The norm's weights into shared memory, in fp32 (a block's threads).
template <typename T, int D>
__device__ __forceinline__ void stage_weights(const RotArgs& a, const void* wt, float* out) {
  if (!wt) return;
  for (int i = threadIdx.x; i < D; i += kWarps * 32)
    out[i] = a.w32 ? __ldg(static_cast<const float*>(wt) + i) : static_cast<float>(static_cast<const T*>(wt)[i]);
}
// Weights of the lane's elements (null: ones).
__device__ __forceinline__ void load_weights(const Place& w, const float* wt, float2 (&v)[2][4]) {
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      float4 x = make_float4(1.f, 1.f, 1.f, 1.f);
      if (wt) x = *reinterpret_cast<const float4*>(wt + w.at[c] + 2 * e);
      v[c][e] = make_float2(x.x, x.y);
      v[c][e + 1] = make_float2(x.z, x.w);
    }
}

template <int PATH>
__device__ __forceinline__ void coefs(const RotArgs& a, const Place& w, const float* cs, const float* sn, const float* wt,
                                      Coef& k) {
  float2 v[2][4];
  load_weights(w, wt, v);
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = w.at[c] + 2 * e;
      if constexpr (PATH == kHalves) {
        const int p = w.at[0] + 2 * e;
        const float2 co = *reinterpret_cast<const float2*>(cs + p), si = *reinterpret_cast<const float2*>(sn + p);
        k.ca[c][e] = fmul2(v[c][e], co);
        k.cb[c][e] = fmul2(v[c ^ 1][e], c == 0 ? make_float2(-si.x, -si.y) : si);
      } else if constexpr (PATH == kNeighbours) {
        const float co = cs[i >> 1], si = sn[i >> 1];
        k.ca[c][e] = make_float2(v[c][e].x * co, v[c][e].y * co);
        k.cb[c][e] = make_float2(-v[c][e].y * si, v[c][e].x * si);
      } else {
        auto one = [&](int j, float wj, float& ca, float& cb) {
          ca = wj;
          cb = 0.f;
          if (j >= a.rot) return;
          const bool first = a.interleaved ? !(j & 1) : j < a.pairs;
          const int p = a.interleaved ? j >> 1 : first ? j : j - a.pairs;
          const int o = a.interleaved ? j ^ 1 : first ? j + a.pairs : j - a.pairs;
          const float wo = wt ? wt[o] : 1.f;
          ca = wj * cs[p];
          cb = (first ? -sn[p] : sn[p]) * wo;
        };
        one(i, v[c][e].x, k.ca[c][e].x, k.cb[c][e].x);
        one(i + 1, v[c][e].y, k.ca[c][e].y, k.cb[c][e].y);
      }
    }
}

// r = 1 / sqrt(mean f^2 + eps) of U rows side by side.  Where a row's squares leave
// fp32's range, f is scaled by by[] first, and r is that of the scaled row (true: some row of
// the warp's is).  Squares past it: elements below 2^128 become 2^48 at most, and one past 2^60,
// which such a row has, 2^-20.  Squares below it: where mean and eps together pass 2^-100, what
// fp32 loses of the squares (2^-150 each) is nothing beside them; else elements of 2^-133 to 2^-46 become
// 2^-53 to 2^34, and eps at most 2^60.  Warp-collective.
template <int D, int U>
__device__ __forceinline__ bool row_norm(float2 (&f)[U][2][4], float eps, float (&r)[U], float (&by)[U]) {
  constexpr int L = D / 16;
  float ss[U];
  auto squares = [&] {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s0 = ffma2(f[u][0][e], f[u][0][e], s0);
        s1 = ffma2(f[u][1][e], f[u][1][e], s1);
      }
      s0 = fadd2(s0, s1);
      ss[u] = s0.x + s0.y;
    }
#pragma unroll
    for (int s = L / 2; s > 0; s >>= 1)
#pragma unroll
      for (int u = 0; u < U; ++u) ss[u] += __shfl_xor_sync(0xffffffffu, ss[u], s);
  };
  squares();
  constexpr float LOW = 7.888609052210118e-31f;  // 2^-100
  bool scaled = false;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    r[u] = fmaf(ss[u], 1.f / D, eps);
    by[u] = 1.f;
    // (not in [LOW, infinity): one comparison of the bits of a number that is not negative)
    scaled |= __float_as_uint(r[u]) - __float_as_uint(LOW) >= 0x7f800000u - __float_as_uint(LOW);
  }
  scaled = __any_sync(0xffffffffu, scaled);
  if (scaled) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      by[u] = r[u] < LOW ? 1.2089258196146292e24f : r[u] < INFINITY ? 1.f : 8.271806125530277e-25f;  // 2^80, 2^-80
      const float2 t2 = make_float2(by[u], by[u]);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) f[u][c][e] = fmul2(f[u][c][e], t2);
    }
    squares();
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = fmaf(ss[u], 1.f / D, eps * by[u] * by[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) r[u] = rsqrtf(r[u]);
  return scaled;
}

// A row's sixteen fp32 elements a lane -> codes of a cache type, and the scale.
template <int CT, int L>
__device__ __forceinline__ void quantise16(const float2 (&y)[2][4], uint2 (&r)[2], float* scale_out) {
  uint32_t top = 0;  // magnitudes as integers: a NaN is larger than infinity
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      top = max(top, max(__float_as_uint(y[c][e].x) & 0x7fffffffu, __float_as_uint(y[c][e].y) & 0x7fffffffu));
#pragma unroll
  for (int s = L / 2; s > 0; s >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, s));
  const bool finite = top < 0x7f800000u;
  const float scale = fmaxf(__fdiv_rn(__uint_as_float(top), kQmax<CT>), kMinScale);
  const float inv = __frcp_rn(scale);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    r[c] = make_uint2(code4<CT>(y[c][0].x, y[c][0].y, y[c][1].x, y[c][1].y, inv),
                      code4<CT>(y[c][2].x, y[c][2].y, y[c][3].x, y[c][3].y, inv));
    if (!finite) r[c] = make_uint2(0u, 0u);
  }
  *scale_out = finite ? scale : __uint_as_float(0x7fc00000u);
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

// The lane's chunks of one group of rows (heads h0 + sub below n) to its own 32
// bytes of a stage; rows that are none as zeros.
template <typename T>
__device__ __forceinline__ void fetch_rows(uint32_t stage, const T* src, long long sh, const Place& w, int h, int n) {
  const bool real = h < n;
  const T* row = src + (real ? h : 0) * sh;
#pragma unroll
  for (int c = 0; c < 2; ++c) cp_async16(stage + 512 * c, row + w.at[c], real);
}
__device__ __forceinline__ uint4 staged(const uint8_t* stage, int c) {
  return *reinterpret_cast<const uint4*>(stage + 512 * c);
}
// Until at most n of the lane's newest groups of copies are on their way.
__device__ __forceinline__ void wait_copies(int n) {
  switch (n) {
    case 0: cp_async_wait<0>(); break;
    case 1: cp_async_wait<1>(); break;
    case 2: cp_async_wait<2>(); break;
    case 3: cp_async_wait<3>(); break;
    case 4: cp_async_wait<4>(); break;
    case 5: cp_async_wait<5>(); break;
    case 6: cp_async_wait<6>(); break;
    case 7: cp_async_wait<7>(); break;
    case 8: cp_async_wait<8>(); break;
    case 9: cp_async_wait<9>(); break;
    case 10: cp_async_wait<10>(); break;
    default: cp_async_wait<11>(); break;
  }
}
static_assert(kRotGroups <= 12, "wait_copies counts to eleven");

}  // namespace

// kRotPlain, kRotNorm and kRotAppend (CT: the cache's type).
template <typename T, int D, int MODE, int CT, bool ANY>
__global__ void __launch_bounds__(kWarps * 32, ANY ? 1 : 2) rotary_kernel(const RotArgs a, const CacheArgs c) {
  constexpr int L = D / 16, RPW = 32 / L;  // lanes a row, rows of a group
  extern __shared__ __align__(16) uint8_t stages[];  // [warp][group of the slice][chunk][lane] 16 bytes
  __shared__ __align__(16) float angles[kWarps][2][kMaxPairs];
  __shared__ __align__(16) float weights[2][MODE == kRotPlain ? 1 : D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x * kWarps + warp;
  const bool real = unit < a.units;
  const int token = static_cast<int>(a.slice_div.div(real ? unit : 0));
  const int slice = (real ? unit : 0) - token * static_cast<int>(a.slice_div.d);
  const int b = static_cast<int>(a.t_div.div(token)), t = token - b * a.T;
  const Place w = place_of<D>(a, lane);
  const int sub = lane / L;
  // groups of the token: of the queries, then the keys, then the values
  const int nq = (a.Hq + RPW - 1) / RPW, nk = (a.Hkv + RPW - 1) / RPW;
  const int g0 = slice * a.slice_groups;
  const int g1 = real ? min(g0 + a.slice_groups, nq + nk * (MODE == kRotAppend ? 2 : 1)) : g0;
  uint8_t* mine = stages + warp * a.slice_groups * 1024 + lane * 16;
  const uint32_t mine_s = smem_u32(mine);
  auto rows = [&](const RotRows& x) { return static_cast<T*>(x.p) + b * x.sb + t * x.st; };
  for (int g = g0; g < g1; ++g) {
    const uint32_t to = mine_s + (g - g0) * 1024;
    if (g < nq) fetch_rows<T>(to, rows(a.q), a.q.sh, w, g * RPW + sub, a.Hq);
    else if (g < nq + nk) fetch_rows<T>(to, rows(a.k), a.k.sh, w, (g - nq) * RPW + sub, a.Hkv);
    else fetch_rows<T>(to, rows(a.v), a.v.sh, w, (g - nq - nk) * RPW + sub, a.Hkv);
    cp_async_commit();
  }
  if constexpr (MODE != kRotPlain) {
    stage_weights<T, D>(a, a.wq, weights[0]);
    stage_weights<T, D>(a, a.wk, weights[1]);
    __syncthreads();
  }
  if (!real) return;
  float *cs = angles[warp][0], *sn = angles[warp][1];
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
  token_angles(a, __ldg(a.pos + b * a.pos_b + t * a.pos_t), lane, cs, sn);

  // a row's elements y to the cache (v: 1, k: 0)
  auto to_cache = [&](int v, int h, bool act, const float2 (&y)[2][4]) {
    const long long row = slot_row + static_cast<long long>(h) * c.page.d;
    if constexpr (CT == kCache16) {
      T* p = static_cast<T*>(v ? c.v : c.k) + row * D;
      if (act) {
#pragma unroll
        for (int i = 0; i < 2; ++i) *reinterpret_cast<uint4*>(p + w.at[i]) = pack8<T>(y[i]);
      }
    } else {
      uint2 o[2];
      float scale;
      quantise16<CT, L>(y, o, &scale);
      uint8_t* p = static_cast<uint8_t*>(v ? c.v : c.k) + row * D;
      if (act) {
#pragma unroll
        for (int i = 0; i < 2; ++i) *reinterpret_cast<uint2*>(p + w.at[i]) = o[i];
        if (lane % L == 0) (v ? c.vs : c.ks)[row] = scale;
      }
    }
  };
  // groups [n0, n1) of the queries (key 0; from group `base` on) or the keys (1)
  auto turn = [&](auto path_tag, int key, const RotRows& in, const RotRows& out, int heads, int base, int n0, int n1) {
    constexpr int PATH = decltype(path_tag)::value;
    const bool cached = MODE == kRotAppend && key;
    if (n0 >= n1 || (cached && slot_row < 0)) return;
    const bool norm = MODE == kRotNorm || (MODE == kRotAppend && (key ? a.wk : a.wq));
    T* dst = rows(out);
    Coef k;
    coefs<PATH>(a, w, cs, sn, norm ? weights[key] : nullptr, k);
    auto some = [&](auto count, int g) {  // groups g .. g + U - 1 side by side
      constexpr int U = decltype(count)::value;
      wait_copies(g1 - U - g);
      float2 f[U][2][4];
      float r[U], by[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint8_t* from = mine + (g + u - g0) * 1024;
        unpack8<T>(staged(from, 0), f[u][0]);
        unpack8<T>(staged(from, 1), f[u][1]);
        r[u] = by[u] = 1.f;
      }
      if (norm) row_norm<D, U>(f, a.eps, r, by);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = (g + u - base) * RPW + sub;
        const bool act = h < heads;
        float2 xp[2][4], y[2][4];
        partners<T, PATH>(a, w, f[u], rows(in) + h * in.sh, act, xp);
        if (norm && PATH == kAny && w.reload) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) xp[i][e] = fmul2(xp[i][e], make_float2(by[u], by[u]));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[i][e] = ffma2(f[u][i][e], k.ca[i][e], fmul2(xp[i][e], k.cb[i][e]));
            if (norm) y[i][e] = fmul2(y[i][e], make_float2(r[u], r[u]));
          }
        if (cached) {
          to_cache(0, h, act, y);
        } else if (act) {
          *reinterpret_cast<uint4*>(dst + h * out.sh + w.at[0]) = pack8<T>(y[0]);
          *reinterpret_cast<uint4*>(dst + h * out.sh + w.at[1]) = pack8<T>(y[1]);
        }
      }
    };
    int g = n0;
    if constexpr (!ANY) {
#pragma unroll 1
      for (; g + 1 < n1; g += 2) some(std::integral_constant<int, 2>{}, g);
    }
#pragma unroll 1
    for (; g < n1; ++g) some(std::integral_constant<int, 1>{}, g);
  };
  auto both = [&](auto path_tag) {
    turn(path_tag, 0, a.q, a.qo, a.Hq, 0, g0, min(g1, nq));
    turn(path_tag, 1, a.k, a.ko, a.Hkv, nq, max(g0, nq), min(g1, nq + nk));
  };
  if constexpr (ANY) both(std::integral_constant<int, kAny>{});
  else if (w.path == kHalves) both(std::integral_constant<int, kHalves>{});
  else both(std::integral_constant<int, kNeighbours>{});
  if constexpr (MODE == kRotAppend) {
    if (slot_row >= 0) {
#pragma unroll 1
      for (int g = max(g0, nq + nk); g < g1; ++g) {
        wait_copies(g1 - 1 - g);
        const uint8_t* from = mine + (g - g0) * 1024;
        const int h = (g - nq - nk) * RPW + sub;
        if constexpr (CT == kCache16) {  // bits as they are
          T* p = static_cast<T*>(c.v) + (slot_row + static_cast<long long>(h) * c.page.d) * D;
          if (h < a.Hkv) {
#pragma unroll
            for (int i = 0; i < 2; ++i) *reinterpret_cast<uint4*>(p + w.at[i]) = staged(from, i);
          }
        } else {
          float2 f[2][4];
          unpack8<T>(staged(from, 0), f[0]);
          unpack8<T>(staged(from, 1), f[1]);
          to_cache(1, h, h < a.Hkv, f);
        }
      }
    }
  }
  cp_async_wait<0>();
}

// Backward of the norm and the rotation.  A block sums its rows' part of dw in
// registers, then over its lanes in a fixed order; the join adds the blocks'.
template <typename T, int D, bool ANY>
__global__ void __launch_bounds__(kWarps * 32, ANY ? 1 : 2) rotary_norm_bwd_kernel(const RotArgs a) {
  constexpr int L = D / 16, RPW = 32 / L;
  extern __shared__ __align__(16) uint8_t stages[];
  __shared__ __align__(16) float angles[kWarps][2][kMaxPairs];
  __shared__ __align__(16) float weights[2][D];
  __shared__ float sums[kWarps][2][D];
  pdl_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  stage_weights<T, D>(a, a.wq, weights[0]);
  stage_weights<T, D>(a, a.wk, weights[1]);
  __syncthreads();
  const Place w = place_of<D>(a, lane);
  const int sub = lane / L;
  float *cs = angles[warp][0], *sn = angles[warp][1];
  float2 accq[2][4] = {}, acck[2][4] = {};
  const int nq = (a.Hq + RPW - 1) / RPW, nk = (a.Hkv + RPW - 1) / RPW;
  uint8_t* mine = stages + warp * a.slice_groups * 2048 + lane * 16;  // [group][input, gradient][chunk][lane]
  const uint32_t mine_s = smem_u32(mine);
  auto walk = [&](auto path_tag) {
    constexpr int PATH = decltype(path_tag)::value;
    const int step = gridDim.x * kWarps;
    for (int unit = blockIdx.x * kWarps + warp; unit < a.units; unit += step) {
      const int token = static_cast<int>(a.slice_div.div(unit)), slice = unit - token * static_cast<int>(a.slice_div.d);
      const int b = static_cast<int>(a.t_div.div(token)), t = token - b * a.T;
      const int g0 = slice * a.slice_groups, g1 = min(g0 + a.slice_groups, nq + nk);
      auto rows = [&](const RotRows& x) { return static_cast<T*>(x.p) + b * x.sb + t * x.st; };
      for (int g = g0; g < g1; ++g) {
        const uint32_t to = mine_s + (g - g0) * 2048;
        if (g < nq) {
          fetch_rows<T>(to, rows(a.q), a.q.sh, w, g * RPW + sub, a.Hq);
          fetch_rows<T>(to + 1024, rows(a.dq), a.dq.sh, w, g * RPW + sub, a.Hq);
        } else {
          fetch_rows<T>(to, rows(a.k), a.k.sh, w, (g - nq) * RPW + sub, a.Hkv);
          fetch_rows<T>(to + 1024, rows(a.dk), a.dk.sh, w, (g - nq) * RPW + sub, a.Hkv);
        }
        cp_async_commit();
      }
      token_angles(a, __ldg(a.pos + b * a.pos_b + t * a.pos_t), lane, cs, sn);
      Coef k;
      coefs<PATH>(a, w, cs, sn, nullptr, k);
      auto rows_of = [&](const RotRows& grad, const RotRows& out, const float* wt, float2 (&acc)[2][4], int heads, int base,
                         int n0, int n1) {
        T* po = rows(out);
#pragma unroll 1
        for (int gr = n0; gr < n1; ++gr) {
          wait_copies(g1 - 1 - gr);
          const uint8_t* from = mine + (gr - g0) * 2048;
          const int h = (gr - base) * RPW + sub;
          const bool act = h < heads;
          float2 fr[1][2][4], g[2][4], gp[2][4];
          float2(&f)[2][4] = fr[0];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            unpack8<T>(staged(from, i), f[i]);
            unpack8<T>(staged(from + 1024, i), g[i]);
          }
          partners<T, PATH>(a, w, g, rows(grad) + h * grad.sh, act, gp);
          float r1[1], by[1];
          const bool scaled = row_norm<D, 1>(fr, a.eps, r1, by);
          const float r = act ? r1[0] : 0.f;  // (without eps a row of zeros has none: rows that are none must add zeros)
          const float2 r2 = make_float2(r, r);
          float2 dot2 = make_float2(0.f, 0.f), wv[2][4];
          load_weights(w, wt, wv);
          float2 y[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y[i][e] = ffma2(g[i][e], k.ca[i][e], fmul2(gp[i][e], k.cb[i][e]));
              f[i][e] = fmul2(f[i][e], r2);  // h = u r
              acc[i][e] = ffma2(y[i][e], f[i][e], acc[i][e]);
              y[i][e] = fmul2(y[i][e], wv[i][e]);
              dot2 = ffma2(y[i][e], f[i][e], dot2);
            }
          const float dot = row_sum<L>(dot2.x + dot2.y) * (-1.f / D);
          const float2 d2 = make_float2(dot, dot), by2 = make_float2(by[0], by[0]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y[i][e] = fmul2(r2, ffma2(f[i][e], d2, y[i][e]));
              if (scaled) y[i][e] = fmul2(y[i][e], by2);  // (r times by may be past fp32's range)
            }
            if (act) *reinterpret_cast<uint4*>(po + h * out.sh + w.at[i]) = pack8<T>(y[i]);
          }
        }
      };
      rows_of(a.dq, a.qo, weights[0], accq, a.Hq, 0, g0, min(g1, nq));
      rows_of(a.dk, a.ko, weights[1], acck, a.Hkv, nq, max(g0, nq), g1);
    }
  };
  if constexpr (ANY) walk(std::integral_constant<int, kAny>{});
  else if (w.path == kHalves) walk(std::integral_constant<int, kHalves>{});
  else walk(std::integral_constant<int, kNeighbours>{});
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 v = m ? acck[i][e] : accq[i][e];
#pragma unroll
        for (int s = 16; s >= L; s >>= 1) {
          v.x += __shfl_xor_sync(0xffffffffu, v.x, s);
          v.y += __shfl_xor_sync(0xffffffffu, v.y, s);
        }
        if (sub == 0) {
          sums[warp][m][w.at[i] + 2 * e] = v.x;
          sums[warp][m][w.at[i] + 2 * e + 1] = v.y;
        }
      }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kWarps * 32) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) v += sums[k][i / D][i % D];
    a.part[static_cast<size_t>(blockIdx.x) * 2 * D + i] = v;
  }
}

// dw[i] = sum of the blocks' partial sums, each of a block's 32 warps over every
// 32nd block, in a fixed order.  A warp's loads are under way together: with 8 warps and four
// at a time the kernel was nine dependent trips to L2.
constexpr int kDwWarps = 32;
template <int D>
__global__ void __launch_bounds__(kDwWarps * 32) rotary_dw_kernel(const float* part, int blocks, float* dwq,
                                                                  float* dwk) {
  constexpr int kMost = (kRotBwdBlocks + kDwWarps - 1) / kDwWarps;
  __shared__ float sums[kDwWarps][32];
  const int lane = threadIdx.x & 31, col = blockIdx.x * 32 + lane, warp = threadIdx.x >> 5;
  pdl_wait();
  float v[kMost];
#pragma unroll
  for (int u = 0; u < kMost; ++u) {
    const int i = warp + kDwWarps * u;
    v[u] = i < blocks ? part[static_cast<size_t>(i) * 2 * D + col] : 0.f;
  }
#pragma unroll
  for (int u = 1; u < kMost; ++u) v[0] += v[u];
  sums[warp][lane] = v[0];
  __syncthreads();
  if (warp == 0) {
    float t[4] = {};
#pragma unroll
    for (int k = 0; k < kDwWarps; ++k) t[k & 3] += sums[k][lane];
    float* out = col < D ? dwq : dwk;
    if (out) out[col % D] = (t[0] + t[1]) + (t[2] + t[3]);
  }
}

template <typename T, int D, int MODE, int CT, bool ANY>
static cudaError_t launch_rows(const RotArgs& a, const CacheArgs& c, cudaStream_t s) {
  auto kern = rotary_kernel<T, D, MODE, CT, ANY>;
  static std::atomic<bool> attr[kMaxDevices];
  cudaError_t e = smem_attr_once(kern, kWarps * kRotGroups * 1024, attr);
  if (e != cudaSuccess) return e;
  const unsigned blocks = static_cast<unsigned>((static_cast<long long>(a.units) + kWarps - 1) / kWarps);
  kern<<<blocks, kWarps * 32, kWarps * a.slice_groups * 1024, s>>>(a, c);
  return cudaGetLastError();
}

template <typename T, int D, bool ANY>
static cudaError_t run_rotary_any(int mode, int ct, const RotArgs& a, const CacheArgs& c, cudaStream_t s) {
  if (mode == kRotPlain) return launch_rows<T, D, kRotPlain, kCache16, ANY>(a, c, s);
  if (mode == kRotNorm) return launch_rows<T, D, kRotNorm, kCache16, ANY>(a, c, s);
  if (mode == kRotAppend) {
    if (ct == kCache16) return launch_rows<T, D, kRotAppend, kCache16, ANY>(a, c, s);
    if (ct == kCacheE4m3) return launch_rows<T, D, kRotAppend, kCacheE4m3, ANY>(a, c, s);
    return launch_rows<T, D, kRotAppend, kCacheI8, ANY>(a, c, s);
  }
  auto kern = rotary_norm_bwd_kernel<T, D, ANY>;
  static std::atomic<bool> attr[kMaxDevices];
  cudaError_t e = smem_attr_once(kern, kWarps * kRotBwdGroups * 2048, attr);
  if (e != cudaSuccess) return e;
  kern<<<a.blocks, kWarps * 32, kWarps * a.slice_groups * 2048, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return pdl_launch(rotary_dw_kernel<D>, dim3(2 * D / 32), kDwWarps * 32, 0, s, static_cast<const float*>(a.part), a.blocks, a.dwq,
                    a.dwk);
}

// Whole rows in halves of whole chunks, or interleaved: the lean instances.
template <typename T, int D>
static cudaError_t run_rotary_d(int mode, int ct, const RotArgs& a, const CacheArgs& c, cudaStream_t s) {
  const bool lean = a.rot == D && (a.interleaved || a.pairs % 8 == 0);
  return lean ? run_rotary_any<T, D, false>(mode, ct, a, c, s) : run_rotary_any<T, D, true>(mode, ct, a, c, s);
}

template <typename T>
static cudaError_t run_rotary_t(int mode, int ct, int D, const RotArgs& a, const CacheArgs& c, cudaStream_t s) {
  switch (D) {
    case 16: return run_rotary_d<T, 16>(mode, ct, a, c, s);
    case 32: return run_rotary_d<T, 32>(mode, ct, a, c, s);
    case 64: return run_rotary_d<T, 64>(mode, ct, a, c, s);
    case 128: return run_rotary_d<T, 128>(mode, ct, a, c, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ta
