// Attention of new tokens over a paged key/value cache, for few query rows
// per key head (one token, a small draft): the keys are read once, and their
// bytes bound the call.
//
//   t_ij = log2(e) sm_scale <q_i, k_j> (+ log2 sv_j for 8-bit caches)
//   O_i  = sum_j 2^(t_ij - m_i) v_j / l_i,   m_i a running maximum of t_ij
//   l_i  = sum_j 2^(t_ij - m_i) (/ sv_j),    L_i = ln 2 (m_i + log2 l_i)
//
// A cached 8-bit row is code * scale.  A key's scale multiplies its finished
// score; a value's scale sv_j is put into the exponent, so that the weights
// 2^(t - m) <= 2^8 multiply the bare codes in fp16 (exact for both code types)
// and are rounded relative to the row's largest contribution; the softmax
// sum takes the scale out again in fp32.
//
// Query rows.  The G query heads that share a key head and the sequence's new
// tokens make up to G * q_len rows, taken 16 at a time (an m16n8k16 tile).  A
// block's four warps take 16 or 32 keys of a tile each and keep their own
// running maximum, sum and accumulators in registers: no barrier between
// tiles.  Every warp copies its keys and values into its own ring in shared
// memory (cp.async, swizzled), kStages tiles ahead.  The warps' states are
// joined through shared memory at the end of a sequence.
//
// Work is cut as attn_cache.cuh says, two blocks per SM.
#include "attn_cache.cuh"

namespace ta {

namespace {

constexpr int kRows = 16;      // query rows per unit
constexpr int kWarps = 4;      // warps per block, each with its own keys
constexpr int kStages = 3;     // tiles in a warp's ring
constexpr int kBlocks = 304;   // two per SM: 152 SMs

template <int CT, int D>
struct Cfg {
  static constexpr int ES = CT == kCache16 ? 2 : 1;         // bytes per element
  static constexpr int RB = D * ES;                         // bytes per row
  static constexpr int KW = RB >= 256 ? 16 : 32;            // keys per warp and tile
  static constexpr int TK = KW * kWarps;                    // keys per tile
  static constexpr int CPR = RB / 16;                       // 16-byte chunks per row
  static constexpr int SLOT = 2 * KW * RB;                  // K and V of one warp and stage
  static constexpr int SCALES = CT == kCache16 ? 0 : KW * 8;  // K and V scales of one warp and stage
  static constexpr int RING = kStages * (SLOT + SCALES);    // one warp
  static constexpr int OBYTES = kRows * D * 4;              // one warp's accumulators
  static_assert(SLOT >= OBYTES, "a slot holds a warp's accumulators");
  static constexpr int SMEM = kWarps * RING + kWarps * kRows * 8 + 64;
};

// Position of 16-byte chunk `ch` of row r in a slot.  16-bit rows are read by
// ldmatrix (eight rows, one chunk column each); 8-bit rows by 16-, 8- or
// 4-byte loads, keys along lane / 4 with chunks along lane % 4 for K and the
// other way round, two rows apart, for V.
template <int CT, int D>
__device__ __forceinline__ int swz(int r, int ch) {
  constexpr int C = Cfg<CT, D>::CPR;
  if constexpr (CT == kCache16) {
    if constexpr (C >= 8) return ch ^ (r & 7);
    else if constexpr (C == 4) return ch ^ ((r >> 1) & 3);
    else return ch ^ ((r >> 2) & 1);
  } else {
    if constexpr (C == 8) return ch ^ (((r >> 1) & 3) << 1) ^ ((r & 1) << 2);
    else if constexpr (C == 4) return ch ^ ((r >> 1) & 3);
    else if constexpr (C == 2) return ch ^ ((r >> 2) & 1);
    else return ch;
  }
}

__device__ __forceinline__ void ldsm_x4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
template <bool BF>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int BYTES>
__device__ __forceinline__ void lds_bytes(uint32_t a, uint32_t (&w)[(BYTES + 3) / 4]) {
  if constexpr (BYTES == 16)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a) : "memory");
  else if constexpr (BYTES == 8)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a) : "memory");
  else if constexpr (BYTES == 4)
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(a) : "memory");
  else {
    uint16_t h;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(a) : "memory");
    w[0] = h;
  }
}
__device__ __forceinline__ float2 lds_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

// A partial state: 16 x D unnormalised accumulators, then m and l per row.
template <int D>
__host__ __device__ constexpr int part_floats() { return kRows * D + 2 * kRows; }

// Where float4 `ch` of row r lies in a warp's staged accumulators (spreads
// both fragment layouts' writes and the row-wise reads over the banks).
template <int D>
__device__ __forceinline__ int oswz(int r, int ch) {
  return ch ^ ((((r & 3) << 1) ^ (ch >> 3)) & (D / 4 - 1) & 7);
}

template <typename T, int CT, int D>
__global__ void __launch_bounds__(kWarps * 32, 2) attn_cache_kernel(CacheArgs c, CacheAttnArgs a) {
  using F = Cfg<CT, D>;
  constexpr bool BF = DT<T>::bf16;
  constexpr bool MBF = BF && CT == kCache16;  // matrix instructions in bf16
  constexpr int KW = F::KW, TK = F::TK, NT = KW / 8;
  constexpr int NK = D / 16;  // k-steps of Q K^T
  extern __shared__ __align__(128) uint8_t smem[];
  using Ln = Line<kRows, TK>;
  __shared__ typename Ln::Shared line;
  let_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, cq = lane & 3;

  long long mine, before;
  const long long len = Ln::template length<kWarps * 32>(c, a, line, &mine, &before);
  const long long x0 = cut(len, gridDim.x, blockIdx.x), x1 = cut(len, gridDim.x, blockIdx.x + 1);
  if (x0 >= x1) return;
  typename Ln::Cursor cc;
  Ln::template find<kWarps * 32>(c, a, line, x0, mine, before, cc);
  typename Ln::Cursor pc = cc;  // the next tile to copy

  uint8_t* const ring = smem + warp * F::RING;
  float* const ml = reinterpret_cast<float*>(smem + kWarps * F::RING);  // [warps][16][2]
  const uint32_t ring_a = smem_u32(ring);

  // Page entry of this lane's key of the next tile to copy, read a tile early.
  int pid = -1, prow = 0;
  auto look_up = [&]() {
    const int n = pc.t * TK + warp * KW + (lane & (KW - 1));
    pid = -1;
    if (n < pc.s.kv) pid = cache_page_id(c, pc.b, n, &prow);
    else prow = -1;
  };
  auto copy_tile = [&](int slot) {
    const int rid = prow < 0 ? -1 : cache_row(c, pc.h, pid, prow);
    const uint32_t dst = ring_a + slot * (F::SLOT + F::SCALES);
#pragma unroll
    for (int i = 0; i < KW * F::CPR / 32; ++i) {
      const int r = (i * 32 + lane) / F::CPR, ch = lane % F::CPR;
      const int src = __shfl_sync(0xffffffffu, rid, r);
      const size_t off = static_cast<size_t>(src < 0 ? 0 : src) * F::RB + ch * 16;
      const uint32_t at = dst + r * F::RB + swz<CT, D>(r, ch) * 16;
      cp_async16(at, static_cast<const uint8_t*>(c.k) + off, src >= 0);
      cp_async16(at + KW * F::RB, static_cast<const uint8_t*>(c.v) + off, src >= 0);
    }
    if constexpr (CT != kCache16) {  // KW == 32: a key per lane
      const size_t off = static_cast<size_t>(rid < 0 ? 0 : rid);
      cp_async4(dst + F::SLOT + lane * 4, c.ks + off, rid >= 0);
      cp_async4(dst + F::SLOT + KW * 4 + lane * 4, c.vs + off, rid >= 0);
    }
  };

  look_up();
#pragma unroll
  for (int s = 0; s < kStages; ++s) {
    if (x0 + s < x1) {
      copy_tile(s);
      Ln::next_tile(c, a, pc);
      if (x0 + s + 1 < x1) look_up();
    }
    cp_async_commit();
  }

  uint32_t qf[NK][4];
  float oa[D / 8][4];
  float m[2], l[2], fac[2];
  int tok[2];  // new token of this thread's rows (lane / 4, + 8); -1: no row
  bool fresh = true;
  bool from_start = false;  // the piece holds its unit's first tile
  int slot = 0;
  for (long long x = x0; x < x1; ++x) {
    if (fresh) {
      fresh = false;
      from_start = cc.t == 0;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) oa[j][0] = oa[j][1] = oa[j][2] = oa[j][3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = cc.rt * kRows + g + 8 * e;
        const int t = static_cast<int>(a.g_div.div(r));
        tok[e] = t < cc.s.q ? t : -1;
        fac[e] = a.scale_log2;
        const T* p = static_cast<const T*>(a.q);
        if (tok[e] >= 0)
          p += cc.b * a.qs[0] + static_cast<long long>(cc.h * a.G + (r - t * a.G)) * a.qs[1] + t * a.qs[2];
        if constexpr (CT == kCache16) {
          const uint32_t* p32 = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
          for (int kk = 0; kk < NK; ++kk) {
            qf[kk][e] = tok[e] >= 0 ? __ldg(p32 + kk * 8 + cq) : 0u;
            qf[kk][2 + e] = tok[e] >= 0 ? __ldg(p32 + kk * 8 + 4 + cq) : 0u;
          }
        } else {
          // this lane's share of a row is D / 4 neighbouring elements, those
          // that it reads of a key's codes: k-step kk takes four of them
          const uint2* p64 = reinterpret_cast<const uint2*>(p + cq * (D / 4));
          uint32_t top = 0;
#pragma unroll
          for (int kk = 0; kk < NK; ++kk) {
            const uint2 w = tok[e] >= 0 ? __ldg(p64 + kk) : make_uint2(0u, 0u);
            qf[kk][e] = w.x;
            qf[kk][2 + e] = w.y;
            if constexpr (BF) {
              top = max(top, max(w.x & 0x7fffu, (w.x >> 16) & 0x7fffu));
              top = max(top, max(w.y & 0x7fffu, (w.y >> 16) & 0x7fffu));
            }
          }
          if constexpr (BF) {
            // bf16 -> fp16 with the row's largest magnitude brought to
            // [1, 2) by a power of two: the elements keep their 8 bits down
            // to 2^-14 of it and are rounded to 2^-25 of it below
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            int ex = static_cast<int>(top >> 7);                  // biased exponent
            ex = ex < 1 ? 1 : (ex > 253 ? 253 : ex);              // zero rows, infinities: some finite power
            const float up = __uint_as_float(static_cast<uint32_t>(254 - ex) << 23);
            fac[e] *= __uint_as_float(static_cast<uint32_t>(ex) << 23);
#pragma unroll
            for (int kk = 0; kk < NK; ++kk) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t w = qf[kk][2 * i + e];
                qf[kk][2 * i + e] = pack2<false>(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
              }
            }
          }
        }
      }
    }

    cp_async_wait<kStages - 1>();
    __syncwarp();
    const uint32_t ks_a = ring_a + slot * (F::SLOT + F::SCALES), vs_a = ks_a + KW * F::RB, sc_a = ks_a + F::SLOT;
    const int n0 = cc.t * TK + warp * KW;          // this warp's first key
    const int past = cc.s.kv - cc.s.q;             // keys every new token sees
    if (n0 < cc.s.kv) {
      float s[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
      if constexpr (CT == kCache16) {
#pragma unroll
        for (int p = 0; p < KW / 16; ++p) {
          const int r = p * 16 + ((lane >> 4) << 3) + (lane & 7);
#pragma unroll
          for (int kk = 0; kk < NK; ++kk) {
            uint32_t b[4];
            ldsm_x4(ks_a + r * F::RB + swz<CT, D>(r, kk * 2 + ((lane >> 3) & 1)) * 16, b);
            mma16816<MBF>(s[2 * p], qf[kk], b[0], b[1]);
            mma16816<MBF>(s[2 * p + 1], qf[kk], b[2], b[3]);
          }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[j][i] *= fac[i >> 1];
      } else {
        constexpr int PB = D / 4;  // bytes of a key's row per lane
        constexpr int PL = PB > 16 ? 16 : PB;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int r = j * 8 + g;
#pragma unroll
          for (int q = 0; q < PB / PL; ++q) {
            uint32_t w[PL / 4];
            const int byte = cq * PB + q * PL;
            lds_bytes<PL>(ks_a + r * F::RB + swz<CT, D>(r, byte / 16) * 16 + (byte & 15), w);
#pragma unroll
            for (int i = 0; i < PL / 4; ++i) {
              uint32_t b0, b1;
              code4_to_f16<CT>(w[i], b0, b1);
              mma16816<false>(s[j], qf[q * (PL / 4) + i], b0, b1);
            }
          }
        }
        // score scales, and each key's value scale in the exponent
        float kscale, vscale;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(kscale) : "r"(sc_a + lane * 4) : "memory");
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vscale) : "r"(sc_a + KW * 4 + lane * 4) : "memory");
        // a scale of zero (a row of a page that the cache does not have reads
        // as zeros) stands for a value of zero whatever its codes
        if (vscale == 0.f) vscale = kMinScale;
        const float lg = lg2(vscale);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float kx = __shfl_sync(0xffffffffu, kscale, j * 8 + 2 * cq + i);
            const float vx = __shfl_sync(0xffffffffu, lg, j * 8 + 2 * cq + i);
            s[j][i] = fmaf(s[j][i], fac[0] * kx, vx);
            s[j][2 + i] = fmaf(s[j][2 + i], fac[1] * kx, vx);
          }
        }
        if (lane < KW)  // the softmax sum's 1 / scale, read back below
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(sc_a + KW * 4 + lane * 4), "f"(vscale == vscale ? __fdividef(1.f, vscale) : 0.f) : "memory");
        __syncwarp();
      }

      // keys behind the end, and new tokens that a row must not see
      const bool masked = n0 + KW > past;
      uint32_t seen[2] = {0xffffffffu, 0xffffffffu};  // bit 2 j + i: score s[j][2 e + i]
      if (masked) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int n = n0 + j * 8 + 2 * cq + i;
              const int d = n - past;
              bool see = tok[e] >= 0 && n < cc.s.kv;
              if (see && d >= 0)
                see = a.tree ? __ldg(a.tree + cc.b * a.tree_b + tok[e] * a.tree_t + d) != 0 : d <= tok[e];
              if (!see) {
                s[j][2 * e + i] = -INFINITY;
                seen[e] &= ~(1u << (2 * j + i));
              }
            }
          }
        }
      }

      // running maximum, raised only when a score passes it by 2^8
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        mx[0] = fmax3(mx[0], s[j][0], s[j][1]);
        mx[1] = fmax3(mx[1], s[j][2], s[j][3]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
      }
      if (__any_sync(0xffffffffu, mx[0] > m[0] + kRescaleThreshold || mx[1] > m[1] + kRescaleThreshold)) {
        float al[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = fmaxf(m[e], mx[e]);
          al[e] = mn == -INFINITY ? 1.f : ex2(m[e] - mn);
          m[e] = mn;
          l[e] *= al[e];
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          oa[j][0] *= al[0];
          oa[j][1] *= al[0];
          oa[j][2] *= al[1];
          oa[j][3] *= al[1];
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ref = m[e] == -INFINITY ? 0.f : m[e];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
          for (int i = 0; i < 2; ++i) s[j][2 * e + i] = ex2(s[j][2 * e + i] - ref);
        }
      }
      if constexpr (CT == kCache16) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          l[0] += s[j][0] + s[j][1];
          l[1] += s[j][2] + s[j][3];
        }
      } else {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float2 iv = lds_f2(sc_a + KW * 4 + (j * 8 + 2 * cq) * 4);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // a hidden key's scale may be anything, a NaN row's among them
            l[e] = (seen[e] >> (2 * j)) & 1u ? fmaf(s[j][2 * e], iv.x, l[e]) : l[e];
            l[e] = (seen[e] >> (2 * j + 1)) & 1u ? fmaf(s[j][2 * e + 1], iv.y, l[e]) : l[e];
          }
        }
      }

      if constexpr (CT == kCache16) {
        // A new token's value may hold infinities or NaN that some rows must
        // not see, and 0 * NaN is NaN in the product: such elements are added
        // to the rows that do see them here and taken out of the tile.
        if (masked && cc.s.kv > past) {
          bool odd = false;
          constexpr uint32_t EXP = BF ? 0x7f80u : 0x7c00u;
#pragma unroll
          for (int i = 0; i < KW * F::CPR / 32; ++i) {
            uint32_t w[4];
            lds_bytes<16>(vs_a + (i * 32 + lane) * 16, w);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              odd |= (w[k] & EXP) == EXP || ((w[k] >> 16) & EXP) == EXP;
          }
          if (__any_sync(0xffffffffu, odd)) {
            for (int r = 0; r < KW; ++r) {
              // weights of key r for this thread's two rows: held by the lane
              // of the same quad at column (r % 8) / 2
              const int from = (lane & ~3) | ((r & 7) >> 1);
              float w0 = 0.f, w1 = 0.f;
#pragma unroll
              for (int j = 0; j < NT; ++j) {
                if (j == (r >> 3)) {
                  w0 = __shfl_sync(0xffffffffu, (r & 1) ? s[j][1] : s[j][0], from);
                  w1 = __shfl_sync(0xffffffffu, (r & 1) ? s[j][3] : s[j][2], from);
                }
              }
#pragma unroll
              for (int j = 0; j < D / 8; ++j) {
                const uint32_t at = vs_a + r * F::RB + swz<CT, D>(r, j) * 16 + cq * 4;
                uint32_t w[1];
                lds_bytes<4>(at, w);
                const T* h = reinterpret_cast<const T*>(w);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const float v = static_cast<float>(h[i]);
                  if ((__float_as_uint(v) & 0x7f800000u) == 0x7f800000u) {
                    if (w0 != 0.f) oa[j][i] = fmaf(w0, v, oa[j][i]);
                    if (w1 != 0.f) oa[j][2 + i] = fmaf(w1, v, oa[j][2 + i]);
                  }
                }
              }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < KW * F::CPR / 32; ++i) {
              const uint32_t at = vs_a + (i * 32 + lane) * 16;
              uint32_t w[4];
              lds_bytes<16>(at, w);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if ((w[k] & EXP) == EXP) w[k] &= 0xffff0000u;
                if (((w[k] >> 16) & EXP) == EXP) w[k] &= 0x0000ffffu;
              }
              sts_v4(at, w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
          }
        }
#pragma unroll
        for (int p = 0; p < KW / 16; ++p) {
          uint32_t pf[4];
          pf[0] = pack2<MBF>(s[2 * p][0], s[2 * p][1]);
          pf[1] = pack2<MBF>(s[2 * p][2], s[2 * p][3]);
          pf[2] = pack2<MBF>(s[2 * p + 1][0], s[2 * p + 1][1]);
          pf[3] = pack2<MBF>(s[2 * p + 1][2], s[2 * p + 1][3]);
          const int r = p * 16 + (((lane >> 3) & 1) << 3) + (lane & 7);
#pragma unroll
          for (int dp = 0; dp < D / 16; ++dp) {
            uint32_t b[4];
            ldsm_x4_t(vs_a + r * F::RB + swz<CT, D>(r, dp * 2 + (lane >> 4)) * 16, b);
            mma16816<MBF>(oa[2 * dp], pf, b[0], b[1]);
            mma16816<MBF>(oa[2 * dp + 1], pf, b[2], b[3]);
          }
        }
      } else {
        // Accumulator tile j's column n is value element n * (D / 8) + j: a
        // lane then reads D / 8 neighbouring codes of its four keys.
        constexpr int VB = D / 8;
#pragma unroll
        for (int p = 0; p < KW / 16; ++p) {
          uint32_t pf[4];
          pf[0] = pack2<false>(s[2 * p][0], s[2 * p][1]);
          pf[1] = pack2<false>(s[2 * p][2], s[2 * p][3]);
          pf[2] = pack2<false>(s[2 * p + 1][0], s[2 * p + 1][1]);
          pf[3] = pack2<false>(s[2 * p + 1][2], s[2 * p + 1][3]);
          uint32_t w[4][(VB + 3) / 4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = p * 16 + (i >> 1) * 8 + 2 * cq + (i & 1);
            lds_bytes<VB>(vs_a + r * F::RB + swz<CT, D>(r, g * VB / 16) * 16 + ((g * VB) & 15), w[i]);
          }
#pragma unroll
          for (int q = 0; q < (VB + 3) / 4; ++q) {
#pragma unroll
            for (int hh = 0; hh < (VB < 4 ? 1 : 2); ++hh) {
              // two codes of each of two keys -> (key, key + 1) pairs
              const uint32_t sel = hh ? 0x7362 : 0x5140;
              uint32_t a0, a1, b0, b1;
              code4_to_f16<CT>(__byte_perm(w[0][q], w[1][q], sel), a0, a1);
              code4_to_f16<CT>(__byte_perm(w[2][q], w[3][q], sel), b0, b1);
              mma16816<false>(oa[q * 4 + hh * 2], pf, a0, b0);
              mma16816<false>(oa[q * 4 + hh * 2 + 1], pf, a1, b1);
            }
          }
        }
      }
    }

    const bool last = cc.t + 1 == cc.ntiles;
    if (last || x + 1 == x1) {
      // ------------------------------------- end of the piece: join the warps
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      }
      if (cq == 0) {
        ml[(warp * kRows + g) * 2] = m[0];
        ml[(warp * kRows + g) * 2 + 1] = l[0];
        ml[(warp * kRows + g + 8) * 2] = m[1];
        ml[(warp * kRows + g + 8) * 2 + 1] = l[1];
      }
      // this warp's accumulators go over the tile it has just used
      __syncwarp();
      uint8_t* const st = ring + slot * (F::SLOT + F::SCALES);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = g + 8 * e;
        float* const row = reinterpret_cast<float*>(st) + r * D;
        if constexpr (CT == kCache16) {
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
            *reinterpret_cast<float2*>(row + oswz<D>(r, 2 * j + (cq >> 1)) * 4 + (cq & 1) * 2) =
                make_float2(oa[j][2 * e], oa[j][2 * e + 1]);
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int j = 0; j < D / 8; j += 2) {
              const int d = (2 * cq + i) * (D / 8) + j;
              *reinterpret_cast<float2*>(row + oswz<D>(r, d >> 2) * 4 + (d & 3)) =
                  make_float2(oa[j][2 * e + i], oa[j + 1][2 * e + i]);
            }
          }
        }
      }
      __syncthreads();
      {
        const int r = threadIdx.x >> 3, sub = threadIdx.x & 7;  // 16 rows, 8 threads each
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, ml[(w * kRows + r) * 2]);
        float f[kWarps], ll = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          f[w] = mm == -INFINITY ? 0.f : ex2(ml[(w * kRows + r) * 2] - mm);
          // a NaN sum stays one where no score was a number
          ll += (mm == -INFINITY ? 1.f : f[w]) * ml[(w * kRows + r) * 2 + 1];
        }
        const bool whole = from_start && last;
        const int qr = cc.rt * kRows + r;
        const int t = static_cast<int>(a.g_div.div(qr)), hq = cc.h * a.G + (qr - t * a.G);
        const bool real = t < cc.s.q;
        float norm = 1.f;
        if (whole) norm = ll == 0.f ? 0.f : 1.f / ll;
        float* const part =
            a.ws + (static_cast<size_t>(blockIdx.x) * 2 + (x + 1 - x0 > cc.t + 1 ? 1 : 0)) * part_floats<D>();
        T* const out = static_cast<T*>(a.o) + cc.b * a.os[0] + hq * a.os[1] + t * a.os[2];
#pragma unroll
        for (int i = 0; i < (D / 4 + 7) / 8; ++i) {
          const int ch = sub + 8 * i;
          if (ch < D / 4) {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              const float4 y = *(reinterpret_cast<const float4*>(smem + w * F::RING + slot * (F::SLOT + F::SCALES)) +
                                 r * (D / 4) + oswz<D>(r, ch));
              v[0] = fmaf(f[w], y.x, v[0]);
              v[1] = fmaf(f[w], y.y, v[1]);
              v[2] = fmaf(f[w], y.z, v[2]);
              v[3] = fmaf(f[w], y.w, v[3]);
            }
            if (whole) {
              if (real) {
                uint2 u;
                u.x = pack2<BF>(v[0] * norm, v[1] * norm);
                u.y = pack2<BF>(v[2] * norm, v[3] * norm);
                *reinterpret_cast<uint2*>(out + ch * 4) = u;
              }
            } else {
              reinterpret_cast<float4*>(part + r * D)[ch] = make_float4(v[0], v[1], v[2], v[3]);
            }
          }
        }
        if (sub == 0) {
          if (!whole) {
            part[kRows * D + 2 * r] = mm;
            part[kRows * D + 2 * r + 1] = ll;
          } else if (real) {
            a.lse[(static_cast<long long>(cc.b) * a.Hq + hq) * c.T + t] =
                ll == 0.f ? -INFINITY : (mm == -INFINITY ? ll : (mm + lg2(ll)) * kLn2);
          }
        }
      }
      __syncthreads();
      fresh = true;
    } else {
      __syncwarp();
    }
    if (x + kStages < x1) {
      copy_tile(slot);
      Ln::next_tile(c, a, pc);
      if (x + kStages + 1 < x1) look_up();
    }
    cp_async_commit();
    slot = slot + 1 == kStages ? 0 : slot + 1;
    Ln::next_tile(c, a, cc);
  }
}

// Joins the partial states of the units that block borders cut: block (i, y)
// joins rows 4 y .. 4 y + 3 of the unit that border i + 1 is the first to cut.
// Two warps share a row.  A unit can have hundreds of parts (one long sequence
// over all blocks), so that everything but the sum of the accumulators runs
// over the parts in parallel, and that sum has eight loads in flight.
template <typename T, int CT, int D>
__global__ void __launch_bounds__(256) attn_cache_join_kernel(CacheArgs c, CacheAttnArgs a) {
  constexpr bool BF = DT<T>::bf16;
  constexpr int VEC = D >= 128 ? 4 : (D >= 64 ? 2 : 1);  // elements per lane
  using Ln = Line<kRows, Cfg<CT, D>::TK>;
  __shared__ typename Ln::Shared line;
  __shared__ int slots[kBlocks];
  __shared__ float fs[4][kBlocks];
  __shared__ float other[4][D + 1];
  typename Ln::Cursor u;
  const int parts = unit_parts<Ln, 256>(c, a, line, kBlocks, blockIdx.x + 1, slots, u);
  wait_for_main_kernel();  // every block: the next kernel in the stream may start when this one has ended
  if (parts == 0 || static_cast<int>(blockIdx.y) * 4 + u.rt * kRows >= u.s.q * a.G) return;
  const int wrow = threadIdx.x >> 6, half = (threadIdx.x >> 5) & 1, lane = threadIdx.x & 31;
  const int r = blockIdx.y * 4 + wrow;
  auto part = [&](int i) { return a.ws + static_cast<size_t>(slots[i]) * part_floats<D>(); };
  // both warps of a row: its maximum and sum, and the parts' factors
  float mm = -INFINITY;
  for (int i = lane; i < parts; i += 32)
    if (slots[i] >= 0) mm = fmaxf(mm, __ldcg(part(i) + kRows * D + 2 * r));
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, s));
  float ll = 0.f;
  for (int i = lane; i < parts; i += 32) {
    float f = 0.f;
    if (slots[i] >= 0) {
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(part(i) + kRows * D + 2 * r));
      f = ml.x == -INFINITY ? 0.f : ex2(ml.x - mm);
      ll += mm == -INFINITY ? ml.y : ml.y * f;  // a NaN sum stays one where no score was a number
    }
    if (half == 0) fs[wrow][i] = f;
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, s);
  __syncthreads();
  float v[VEC] = {};
  const bool lane_on = lane * VEC < D;
  if (lane_on) {
#pragma unroll 8
    for (int i = half; i < parts; i += 2) {
      const float f = fs[wrow][i];
      // (a block without a piece has factor 0; the first one listed always has a piece)
      const float* p = part(slots[i] < 0 ? 0 : i) + r * D + lane * VEC;
      if constexpr (VEC == 4) {
        const float4 y = __ldcg(reinterpret_cast<const float4*>(p));
        v[0] = fmaf(y.x, f, v[0]);
        v[1] = fmaf(y.y, f, v[1]);
        v[2] = fmaf(y.z, f, v[2]);
        v[3] = fmaf(y.w, f, v[3]);
      } else if constexpr (VEC == 2) {
        const float2 y = __ldcg(reinterpret_cast<const float2*>(p));
        v[0] = fmaf(y.x, f, v[0]);
        v[1] = fmaf(y.y, f, v[1]);
      } else {
        v[0] = fmaf(__ldcg(p), f, v[0]);
      }
    }
    if (half) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) other[wrow][lane * VEC + k] = v[k];
    }
  }
  __syncthreads();
  if (half) return;
  const int qr = u.rt * kRows + r;
  const int t = static_cast<int>(a.g_div.div(qr)), hq = u.h * a.G + (qr - t * a.G);
  if (t >= u.s.q) return;
  const float norm = ll == 0.f ? 0.f : 1.f / ll;
  if (lane_on) {
    T* out = static_cast<T*>(a.o) + u.b * a.os[0] + hq * a.os[1] + t * a.os[2] + lane * VEC;
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = (v[k] + other[wrow][lane * VEC + k]) * norm;
    if constexpr (VEC == 4) {
      uint2 w;
      w.x = pack2<BF>(v[0], v[1]);
      w.y = pack2<BF>(v[2], v[3]);
      *reinterpret_cast<uint2*>(out) = w;
    } else if constexpr (VEC == 2) {
      *reinterpret_cast<uint32_t*>(out) = pack2<BF>(v[0], v[1]);
    } else {
      const uint32_t w = pack2<BF>(v[0], 0.f);
      *reinterpret_cast<uint16_t*>(out) = static_cast<uint16_t>(w);
    }
  }
  if (lane == 0)
    a.lse[(static_cast<long long>(u.b) * a.Hq + hq) * c.T + t] =
        ll == 0.f ? -INFINITY : (mm == -INFINITY ? ll : (mm + lg2(ll)) * kLn2);
}

template <typename T, int CT, int D>
cudaError_t run(const CacheArgs& c, const CacheAttnArgs& a, cudaStream_t s) {
  static std::atomic<bool> done[kMaxDevices];
  auto* kern = attn_cache_kernel<T, CT, D>;
  constexpr int smem = Cfg<CT, D>::SMEM;
  cudaError_t e = smem_attr_once(kern, smem, done);
  if (e != cudaSuccess) return e;
  prof_begin("attn_cache", s);
  kern<<<kBlocks, kWarps * 32, smem, s>>>(c, a);
  prof_end(s);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  prof_begin("attn_cache_join", s);
  e = launch_join(attn_cache_join_kernel<T, CT, D>, dim3(kBlocks - 1, kRows / 4), 256, s, c, a);
  prof_end(s);
  return e;
}

template <typename T, int CT>
cudaError_t run_d(int D, const CacheArgs& c, const CacheAttnArgs& a, cudaStream_t s) {
  switch (D) {
    case 16: return run<T, CT, 16>(c, a, s);
    case 32: return run<T, CT, 32>(c, a, s);
    case 64: return run<T, CT, 64>(c, a, s);
    case 128: return run<T, CT, 128>(c, a, s);
    default: return cudaErrorInvalidValue;
  }
}
template <typename T>
cudaError_t run_c(int ct, int D, const CacheArgs& c, const CacheAttnArgs& a, cudaStream_t s) {
  if (ct == kCache16) return run_d<T, kCache16>(D, c, a, s);
  if (ct == kCacheE4m3) return run_d<T, kCacheE4m3>(D, c, a, s);
  return run_d<T, kCacheI8>(D, c, a, s);
}

}  // namespace

size_t attn_cache_ws_bytes(int D) {
  return static_cast<size_t>(kBlocks) * 2 * (kRows * D + 2 * kRows) * sizeof(float);
}

cudaError_t launch_attn_cache(bool bf16, int ct, int D, const CacheArgs& c, const CacheAttnArgs& a, cudaStream_t s) {
  return bf16 ? run_c<__nv_bfloat16>(ct, D, c, a, s) : run_c<__half>(ct, D, c, a, s);
}

}  // namespace ta

TA_GUARD_ACCESSOR(attn_cache)
