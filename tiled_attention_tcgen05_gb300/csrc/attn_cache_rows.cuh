// Attention of new tokens over a paged key/value cache, for few query rows
// per key head (one token, a small draft): the keys are read once, and their
// bytes bound the call.
//
//   t_ij = log2(e) sm_scale <q_i, k_j> (+ log2 sv_j for 8-bit caches)
//   O_i  = sum_j 2^(t_ij - m_i) v_j / l_i,   m_i a running maximum of t_ij
//   l_i  = sum_j 2^(t_ij - log2 sv_j - m_i),  L_i = ln 2 (m_i + log2 l_i)
//
// A cached 8-bit row is code * scale.  A key's scale multiplies its finished
// score; a value's scale sv_j is put into the exponent, so that the weights
// 2^(t - m) <= 2^8 multiply the bare codes in fp16 (exact for both code types)
// and are rounded relative to the row's largest contribution; the softmax
// sum takes the scale out again in fp32 (attn_cache.cuh).
//
// Query rows.  The G query heads that share a key head and the sequence's new
// tokens make up to G * q_len rows, taken 16 MT at a time (MT m16n8k16 tiles:
// a key's fragment is loaded, or converted, once for all of them).  A block's
// four warps take 16 or 32 keys of a tile each and keep their own running
// maximum, sum and accumulators in registers: no barrier between tiles.  Every warp copies its keys and values into its own ring in shared
// memory (cp.async, swizzled).  The warps' states are
// joined through shared memory at the end of a sequence.
//
// Work is cut as attn_cache.cuh says, two blocks per SM.  Few units of short
// sequences are taken by a cluster of eight blocks each instead (CLUSTER): they
// share the unit's keys and join their states over distributed shared memory,
// which saves the look at all sequences' lengths and the second kernel.
#pragma once
#include "attn_cache.cuh"
#include "cluster.cuh"

namespace ta {

namespace {

constexpr int kWarps = 4;      // warps per block, each with its own keys

template <int CT, int D, int MT>
struct Cfg {
  static constexpr int ROWS = 16 * MT;                      // query rows per unit
  // Two blocks per SM and two tiles in a warp's ring, for [64, 32/8, 1, 8192,
  // 128] bf16 and [3, 32/4, 1, 131071, 128] e4m3: 204 and 73 us; three
  // stages 214 and 76; three blocks (168 registers) of two stages 210 and 80;
  // one block of six stages 268 and 111.
  static constexpr int BPS = 2;
  static constexpr int BLOCKS = 152 * BPS;
  static constexpr int STAGES = 2;
  static constexpr int ES = CT == kCache16 ? 2 : 1;         // bytes per element
  static constexpr int RB = D * ES;                         // bytes per row
  static constexpr int KW = RB >= 256 ? 16 : 32;            // keys per warp and tile
  static constexpr int TK = KW * kWarps;                    // keys per tile
  static constexpr int CPR = RB / 16;                       // 16-byte chunks per row
  static constexpr int SLOT = 2 * KW * RB;                  // K and V of one warp and stage
  static constexpr int SCALES = CT == kCache16 ? 0 : KW * 12;  // K scale, V scale (then its log2), sum's factor
  static constexpr int RING = STAGES * (SLOT + SCALES);    // one warp
  static_assert(SLOT >= 16 * D * 4, "a slot holds a row tile of a warp's accumulators");
  static constexpr int QBYTES = MT > 1 ? MT * D * 32 : 0;   // Q fragments (one row tile's stay in registers)
  static constexpr int SMEM = kWarps * RING + kWarps * ROWS * 8 + QBYTES + ROWS * 4;
  // state of a unit: ROWS x D unnormalised accumulators, then m and l per row
  static constexpr int PART = ROWS * (D + 2);
};

// Position of 16-byte chunk `ch` of row r in a slot.  16-bit rows are read by
// ldmatrix (eight rows, one chunk column each); 8-bit rows by 16-, 8- or
// 4-byte loads, keys along lane / 4 with chunks along lane % 4 for K and the
// other way round, two rows apart, for V.
template <int CT, int D>
__device__ __forceinline__ int swz(int r, int ch) {
  constexpr int C = Cfg<CT, D, 1>::CPR;
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

// Where float4 `ch` of row r lies in a warp's staged accumulators (spreads
// both fragment layouts' writes and the row-wise reads over the banks).
template <int D>
__device__ __forceinline__ int oswz(int r, int ch) {
  return ch ^ ((((r & 3) << 1) ^ (ch >> 3)) & (D / 4 - 1) & 7);
}

constexpr int kCluster = 8;

template <typename T, int CT, int D, int MT, bool CLUSTER>
__global__ void __launch_bounds__(kWarps * 32, Cfg<CT, D, MT>::BPS) attn_cache_kernel(CacheArgs c, CacheAttnArgs a) {
  using F = Cfg<CT, D, MT>;
  constexpr bool BF = DT<T>::bf16;
  constexpr bool MBF = BF && CT == kCache16;  // matrix instructions in bf16
  constexpr int KW = F::KW, TK = F::TK, NT = KW / 8, ROWS = F::ROWS;
  constexpr int NK = D / 16;  // k-steps of Q K^T
  extern __shared__ __align__(128) uint8_t smem[];
  using Ln = Line<ROWS, TK>;
  __shared__ typename Ln::Shared line;
  if constexpr (!CLUSTER) let_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, cq = lane & 3;

  // This block's places x0 .. x1 of the line (CLUSTER: its tiles of the unit),
  // and the first of them.
  typename Ln::Cursor cc;
  long long x0, x1;
  [[maybe_unused]] long long len = 0;
  CutUnit* const cuts = reinterpret_cast<CutUnit*>(a.ws + static_cast<size_t>(F::BLOCKS) * 2 * F::PART);
  if constexpr (CLUSTER) {
    const int unit = blockIdx.x / kCluster, rank = blockIdx.x % kCluster;
    cc.b = unit / c.Hkv;
    cc.h = unit - cc.b * c.Hkv;
    cc.rt = 0;
    cc.s = Ln::seq(c, a, cc.b);
    cc.ntiles = cc.s.nrt > 0 ? Ln::tiles(a, cc.s, 0) : 0;
    x0 = cc.ntiles * rank / kCluster;
    x1 = cc.ntiles * (rank + 1) / kCluster;
    cc.t = static_cast<int>(x0);
  } else {
    long long mine, before;
    len = Ln::template length<kWarps * 32>(c, a, line, &mine, &before);
    x0 = cut<F::BLOCKS>(len, blockIdx.x);
    x1 = cut<F::BLOCKS>(len, blockIdx.x + 1);
    if (x0 >= x1) {
      if (threadIdx.x == 0) write_cut<F::BLOCKS, typename Ln::Cursor>(cuts, len, blockIdx.x, x0, x1, nullptr);
      return;
    }
    Ln::template find<kWarps * 32>(c, a, line, x0, mine, before, cc);
  }
  typename Ln::Cursor pc = cc;  // the next tile to copy

  uint8_t* const ring = smem + warp * F::RING;
  float* const ml = reinterpret_cast<float*>(smem + kWarps * F::RING);      // [warps][ROWS][2]
  uint4* const qs = reinterpret_cast<uint4*>(ml + kWarps * ROWS * 2);       // [MT][NK][32], MT > 1
  float* const facs = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(qs) + F::QBYTES);  // [ROWS]
  float* const state = facs + ROWS;  // CLUSTER: this block's state, PART floats
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

  // Fragments of row tile mt of the unit at cc, rows g and g + 8: element pairs
  // of 16-bit caches in the order of the matrix instruction; for 8-bit caches
  // a lane's share of a row is D / 4 neighbouring elements, those that it reads
  // of a key's codes, four to a k-step.  f: the rows' factors of the scores.
  auto load_q = [&](int mt, uint32_t (&qf)[NK][4], float (&f)[2]) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = cc.rt * ROWS + mt * 16 + g + 8 * e;
      const int t = static_cast<int>(a.g_div.div(r));
      const bool has = t < cc.s.q;
      f[e] = a.scale_log2;
      const T* p = static_cast<const T*>(a.q);
      if (has) p += cc.b * a.qs[0] + static_cast<long long>(cc.h * a.G + (r - t * a.G)) * a.qs[1] + t * a.qs[2];
      if constexpr (CT == kCache16) {
        const uint32_t* p32 = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) {
          qf[kk][e] = has ? __ldg(p32 + kk * 8 + cq) : 0u;
          qf[kk][2 + e] = has ? __ldg(p32 + kk * 8 + 4 + cq) : 0u;
        }
      } else {
        const uint2* p64 = reinterpret_cast<const uint2*>(p + cq * (D / 4));
        uint32_t top = 0;
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) {
          const uint2 w = has ? __ldg(p64 + kk) : make_uint2(0u, 0u);
          qf[kk][e] = w.x;
          qf[kk][2 + e] = w.y;
          if constexpr (BF) {
            top = max(top, max(w.x & 0x7fffu, (w.x >> 16) & 0x7fffu));
            top = max(top, max(w.y & 0x7fffu, (w.y >> 16) & 0x7fffu));
          }
        }
        if constexpr (BF) {
          // bf16 -> fp16 with the row's largest magnitude brought to [1, 2) by
          // a power of two: the elements keep their 8 bits down to 2^-14 of it
          // and are rounded to 2^-25 of it below
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          int ex = static_cast<int>(top >> 7);      // biased exponent
          ex = ex < 1 ? 1 : (ex > 253 ? 253 : ex);  // zero rows, infinities: some finite power
          const float up = __uint_as_float(static_cast<uint32_t>(254 - ex) << 23);
          f[e] *= __uint_as_float(static_cast<uint32_t>(ex) << 23);
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
  };

  if (x0 < x1) look_up();
#pragma unroll
  for (int s = 0; s < F::STAGES; ++s) {
    if (x0 + s < x1) {
      copy_tile(s);
      Ln::next_tile(c, a, pc);
      if (x0 + s + 1 < x1) look_up();
    }
    cp_async_commit();
  }

  // (behind the first loads: its divisions take as long)
  if constexpr (!CLUSTER) {
    if (threadIdx.x == 32) write_cut<F::BLOCKS>(cuts, len, blockIdx.x, x0, x1, &cc);
  }

  uint32_t qf[MT == 1 ? NK : 1][4];
  float f1[2];  // MT == 1: the rows' score factors
  float oa[MT][D / 8][4];
  float m[MT][2], l[MT][2];
  bool fresh = true;
  bool from_start = false;  // the piece holds its unit's first tile
  int slot = 0;
  for (long long x = x0; x < x1; ++x) {
    if (fresh) {
      fresh = false;
      from_start = cc.t == 0;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        m[mt][0] = m[mt][1] = -INFINITY;
        l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) oa[mt][j][0] = oa[mt][j][1] = oa[mt][j][2] = oa[mt][j][3] = 0.f;
      }
      if constexpr (MT == 1) {
        load_q(0, qf, f1);
      } else {  // warp i brings row tile i
        if (warp < MT) {
          uint32_t w[NK][4];
          load_q(warp, w, f1);
#pragma unroll
          for (int kk = 0; kk < NK; ++kk) qs[(warp * NK + kk) * 32 + lane] = make_uint4(w[kk][0], w[kk][1], w[kk][2], w[kk][3]);
          if (cq == 0) {
            facs[warp * 16 + g] = f1[0];
            facs[warp * 16 + g + 8] = f1[1];
          }
        }
        __syncthreads();
      }
    }
    auto q_frag = [&](int mt, int kk, uint32_t (&w)[4]) {
      if constexpr (MT == 1) {
        w[0] = qf[kk][0], w[1] = qf[kk][1], w[2] = qf[kk][2], w[3] = qf[kk][3];
      } else {
        const uint4 v = qs[(mt * NK + kk) * 32 + lane];
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
      }
    };

    cp_async_wait<F::STAGES - 1>();
    __syncwarp();
    const uint32_t ks_a = ring_a + slot * (F::SLOT + F::SCALES), vs_a = ks_a + KW * F::RB, sc_a = ks_a + F::SLOT;
    const int n0 = cc.t * TK + warp * KW;          // this warp's first key
    const int past = cc.s.kv - cc.s.q;             // keys every new token sees
    if (n0 < cc.s.kv) {
      float s[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < NT; ++j) s[mt][j][0] = s[mt][j][1] = s[mt][j][2] = s[mt][j][3] = 0.f;
      if constexpr (CT == kCache16) {
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) {
          uint32_t b[KW / 16][4];
#pragma unroll
          for (int p = 0; p < KW / 16; ++p) {
            const int r = p * 16 + ((lane >> 4) << 3) + (lane & 7);
            ldsm_x4(ks_a + r * F::RB + swz<CT, D>(r, kk * 2 + ((lane >> 3) & 1)) * 16, b[p]);
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t q[4];
            q_frag(mt, kk, q);
#pragma unroll
            for (int p = 0; p < KW / 16; ++p) {
              mma16816<MBF>(s[mt][2 * p], q, b[p][0], b[p][1]);
              mma16816<MBF>(s[mt][2 * p + 1], q, b[p][2], b[p][3]);
            }
          }
        }
      } else {
        // this lane's key: its value scale's log2 and the square root of 2^kSumUp /
        // scale take its place
        {
          float vscale;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vscale) : "r"(sc_a + KW * 4 + lane * 4) : "memory");
          if constexpr (!BF) {
            float kscale;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(kscale) : "r"(sc_a + lane * 4) : "memory");
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(sc_a + lane * 4), "f"(kscale * a.scale_log2) : "memory");
          }
          // no scale (a row past the end, or of a page that the cache does not
          // have) stands for a value of zero; the scores of a key whose value's
          // scale is NaN, or negative, are NaN, and its factor must not reach other
          // rows' sums
          vscale = vscale >= 0.f ? fmaxf(vscale, kMinScale) : __uint_as_float(0x7fc00000u);
          const float lsv = lg2(vscale);
          const float root = vscale == vscale ? ex2(0.5f * (kSumUp - lsv)) : 0.f;
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(sc_a + KW * 4 + lane * 4), "f"(lsv) : "memory");
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(sc_a + KW * 8 + lane * 4), "f"(root) : "memory");
          __syncwarp();
        }
        constexpr int PB = D / 4;  // bytes of a key's row per lane
        constexpr int PL = PB > 16 ? 16 : PB;
#pragma unroll
        for (int q = 0; q < PB / PL; ++q) {
          uint32_t w[NT][PL / 4];
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const int r = j * 8 + g, byte = cq * PB + q * PL;
            lds_bytes<PL>(ks_a + r * F::RB + swz<CT, D>(r, byte / 16) * 16 + (byte & 15), w[j]);
          }
#pragma unroll
          for (int i = 0; i < PL / 4; ++i) {
            uint32_t b[NT][2];
#pragma unroll
            for (int j = 0; j < NT; ++j) code4_to_f16<CT>(w[j][i], b[j][0], b[j][1]);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              uint32_t qq[4];
              q_frag(mt, q * (PL / 4) + i, qq);
#pragma unroll
              for (int j = 0; j < NT; ++j) mma16816<false>(s[mt][j], qq, b[j][0], b[j][1]);
            }
          }
        }
        // score scales, and each key's value scale in the exponent
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const float2 kx = lds_f2(sc_a + (j * 8 + 2 * cq) * 4), vx = lds_f2(sc_a + KW * 4 + (j * 8 + 2 * cq) * 4);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float2 k2 = kx;  // fp16 queries: the factor is in it already
              if constexpr (BF) {
                float f;
                if constexpr (MT == 1) f = f1[e];
                else f = facs[mt * 16 + g + 8 * e];
                k2 = fmul2(make_float2(f, f), kx);
              }
              const float2 t = ffma2(make_float2(s[mt][j][2 * e], s[mt][j][2 * e + 1]), k2, vx);
              s[mt][j][2 * e] = t.x, s[mt][j][2 * e + 1] = t.y;
            }
          }
        }
      }

      // keys behind the end, and new tokens that a row must not see
      const bool masked = n0 + KW > past;
      auto sees = [&](int t, int n) {  // new token t, key n
        const int d = n - past;
        if (t >= cc.s.q || n >= cc.s.kv) return false;
        return d < 0 || (a.tree ? __ldg(a.tree + cc.b * a.tree_b + t * a.tree_t + d) != 0 : d <= t);
      };
      if (masked) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int t = static_cast<int>(a.g_div.div(cc.rt * ROWS + mt * 16 + g + 8 * e));  // new token of the row
#pragma unroll
            for (int j = 0; j < NT; ++j) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                if (!sees(t, n0 + j * 8 + 2 * cq + i)) s[mt][j][2 * e + i] = -INFINITY;
              }
            }
          }
        }
      }

      uint32_t pf[MT][KW / 16][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        // running maximum, raised only when a score passes it by 2^8
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mx[0] = fmax3(mx[0], s[mt][j][0], s[mt][j][1]);
          mx[1] = fmax3(mx[1], s[mt][j][2], s[mt][j][3]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
        }
        if constexpr (CT == kCache16) mx[0] *= a.scale_log2, mx[1] *= a.scale_log2;
        if (__any_sync(0xffffffffu,
                       mx[0] > m[mt][0] + kRescaleThreshold || mx[1] > m[mt][1] + kRescaleThreshold)) {
          float al[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mn = fmaxf(m[mt][e], mx[e]);
            al[e] = mn == -INFINITY ? 1.f : ex2(m[mt][e] - mn);
            if constexpr (CT == kCache16) l[mt][e] *= al[e];
            else l[mt][e] = mn == -INFINITY ? l[mt][e] : lower_sum(l[mt][e], m[mt][e] - mn);
            m[mt][e] = mn;
            al[e] = keep_infinite(al[e]);
          }
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            oa[mt][j][0] *= al[0];
            oa[mt][j][1] *= al[0];
            oa[mt][j][2] *= al[1];
            oa[mt][j][3] *= al[1];
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float ref = m[mt][e] == -INFINITY ? 0.f : -m[mt][e];
          const float2 ref2 = make_float2(ref, ref), sc2 = make_float2(a.scale_log2, a.scale_log2);
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            float2 t = make_float2(s[mt][j][2 * e], s[mt][j][2 * e + 1]);
            if constexpr (CT == kCache16) {
              t = ffma2(t, sc2, ref2);
              t = make_float2(ex2(t.x), ex2(t.y));
              sum = fadd2(sum, t);
            } else {
              t = ffma2(t, make_float2(0.5f, 0.5f), make_float2(0.5f * ref, 0.5f * ref));
              t = make_float2(ex2(t.x), ex2(t.y));
              const float2 x = fmul2(t, lds_f2(sc_a + KW * 8 + (j * 8 + 2 * cq) * 4));
              sum = ffma2(x, x, sum);
              t = fmul2(t, t);
            }
            s[mt][j][2 * e] = t.x, s[mt][j][2 * e + 1] = t.y;
          }
          l[mt][e] += sum.x + sum.y;
        }
#pragma unroll
        for (int p = 0; p < KW / 16; ++p) {
          pf[mt][p][0] = pack2<MBF>(s[mt][2 * p][0], s[mt][2 * p][1]);
          pf[mt][p][1] = pack2<MBF>(s[mt][2 * p][2], s[mt][2 * p][3]);
          pf[mt][p][2] = pack2<MBF>(s[mt][2 * p + 1][0], s[mt][2 * p + 1][1]);
          pf[mt][p][3] = pack2<MBF>(s[mt][2 * p + 1][2], s[mt][2 * p + 1][3]);
        }
      }

      if constexpr (CT == kCache16) {
        // A new token's value may hold infinities or NaN that some rows must
        // not see, and 0 * NaN is NaN in the product: such elements are added
        // to the rows that do see them here, however small their weight, and
        // taken out of the tile.
        if (masked) {
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
              bool see[MT][2];
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  see[mt][e] = sees(static_cast<int>(a.g_div.div(cc.rt * ROWS + mt * 16 + g + 8 * e)), n0 + r);
#pragma unroll
              for (int j = 0; j < D / 8; ++j) {
                uint32_t w[1];
                lds_bytes<4>(vs_a + r * F::RB + swz<CT, D>(r, j) * 16 + cq * 4, w);
                const T* h = reinterpret_cast<const T*>(w);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const float v = static_cast<float>(h[i]);
                  if ((__float_as_uint(v) & 0x7f800000u) == 0x7f800000u) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                      if (see[mt][0]) oa[mt][j][i] += v;
                      if (see[mt][1]) oa[mt][j][2 + i] += v;
                    }
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
          const int r = p * 16 + (((lane >> 3) & 1) << 3) + (lane & 7);
#pragma unroll
          for (int dp = 0; dp < D / 16; ++dp) {
            uint32_t b[4];
            ldsm_x4_t(vs_a + r * F::RB + swz<CT, D>(r, dp * 2 + (lane >> 4)) * 16, b);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma16816<MBF>(oa[mt][2 * dp], pf[mt][p], b[0], b[1]);
              mma16816<MBF>(oa[mt][2 * dp + 1], pf[mt][p], b[2], b[3]);
            }
          }
        }
      } else {
        // Accumulator tile j's column n is value element n * (D / 8) + j: a
        // lane then reads D / 8 neighbouring codes of its four keys.
        constexpr int VB = D / 8;
#pragma unroll
        for (int p = 0; p < KW / 16; ++p) {
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
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma16816<false>(oa[mt][q * 4 + hh * 2], pf[mt][p], a0, b0);
                mma16816<false>(oa[mt][q * 4 + hh * 2 + 1], pf[mt][p], a1, b1);
              }
            }
          }
        }
      }
    }

    const bool last = cc.t + 1 == cc.ntiles;
    if (last || x + 1 == x1) {
      // ------------------------------------- end of the piece: join the warps
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[mt][e] += __shfl_xor_sync(0xffffffffu, l[mt][e], 1);
          l[mt][e] += __shfl_xor_sync(0xffffffffu, l[mt][e], 2);
          if (cq == 0) {
            float* p = ml + (warp * ROWS + mt * 16 + g + 8 * e) * 2;
            p[0] = m[mt][e];
            p[1] = l[mt][e];
          }
        }
      }
      const bool whole = !CLUSTER && from_start && last;
      float* const part =
          CLUSTER ? state : a.ws + (static_cast<size_t>(blockIdx.x) * 2 + (x - x0 > cc.t ? 1 : 0)) * F::PART;
      uint8_t* const st = ring + slot * (F::SLOT + F::SCALES);  // the tile this warp has just used
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = g + 8 * e;
          float* const row = reinterpret_cast<float*>(st) + r * D;
          if constexpr (CT == kCache16) {
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
              *reinterpret_cast<float2*>(row + oswz<D>(r, 2 * j + (cq >> 1)) * 4 + (cq & 1) * 2) =
                  make_float2(oa[mt][j][2 * e], oa[mt][j][2 * e + 1]);
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
              for (int j = 0; j < D / 8; j += 2) {
                const int d = (2 * cq + i) * (D / 8) + j;
                *reinterpret_cast<float2*>(row + oswz<D>(r, d >> 2) * 4 + (d & 3)) =
                    make_float2(oa[mt][j][2 * e + i], oa[mt][j + 1][2 * e + i]);
              }
            }
          }
        }
        __syncthreads();
        const int r = threadIdx.x >> 3, sub = threadIdx.x & 7;  // 16 rows, 8 threads each
        const int ur = mt * 16 + r;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, ml[(w * ROWS + ur) * 2]);
        float f[kWarps], ll = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          f[w] = mm == -INFINITY ? 0.f : ex2(ml[(w * ROWS + ur) * 2] - mm);
          const float wl = ml[(w * ROWS + ur) * 2 + 1];
          // a NaN sum stays one where no score was a number
          if constexpr (CT == kCache16) ll += (mm == -INFINITY ? 1.f : f[w]) * wl;
          else ll += mm == -INFINITY ? wl : lower_sum(wl, ml[(w * ROWS + ur) * 2] - mm);
          f[w] = keep_infinite(f[w]);
        }
        const int qr = cc.rt * ROWS + ur;
        const int t = static_cast<int>(a.g_div.div(qr)), hq = cc.h * a.G + (qr - t * a.G);
        const bool real = t < cc.s.q;
        float norm = 1.f;
        if (whole) norm = sum_norm<CT>(ll);
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
                uint2 o;
                o.x = pack2<BF>(v[0] * norm, v[1] * norm);
                o.y = pack2<BF>(v[2] * norm, v[3] * norm);
                *reinterpret_cast<uint2*>(out + ch * 4) = o;
              }
            } else {
              reinterpret_cast<float4*>(part + ur * D)[ch] = make_float4(v[0], v[1], v[2], v[3]);
            }
          }
        }
        if (sub == 0) {
          if (!whole) {
            part[ROWS * D + 2 * ur] = mm;
            part[ROWS * D + 2 * ur + 1] = ll;
          } else if (real) {
            a.lse[(static_cast<long long>(cc.b) * a.Hq + hq) * c.T + t] = row_lse<CT>(mm, ll);
          }
        }
        __syncthreads();
      }
      fresh = true;
    } else {
      __syncwarp();
    }
    if (x + F::STAGES < x1) {
      copy_tile(slot);
      Ln::next_tile(c, a, pc);
      if (x + F::STAGES + 1 < x1) look_up();
    }
    cp_async_commit();
    slot = slot + 1 == F::STAGES ? 0 : slot + 1;
    if (!CLUSTER || x + 1 < x1) Ln::next_tile(c, a, cc);
  }

  if constexpr (CLUSTER) {
    if (x0 >= x1) {  // no tiles: an empty state
      for (int i = threadIdx.x; i < ROWS * D; i += kWarps * 32) state[i] = 0.f;
      for (int i = threadIdx.x; i < ROWS; i += kWarps * 32) {
        state[ROWS * D + 2 * i] = -INFINITY;
        state[ROWS * D + 2 * i + 1] = 0.f;
      }
    }
    cluster_sync_all();
    // rows rank, rank + 8, ... of the unit, D / 4 threads a row
    const int rank = static_cast<int>(cluster_ctarank());
    constexpr int TPR = D / 4, RPP = kWarps * 32 / TPR;
    const int ch = threadIdx.x % TPR;
    for (int k = threadIdx.x / TPR; k < ROWS / kCluster; k += RPP) {
      const int r = rank + kCluster * k;
      const int t = static_cast<int>(a.g_div.div(r)), hq = cc.h * a.G + (r - t * a.G);
      if (t >= cc.s.q) continue;
      const uint32_t at = smem_u32(state);
      float pm[kCluster], pl[kCluster];
      float4 y[kCluster];
#pragma unroll
      for (int p = 0; p < kCluster; ++p) {
        const uint32_t peer = mapa_shared(at, p);
        pm[p] = ld_cluster_f32(peer + (ROWS * D + 2 * r) * 4);
        pl[p] = ld_cluster_f32(peer + (ROWS * D + 2 * r + 1) * 4);
        y[p] = ld_cluster_v4(peer + (r * D + ch * 4) * 4);
      }
      float mm = -INFINITY;
#pragma unroll
      for (int p = 0; p < kCluster; ++p) mm = fmaxf(mm, pm[p]);
      float ll = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int p = 0; p < kCluster; ++p) {
        float f = pm[p] == -INFINITY ? 0.f : ex2(pm[p] - mm);
        // a NaN sum stays one where no score was a number
        ll += mm == -INFINITY ? pl[p] : CT == kCache16 ? pl[p] * f : lower_sum(pl[p], pm[p] - mm);
        f = keep_infinite(f);
        v[0] = fmaf(y[p].x, f, v[0]);
        v[1] = fmaf(y[p].y, f, v[1]);
        v[2] = fmaf(y[p].z, f, v[2]);
        v[3] = fmaf(y[p].w, f, v[3]);
      }
      const float norm = sum_norm<CT>(ll);
      uint2 o;
      o.x = pack2<BF>(v[0] * norm, v[1] * norm);
      o.y = pack2<BF>(v[2] * norm, v[3] * norm);
      *reinterpret_cast<uint2*>(static_cast<T*>(a.o) + cc.b * a.os[0] + hq * a.os[1] + t * a.os[2] + ch * 4) = o;
      if (ch == 0) a.lse[(static_cast<long long>(cc.b) * a.Hq + hq) * c.T + t] = row_lse<CT>(mm, ll);
    }
    cluster_sync_all();  // the peers have read this block's state
  }
}

// Joins the partial states of the units that block borders cut: block (i, y)
// joins rows 8 y .. 8 y + 7 of the unit that border i + 1 is the first to cut.
// Two warps share a row.  A unit can have hundreds of parts (one long sequence
// over all blocks), so that everything but the sum of the accumulators runs
// over the parts in parallel, and that sum has eight loads in flight.
template <typename T, int CT, int D, int MT>
__global__ void __launch_bounds__(512) attn_cache_join_kernel(CacheArgs c, CacheAttnArgs a) {
  constexpr bool BF = DT<T>::bf16;
  constexpr int VEC = D >= 128 ? 4 : (D >= 64 ? 2 : 1);  // elements per lane
  using F = Cfg<CT, D, MT>;
  constexpr int ROWS = F::ROWS;
  __shared__ int slots[F::BLOCKS];
  __shared__ float2 ml[8][2][F::BLOCKS];  // per row and warp: the parts' m and l, then their factors
  __shared__ float other[8][D + 1];
  wait_for_main_kernel();  // every block: the next kernel in the stream may start when this one has ended
  const CutUnit u = reinterpret_cast<const CutUnit*>(a.ws + static_cast<size_t>(F::BLOCKS) * 2 * F::PART)[blockIdx.x + 1];
  const int parts = u.parts;
  if (parts == 0 || static_cast<int>(blockIdx.y) * 8 + u.rt * ROWS >= u.q * a.G) return;
  const int wrow = threadIdx.x >> 6, half = (threadIdx.x >> 5) & 1, lane = threadIdx.x & 31;
  const int r = blockIdx.y * 8 + wrow;
  auto part = [&](int slot) { return a.ws + static_cast<size_t>(slot) * F::PART; };
  const bool lane_on = lane * VEC < D;
  auto load = [&](int i, float (&y)[VEC]) {
    if (slots[i] < 0) {  // a block without a piece
#pragma unroll
      for (int e = 0; e < VEC; ++e) y[e] = 0.f;
      return;
    }
    const float* p = part(slots[i]) + r * D + lane * VEC;
    if constexpr (VEC == 4) {
      const float4 w = __ldcg(reinterpret_cast<const float4*>(p));
      y[0] = w.x, y[1] = w.y, y[2] = w.z, y[3] = w.w;
    } else if constexpr (VEC == 2) {
      const float2 w = __ldcg(reinterpret_cast<const float2*>(p));
      y[0] = w.x, y[1] = w.y;
    } else {
      y[0] = __ldcg(p);
    }
  };
  // Maxima and sums, a part per lane, by both warps of a row; kept in shared
  // memory between the two passes.
  for (int i = threadIdx.x; i < parts; i += 512) slots[i] = part_slot<F::BLOCKS>(u, i);
  __syncthreads();
  float2* const mls = ml[wrow][half];
  float mm = -INFINITY;
  for (int i = lane; i < parts; i += 32) {
    const float2 v = slots[i] < 0 ? make_float2(-INFINITY, 0.f)
                                  : __ldcg(reinterpret_cast<const float2*>(part(slots[i]) + ROWS * D + 2 * r));
    mls[i] = v;
    mm = fmaxf(mm, v.x);
  }
  // the first parts' accumulators are on their way meanwhile
  constexpr int AHEAD = 8;
  float y[AHEAD][VEC] = {};
  if (lane_on) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (half + 2 * k < parts) load(half + 2 * k, y[k]);
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, s));
  float ll = 0.f;
  for (int i = lane; i < parts; i += 32) {
    const float2 v = mls[i];
    const float f = v.x == -INFINITY ? 0.f : ex2(v.x - mm);
    // a NaN sum stays one where no score was a number
    ll += mm == -INFINITY ? v.y : CT == kCache16 ? v.y * f : lower_sum(v.y, v.x - mm);
    mls[i].x = keep_infinite(f);
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, s);
  __syncwarp();
  float v[VEC] = {};
  if (lane_on) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const float f = half + 2 * k < parts ? mls[half + 2 * k].x : 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = fmaf(y[k][e], f, v[e]);
    }
    for (int i0 = half + 2 * AHEAD; i0 < parts; i0 += 2 * AHEAD) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (i0 + 2 * k < parts) load(i0 + 2 * k, y[k]);
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const float f = i0 + 2 * k < parts ? mls[i0 + 2 * k].x : 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (i0 + 2 * k < parts) v[e] = fmaf(y[k][e], f, v[e]);
      }
    }
    if (half) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) other[wrow][lane * VEC + k] = v[k];
    }
  }
  __syncthreads();
  if (half) return;
  const int qr = u.rt * ROWS + r;
  const int t = static_cast<int>(a.g_div.div(qr)), hq = u.h * a.G + (qr - t * a.G);
  if (t >= u.q) return;
  const float norm = sum_norm<CT>(ll);
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
  if (lane == 0) a.lse[(static_cast<long long>(u.b) * a.Hq + hq) * c.T + t] = row_lse<CT>(mm, ll);
}

// Whether each unit gets a cluster: few units, of sequences that cannot be long
// as far as their page tables go (the lengths are on the device).  Measured, one
// token a sequence, 4 query heads per key head of 128, us of a replayed graph, cut
// line / clusters:
//   tokens         1024          4096          8192          16384
//   bf16,  1 unit  25.7 / 11.4   29.8 / 17.5   29.8 / 25.7   31.9 / 40.1
//   bf16,  8       17.5 / 13.4   19.6 / 17.5   21.6 / 25.7   27.8 / 42.1
//   bf16, 32       19.6 / 13.4   27.7 / 23.7   38.0 / 31.9   56.4 / 52.4
//   int8,  8       19.6 / 13.4   19.6 / 17.5   21.7 / 21.6   25.8 / 29.8
//   int8, 32       19.6 / 13.4   25.7 / 19.6   31.9 / 25.7   42.1 / 38.0
// (where there are more units clusters would win longer, but only for
// sequences of about one length).
template <typename F>
inline bool few_units(const CacheArgs& c, const CacheAttnArgs& a) {
  return static_cast<long long>(a.G) * c.T <= F::ROWS && static_cast<long long>(c.B) * c.Hkv <= F::BLOCKS / kCluster &&
         c.capacity <= 8192 && static_cast<long long>(c.capacity) * F::RB <= 4096 * 256;
}

template <typename T, int CT, int D, int MT>
cudaError_t run_rows(const CacheArgs& c, const CacheAttnArgs& a, cudaStream_t s) {
  static std::atomic<bool> done[kMaxDevices];
  using F = Cfg<CT, D, MT>;
  if constexpr (MT <= 2) {
    if (few_units<F>(c, a)) {
      static std::atomic<bool> cdone[kMaxDevices];
      auto* kern = attn_cache_kernel<T, CT, D, MT, true>;
      constexpr int smem = F::SMEM + F::PART * 4;
      cudaError_t e = smem_attr_once(kern, smem, cdone);
      if (e != cudaSuccess) return e;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(c.B * c.Hkv * kCluster);
      cfg.blockDim = dim3(kWarps * 32);
      cfg.dynamicSmemBytes = smem;
      cfg.stream = s;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = kCluster;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      prof_begin("attn_cache_cluster", s);
      e = cudaLaunchKernelEx(&cfg, kern, c, a);
      prof_end(s);
      return e;
    }
  }
  auto* kern = attn_cache_kernel<T, CT, D, MT, false>;
  cudaError_t e = smem_attr_once(kern, F::SMEM, done);
  if (e != cudaSuccess) return e;
  prof_begin("attn_cache", s);
  kern<<<F::BLOCKS, kWarps * 32, F::SMEM, s>>>(c, a);
  prof_end(s);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  prof_begin("attn_cache_join", s);
  e = launch_join(attn_cache_join_kernel<T, CT, D, MT>, dim3(F::BLOCKS - 1, (min(a.G * c.T, F::ROWS) + 7) / 8), 512, s, c, a);
  prof_end(s);
  return e;
}

template <typename T, int CT, int D>
cudaError_t run_mt(int mt, const CacheArgs& c, const CacheAttnArgs& a, cudaStream_t s) {
  if (mt == 1) return run_rows<T, CT, D, 1>(c, a, s);
  if (mt == 2) return run_rows<T, CT, D, 2>(c, a, s);
  if constexpr (D <= 64) {  // (MT x D / 2 accumulators a lane)
    if (mt == 3) return run_rows<T, CT, D, 3>(c, a, s);
  }
  if constexpr (D <= 32) {
    if (mt == 4) return run_rows<T, CT, D, 4>(c, a, s);
  }
  return cudaErrorInvalidValue;
}
template <typename T, int CT>
cudaError_t run_d(int D, int mt, const CacheArgs& c, const CacheAttnArgs& a, cudaStream_t s) {
  switch (D) {
    case 16: return run_mt<T, CT, 16>(mt, c, a, s);
    case 32: return run_mt<T, CT, 32>(mt, c, a, s);
    case 64: return run_mt<T, CT, 64>(mt, c, a, s);
    case 128: return run_mt<T, CT, 128>(mt, c, a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace
}  // namespace ta
