// Forward attention of packed sequences with shared key heads (sm_103a).
//
//   O_i = sum_j p_ij V_j / sum_j p_ij,  p_ij = exp(c q_i . k_j - m_i),  L_i = m_i + ln sum_j p_ij
//
// over the keys j of the query's own sequence, causal ones up to i + n_k - n_q.
//
// A CTA works on two 128-row query tiles of one key head (packed.cuh: TB tokens x G
// heads each) that share every K/V tile: warps 0-3 and 4-7 run their softmax, one
// thread a row, warp 8 feeds Q and the K and V rings by TMA, warp 9 issues the
// MMAs, alternating between the tiles so that one's softmax runs beside the other's
// products, and warps 10 and 11 look after the key tiles that some row sees only in part:
//   * the rows behind the sequence's keys belong to another sequence or to
//     nobody, and a weight of zero times an infinity there would be NaN:
//     they become zeros;
//   * so would an infinity or a NaN in the value of a key that only some rows
//     see: such elements become zeros for the product, and the rows that see them
//     get them back from memory at the end.
// They follow every V tile between its arrival and its product.  A CTA takes
// over the units of CTAs that have not started (UnitRing); the rings run on
// from one unit to the next.
#include <cstdio>

#include "launch.h"
#include "packed.cuh"

namespace ta {

namespace {

constexpr int kThreads = 384;
constexpr int kProducer = 8, kMma = 9, kCare = 10;  // warps; kCare and the one behind it
template <int D>
struct PfCfg {
  static constexpr int TILE = (D / 64) * kBM * 128;
  static constexpr int KST = D == 128 ? 3 : 4;  // K ring depth
  static constexpr int VST = D == 128 ? 2 : 4;  // V ring depth
  static constexpr int QB = D == 128 ? 1 : 2;   // pairs of Q tiles (their memory takes O on its way out)
  static constexpr int SMEM = (2 * QB + KST + VST) * TILE + 1024;
  static_assert(SMEM + 2048 <= kSmemMax, "tiles do not fit in shared memory");
};

template <int D>
__device__ __forceinline__ void load_rows(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int c1, int c2) {
#pragma unroll
  for (int kb = 0; kb < D / 64; ++kb) tma_load_3d(dst + kb * (kBM * 128), map, bar, kb * 64, c1, c2);
}

// d (+)= P V: P 128 x 128 (16-bit, TMEM, two a column), V 128 keys x D with D contiguous.
template <int D>
__device__ __forceinline__ void mma_pv(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_smem, uint32_t idesc, bool accumulate) {
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

// 0xffff in the halves of w that are infinities or NaN.
template <bool BF>
__device__ __forceinline__ uint32_t non_finite2(uint32_t w) {
  constexpr uint32_t E = BF ? 0x7f807f80u : 0x7c007c00u;
  return __vcmpeq2(w & E, E);
}

// What the roles derive from a unit.
struct Pair {
  int head, row, krow, n;   // key head, first token's row, first key's row, keys
  int left[2], n_t[2];      // of each tile: tokens from its first to the sequence's end, key tiles
  int off;                  // last key that the first token sees
  int causal, nt, t_part;   // key tiles; from t_part on some row sees a tile in part, or it ends behind the keys
  __device__ __forceinline__ Pair(const PackedUnit& u, int TB) {
    head = u.pad[1];
    causal = u.pad[0];
    row = u.row;
    krow = u.krow;
    n = u.n;
    off = u.off;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      left[w] = u.left - w * TB;
      n_t[w] = packed_key_tiles(min(left[w], TB), off + w * TB, n, causal);
    }
    nt = max(n_t[0], n_t[1]);
    t_part = n / kBN;
    if (causal) t_part = min(t_part, off < 0 ? 0 : (off + 1) / kBN);
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    packed_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                      const PackedArgs args) {
  using C = PfCfg<D>;
  constexpr bool BF = DT<T>::bf16;
  constexpr int KST = C::KST, VST = C::VST, QB = C::QB;

  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) UnitRing ring;
  __shared__ __align__(8) uint64_t bar_q[QB], bar_qfree[QB], bar_ofinal[QB];
  __shared__ __align__(8) uint64_t bar_k[KST], bar_kempty[KST], bar_v[VST], bar_vempty[VST], bar_care[VST];
  __shared__ __align__(8) uint64_t bar_s[2], bar_p[2], bar_o[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ int care_odd[VST][2];  // a V tile held non-finite values that only some rows see (by caring warp)
  __shared__ int unit_odd[2];       // any of unit i's did, at i % 2

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  PackedUnit first;
  if (!packed_unit(args, kPackedFwd, blockIdx.x, &first)) return;
  const int G = args.shape.G, TB = args.shape.TB;

  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto sQ = [&](int qb, int w) { return base + (2 * qb + w) * C::TILE; };
  auto sK = [&](int st) { return base + (2 * QB + st) * C::TILE; };
  auto sV = [&](int st) { return base + (2 * QB + KST + st) * C::TILE; };

  WaitCtl ctl{args.err, args.timeout_ns, &abort_flag};
  if (threadIdx.x == 0) {
    abort_flag = 0;
    ring_init(&ring, 8 + 1 + 3 + 1, first);  // softmax warps, MMA, three producing lanes, warp 10
    for (int q = 0; q < QB; ++q) {
      mbar_init(&bar_q[q], 1);
      mbar_init(&bar_qfree[q], 8);
      mbar_init(&bar_ofinal[q], 2);
    }
    for (int s = 0; s < KST; ++s) {
      mbar_init(&bar_k[s], 1);
      mbar_init(&bar_kempty[s], 1);
    }
    for (int s = 0; s < VST; ++s) {
      mbar_init(&bar_v[s], 1);
      mbar_init(&bar_vempty[s], 1);
      mbar_init(&bar_care[s], 2);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&bar_s[w], 1);
      mbar_init(&bar_p[w], 4);
      mbar_init(&bar_o[w], 1);
    }
    fence_mbar_init();
  }
  if (warp == kMma) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint32_t col_s[2] = {0u, 128u};
  const uint32_t col_o[2] = {256u, 256u + D};

  // registers: 384 x 168 at launch = 256 x 200 (softmax) + 128 x 104
  if (warp == kProducer) {
    // ---------------- TMA producer: lane 0 the K ring, lane 1 the V ring, lane 2 Q
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (lane < 3) {
      int issued = 0;  // tiles of the ring, or pairs of Q tiles, so far
      bool ok = true;
      const int depth = lane == 0 ? KST : VST;
      uint64_t* full = lane == 0 ? bar_k : bar_v;
      uint64_t* empty = lane == 0 ? bar_kempty : bar_vempty;
      const CUtensorMap* map = lane == 0 ? &tm_k : &tm_v;
      for (int i = 0;; ++i) {
        if (!ring_take(&ring, i, ctl)) break;
        const Pair p(ring_unit(&ring, i), TB);
        if (lane < 2) {
          for (int t = 0; t < p.nt; ++t, ++issued) {
            const int st = issued % depth;
            if (issued >= depth && !(ok = mbar_wait(&empty[st], ((issued / depth) - 1) & 1, ctl, kErrTimeoutMma))) break;
            mbar_expect_tx(&full[st], C::TILE);
            load_rows<D>(lane == 0 ? sK(st) : sV(st), map, &full[st], p.krow + t * kBN, p.head);
          }
        } else if (p.nt > 0) {
          const int qb = issued % QB;
          ok = issued < QB || mbar_wait(&bar_qfree[qb], ((issued / QB) - 1) & 1, ctl, kErrTimeoutSoftmax);
          if (ok) {
            const int tiles = p.left[1] > 0 ? 2 : 1;
            mbar_expect_tx(&bar_q[qb], tiles * (D / 64) * TB * G * 128);  // rows past a tile's TB x G are not loaded
            for (int w = 0; w < tiles; ++w) load_rows<D>(sQ(qb, w), &tm_q, &bar_q[qb], p.head * G, p.row + w * TB);
            ++issued;
          }
        }
        if (!ok) break;
        mbar_arrive(&ring.left[i & 1]);
      }
      // never leave a TMA write in flight behind an exit
      int zero = 0;
      WaitCtl drain{args.err, args.timeout_ns, reinterpret_cast<volatile int*>(&zero)};
      if (lane == 2) {
        for (int u = issued - QB > 0 ? issued - QB : 0; u < issued; ++u)
          mbar_wait(&bar_q[u % QB], (u / QB) & 1, drain, kErrTimeoutTma);
      } else {
        for (int t = issued - depth > 0 ? issued - depth : 0; t < issued; ++t)
          mbar_wait(&full[t % depth], (t / depth) & 1, drain, kErrTimeoutTma);
      }
    }
  } else if (warp == kMma) {
    // --------------------------------------------------------- MMA issuer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    constexpr uint32_t idesc_qk = idesc_f16(kBM, kBN, BF, false, false);
    constexpr uint32_t idesc_pv = idesc_f16(kBM, D, BF, false, true);
    int ik = 0, iv = 0, uq = 0;  // K tiles, V tiles and units with keys so far
    int np[2] = {0, 0};          // tiles of each group so far
    bool ok = true;
    for (int i = 0;; ++i) {
      if (!__all_sync(0xffffffffu, ring_take(&ring, i, ctl))) break;
      const Pair p(ring_unit(&ring, i), TB);
      if (p.nt > 0) {
        const int qb = uq % QB;
        const uint32_t aQ[2] = {smem_u32(sQ(qb, 0)), smem_u32(sQ(qb, 1))};
        int odd = 0;
        ok = warp_wait(&bar_q[qb], (uq / QB) & 1, ctl, kErrTimeoutTma) &&
             warp_wait(&bar_k[ik % KST], (ik / KST) & 1, ctl, kErrTimeoutTma);
        if (ok) {
          tc_fence_after();
          const int sk = ik % KST;
#pragma unroll
          for (int w = 0; w < 2; ++w)
            if (p.n_t[w] > 0) {
              mma_abT<D>(tmem + col_s[w], aQ[w], smem_u32(sK(sk)), idesc_qk);
              commit_el(&bar_s[w]);
            }
          commit_el(&bar_kempty[sk]);
          ++ik;
        }
        for (int t = 0; ok && t < p.nt; ++t, ++iv) {
          const int sv = iv % VST;
          const int sk1 = ik % KST;
          if (!(ok = warp_wait(&bar_care[sv], (iv / VST) & 1, ctl, kErrTimeoutTma))) break;
          if (t >= p.t_part) odd |= care_odd[sv][0] | care_odd[sv][1];
          const bool next = t + 1 < p.nt;
          if (next && !(ok = warp_wait(&bar_k[sk1], (ik / KST) & 1, ctl, kErrTimeoutTma))) break;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (t < p.n_t[w]) {
              if (!(ok = warp_wait(&bar_p[w], np[w] & 1, ctl, kErrTimeoutSoftmax))) break;
              ++np[w];
              tc_fence_after();
              mma_pv<D>(tmem + col_o[w], tmem + col_s[w], smem_u32(sV(sv)), idesc_pv, t > 0);
              commit_el(&bar_o[w]);
            }
            if (next && t + 1 < p.n_t[w]) {
              mma_abT<D>(tmem + col_s[w], aQ[w], smem_u32(sK(sk1)), idesc_qk);
              commit_el(&bar_s[w]);
            }
          }
          if (!ok) break;
          commit_el(&bar_vempty[sv]);
          if (next) {
            commit_el(&bar_kempty[sk1]);
            ++ik;
          }
        }
        if (!ok) break;
        commit_el(&bar_ofinal[qb]);
        if (lane == 0) {
          unit_odd[i & 1] = odd;
          mbar_arrive(&bar_ofinal[qb]);  // (with the flag behind it)
        }
        ++uq;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.left[i & 1]);
    }
  } else if (warp >= kCare) {
    // ------------------ value tiles that some row sees in part; warp 11: units ahead
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    const int half = warp - kCare;
    const int r0 = half * 64;  // each warp's half of the tile's rows
    RingAsker asker;
    if (half == 1 && lane == 0) asker.ask(&ring);
    int iv = 0;
    bool ok = true;
    for (int i = 0;; ++i) {
      if (!__all_sync(0xffffffffu, ring_take(&ring, i, ctl))) break;
      if (half == 1) {
        if (lane == 0) ok = asker.pass(&ring, args, kPackedFwd, i, ctl);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
      }
      const Pair p(ring_unit(&ring, i), TB);
      for (int t = 0; t < p.nt; ++t, ++iv) {
        const int sv = iv % VST;
        if (!(ok = warp_wait(&bar_v[sv], (iv / VST) & 1, ctl, kErrTimeoutTma))) break;
        if (t >= p.t_part) {
          const int valid = min(kBN, p.n - t * kBN);  // rows of the tile that are keys
          bool odd = false;
#pragma unroll
          for (int kb = 0; kb < D / 64; ++kb) {
            uint4* rows = reinterpret_cast<uint4*>(sV(sv) + kb * (kBM * 128) + r0 * 128);
            const int keys = min(max(valid - r0, 0), 64) * 8;  // 16-byte pieces
            for (int j = keys + lane; j < 64 * 8; j += 32) rows[j] = make_uint4(0u, 0u, 0u, 0u);
            if (p.causal) {
#pragma unroll 4
              for (int j = lane; j < keys; j += 32) {
                uint4 x = rows[j];
                const uint4 m = make_uint4(non_finite2<BF>(x.x), non_finite2<BF>(x.y), non_finite2<BF>(x.z),
                                           non_finite2<BF>(x.w));
                if (m.x | m.y | m.z | m.w) {
                  odd = true;
                  rows[j] = make_uint4(x.x & ~m.x, x.y & ~m.y, x.z & ~m.z, x.w & ~m.w);
                }
              }
            }
          }
          odd = __any_sync(0xffffffffu, odd);
          if (lane == 0) care_odd[sv][half] = odd;
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(&bar_care[sv]);
      }
      if (!ok) break;
      __syncwarp();
      if (half == 0 && lane == 0) mbar_arrive(&ring.left[i & 1]);
    }
    if (half == 1 && lane == 0) {
      int zero = 0;
      WaitCtl drain{args.err, args.timeout_ns, reinterpret_cast<volatile int*>(&zero)};
      asker.drain(&ring, drain);
    }
  } else {
    // ------------------------------- softmax / correction / epilogue (tile w)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int w = warp >> 2;
    const int r = threadIdx.x & 127;
    const int tok = static_cast<int>(args.g_div.div(r)), g = r - tok * G;  // of the tile
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t scol = w ? col_s[1] : col_s[0], ocol = w ? col_o[1] : col_o[0];
    int np = 0, uq = 0;  // tiles of this group, units with keys so far
    bool ok = true;
    for (int i = 0;; ++i) {
      if (!__all_sync(0xffffffffu, ring_take(&ring, i, ctl))) break;
      int n, sees, t_part;  // key tiles, last key of this row (the rest of the unit is read again behind the loop)
      {
        const Pair p(ring_unit(&ring, i), TB);
        n = w ? p.n_t[1] : p.n_t[0];
        sees = p.causal ? min(p.n - 1, p.off + w * TB + tok) : p.n - 1;
        t_part = p.t_part;
      }
      float m_ref = -INFINITY, l = 0.f;
      for (int t = 0; t < n; ++t, ++np) {
        if (!(ok = warp_wait(&bar_s[w], np & 1, ctl, kErrTimeoutMma))) break;
        tc_fence_after();
        uint32_t s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_x32(lane_addr + scol + 32 * c, TB_CHUNK(s, c));
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait(TB_CHUNK(s, c));
        float x[128];
#pragma unroll
        for (int j = 0; j < 128; ++j) x[j] = __uint_as_float(s[j]);
        if (t >= t_part) {
          const int lim = sees - t * kBN;
#pragma unroll
          for (int j = 0; j < 128; ++j)
            if (j > lim) x[j] = -INFINITY;
        }
        float mx8[8];  // eight three-input max chains of 16 scores each
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          mx8[k] = fmax3(x[k], x[8 + k], x[16 + k]);
#pragma unroll
          for (int j = 24; j < 120; j += 16) mx8[k] = fmax3(mx8[k], x[j + k], x[j + 8 + k]);
          mx8[k] = fmaxf(mx8[k], x[120 + k]);
        }
        const float mx = fmaxf(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(fmax3(mx8[3], mx8[4], mx8[5]), mx8[6], mx8[7]));
        const float m_new = fmaxf(m_ref, mx * args.scale_log2);
        bool resc = false;
        float alpha = 1.f;
        if (t == 0) {
          m_ref = m_new;
        } else if (m_new > m_ref + kRescaleThreshold) {
          resc = true;
          alpha = ex2(m_ref - m_new);
          m_ref = m_new;
        }
        const float neg_m = (m_ref == -INFINITY) ? 0.f : -m_ref;
        const float2 sc2 = make_float2(args.scale_log2, args.scale_log2);
        const float2 nm2 = make_float2(neg_m, neg_m);
        float2 rs2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 8; ++c) {  // 16 columns of S, 8 packed columns of P, at a time
          uint32_t pk[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 y = ffma2(make_float2(x[16 * c + 2 * e], x[16 * c + 2 * e + 1]), sc2, nm2);
            const float2 pr = make_float2(ex2(y.x), ex2(y.y));
            rs2[e & 3] = fadd2(rs2[e & 3], pr);
            pk[e] = pack2<BF>(pr.x, pr.y);
          }
          tmem_st_x8(lane_addr + scol + 8 * c, pk);
        }
        const float2 rsa = fadd2(fadd2(rs2[0], rs2[1]), fadd2(rs2[2], rs2[3]));
        l = l * alpha + (rsa.x + rsa.y);
        if (t > 0 && __any_sync(0xffffffffu, resc)) {
          if (!(ok = warp_wait(&bar_o[w], (np - 1) & 1, ctl, kErrTimeoutMma))) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld_x32(lane_addr + ocol + 32 * c, ov);
            tmem_ld_wait(ov);
#pragma unroll
            for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * alpha);
            tmem_st_x32(lane_addr + ocol + 32 * c, ov);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_p[w]);
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      const Pair p(ring_unit(&ring, i), TB);
      const int left = w ? p.left[1] : p.left[0];
      const int qb = uq % QB;
      if (p.nt > 0) {
        if (!(ok = warp_wait(&bar_ofinal[qb], (uq / QB) & 1, ctl, kErrTimeoutMma))) break;
        ++uq;
      }
      tc_fence_after();
      const int tokens = min(left, TB);  // (none: the sequence ends before this tile)
      if (tokens > 0) {
        const size_t qrow = static_cast<size_t>(p.row) + w * TB;
        if (tok < tokens)
          args.lse[(qrow + tok) * args.shape.Hq + p.head * G + g] =
              (n > 0 && l != 0.f) ? (m_ref + lg2(l)) * kLn2 : -INFINITY;
        T* const out = static_cast<T*>(args.o) + static_cast<long long>(qrow) * args.o_t + p.head * G * args.o_h;
        auto out_row = [&](int j) -> void* {
          if (j >= tokens * G) return nullptr;
          const int k = static_cast<int>(args.g_div.div(j));
          return out + k * args.o_t + (j - k * G) * args.o_h;
        };
        if (n == 0) {  // rows that see nothing
          const int c = args.dg >> 3;
          for (int j = r; j < tokens * G * c; j += 128) {
            const int row = j / c;
            static_cast<uint4*>(out_row(row))[j - row * c] = make_uint4(0u, 0u, 0u, 0u);
          }
        } else {
          const float inv_l = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
          // non-finite values that were taken out of this unit's tiles: this row's are added to O here
          const bool odd = p.causal && *reinterpret_cast<volatile int*>(&unit_odd[i & 1]) != 0;
          const uint32_t stage = smem_u32(sQ(qb, w));
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld_x32(lane_addr + ocol + 32 * c, ov);
            tmem_ld_wait(ov);
            float scale = inv_l;
            if (odd && tok < tokens && l > 0.f) {
              const int ng = chunk_groups(args.dg, 32 * c);
#pragma unroll
              for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * inv_l);
              for (int k = t_part * kBN; k <= min(sees, n * kBN - 1); ++k) {
                const T* vrow = static_cast<const T*>(args.v) + (static_cast<long long>(p.krow) + k) * args.vt +
                                p.head * args.vh + 32 * c;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  if (q >= ng) break;
                  const uint4 xv = __ldg(reinterpret_cast<const uint4*>(vrow) + q);
                  const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const uint32_t m = non_finite2<BF>(xs[e]);
                    if (!m) continue;
                    const uint32_t y = xs[e] & m;
                    const T* h = reinterpret_cast<const T*>(&y);
                    if (m & 0xffffu)
                      ov[8 * q + 2 * e] = __float_as_uint(__uint_as_float(ov[8 * q + 2 * e]) + static_cast<float>(h[0]));
                    if (m >> 16)
                      ov[8 * q + 2 * e + 1] =
                          __float_as_uint(__uint_as_float(ov[8 * q + 2 * e + 1]) + static_cast<float>(h[1]));
                  }
                }
              }
              scale = 1.f;
            }
            stage_row_chunk_sw128<BF>(stage, r, c, ov, scale);
          }
          tc_fence_before();  // O's columns are free for the next unit
          fence_proxy_async_smem();
          named_bar_sync(1 + w, 4 * 32);  // the tile's four warps have staged their rows
          if (left >= TB) {  // whole: a box
            if ((warp & 3) == 0 && lane == 0) {
#pragma unroll
              for (int kb = 0; kb < D / 64; ++kb)
                tma_store_3d(&tm_o, sQ(qb, w) + kb * (kBM * 128), kb * 64, p.head * G, p.row + w * TB);
              tma_store_commit_and_wait_read();
            }
          } else {  // the rows behind it are another sequence's
            copy_tile_rows(sQ(qb, w), args.dg, r, 128, out_row);
          }
        }
      }
      __syncwarp();
      if (lane == 0) {
        if (p.nt > 0) mbar_arrive(&bar_qfree[qb]);
        mbar_arrive(&ring.left[i & 1]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc(tmem, 512);
}

template <typename T, int D>
cudaError_t run(const PackedMaps& m, const PackedArgs& a, cudaStream_t s) {
  using C = PfCfg<D>;
  auto kern = packed_fwd_kernel<T, D>;
  static std::atomic<bool> attr[kMaxDevices];
  cudaError_t e = smem_attr_once(kern, C::SMEM, attr);
  if (e != cudaSuccess) return e;
  const long long blocks = a.shape.bound(kPackedFwd) * a.shape.Hkv;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  kern<<<static_cast<unsigned>(blocks), kThreads, C::SMEM, s>>>(m.q, m.k, m.v, m.o, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_packed_fwd(bool bf16, int D, const PackedMaps& m, const PackedArgs& a, cudaStream_t s) {
  if (D == 64) return bf16 ? run<__nv_bfloat16, 64>(m, a, s) : run<__half, 64>(m, a, s);
  if (D == 128) return bf16 ? run<__nv_bfloat16, 128>(m, a, s) : run<__half, 128>(m, a, s);
  return cudaErrorInvalidValue;
}

}  // namespace ta

TA_GUARD_ACCESSOR(packed_fwd)
