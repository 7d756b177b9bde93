// Backward of packed attention with shared key heads (sm_103a), in two passes:
//
//   dQ (query-stationary):  delta = rowsum(dO o O),  P = exp(c Q K^T - L),
//       dS = P o (dO V^T - delta),  dQ = c dS K
//   dK, dV (key-stationary):  dV = sum over the heads P^T dO,  dK = c sum dS^T Q
//
// The dQ pass runs first and stores delta for the other.  Query tiles hold the G
// heads of a key head (packed.cuh), so the key-stationary pass sums over heads
// and tokens in the same loop, in a fixed order and without atomics.
//
// Warps: 0-7 the element-wise part (warp % 4 selects the 32 TMEM lanes, warp / 4
// the half of a tile's 128 columns), 8 the TMA producer, 9 the MMA issuer, 10
// zeroes the rows of the last streamed tile that belong to no token of the
// sequence: their P and dS are zero, and a neighbour's infinity in a product with
// zero would be NaN.
#include "launch.h"
#include "packed.cuh"

namespace ta {

namespace {

constexpr int kThreads = 352;
constexpr int kProducer = 8, kMma = 9, kCare = 10;
constexpr int kRowWarps = 8;

template <int D>
__device__ __forceinline__ void load_rows(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int c1, int c2) {
#pragma unroll
  for (int kb = 0; kb < D / 64; ++kb) tma_load_3d(dst + kb * (kBM * 128), map, bar, kb * 64, c1, c2);
}

// d = A B^T over D: A (128 rows, 16-bit) in TMEM, B a 128-row K-major tile in shared memory.
template <int D>
__device__ __forceinline__ void mma_tmem_abT(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_smem, uint32_t idesc) {
  const uint64_t db0 = sdesc_sw128(b_smem, 16, 1024);
  uint32_t a[D / 16];
  uint64_t b[D / 16];
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    a[kk] = a_tmem + kk * 8;
    b[kk] = db0 + static_cast<uint64_t>(((kk >> 2) * (kBM * 128) + (kk & 3) * 32) >> 4);
  }
  mma_ts_n<D / 16>(d_tmem, a, b, idesc, 0u);
}

// d (+)= X Y over the K-steps of chunk group C: X 128 x 128 16-bit in TMEM, its
// column halves 64 columns apart; Y a 128-row x D tile read as rows = K.
template <int C>
__device__ __forceinline__ void mma_half_y(uint32_t d_tmem, uint32_t x_tmem, uint32_t y_smem, uint32_t idesc,
                                           bool accumulate) {
  const uint64_t dy = sdesc_sw128(y_smem, kBM * 128, 1024);
  uint32_t a[4];
  uint64_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int kk = chunk_kstep(C, i);
    a[i] = x_tmem + (kk & 3) * 8 + (kk >> 2) * 64;
    b[i] = dy + static_cast<uint64_t>((kk * 16 * 128) >> 4);
  }
  mma_ts_n<4>(d_tmem, a, b, idesc, accumulate ? 1u : 0u);
}

// Half of <a_r, b_r>: a from the thread's TMEM lane (two elements a column),
// b from its swizzled tile.
template <typename T, int D>
__device__ __forceinline__ float half_dot(uint32_t a_tmem, const uint8_t* b, int r, int half) {
  constexpr int NC = D / 4;
  uint32_t x[NC];
  if constexpr (NC == 32) tmem_ld_x32(a_tmem + half * NC, x);
  else tmem_ld_x16(a_tmem + half * NC, x);
  tmem_ld_wait(x);
  float acc = 0.f;
#pragma unroll
  for (int c8 = 0; c8 < D / 16; ++c8) {
    const int gc = half * (D / 16) + c8;
    const uint4 y = *reinterpret_cast<const uint4*>(b + (gc >> 3) * (kBM * 128) + r * 128 + (((gc & 7) ^ (r & 7)) * 16));
    const uint4 xv = make_uint4(x[4 * c8], x[4 * c8 + 1], x[4 * c8 + 2], x[4 * c8 + 3]);
    const T* xp = reinterpret_cast<const T*>(&xv);
    const T* yp = reinterpret_cast<const T*>(&y);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc = fmaf(static_cast<float>(xp[i]), static_cast<float>(yp[i]), acc);
  }
  return acc;
}

// ======================================================================
//                         dQ (query-stationary)
// ======================================================================
// Q and dO are the A operands of every score product and live in TMEM; they
// come through the last slot of the K/V ring.  O arrives behind the first K/V
// tile, and delta is formed while the first products run.
template <int D>
struct PdqCfg {
  static constexpr int TILE = (D / 64) * kBM * 128;
  static constexpr int STAGE = 2 * TILE;  // K, V
  static constexpr int ST_FIT = (kSmemMax - 2048 - TILE) / STAGE;
  static constexpr int STAGES = ST_FIT > 4 ? 4 : ST_FIT;
  static constexpr int OFF_O = STAGES * STAGE;
  static constexpr int SMEM = OFF_O + TILE + 1024;
  static constexpr uint32_t COL_A = 0, COL_B = 128, COL_DQ = 256;
  static constexpr uint32_t COL_QT = 256 + D, COL_DOT = 256 + D + D / 2;
  static_assert(STAGES >= 3 && SMEM + 2048 <= kSmemMax, "shared memory");
  static_assert(COL_DOT + D / 2 <= 512, "TMEM");
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    packed_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                     const __grid_constant__ CUtensorMap tm_dq, const __grid_constant__ CUtensorMap tm_o,
                     const PackedArgs args) {
  using C = PdqCfg<D>;
  constexpr bool BF = DT<T>::bf16;
  constexpr int STAGES = C::STAGES;

  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_q, bar_qfree, bar_kv[STAGES], bar_kvempty[STAGES];
  __shared__ __align__(8) uint64_t bar_s, bar_consumed, bar_dp, bar_ds[2], bar_done, bar_o, bar_last, bar_care;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const PackedList list = packed_list(args, kPackedDq);
  if (blockIdx.x >= list.items) return;
  const PackedUnit unit = packed_item(args, list, blockIdx.x);
  const int causal = unit.pad[0], head = unit.pad[1];
  const int G = args.shape.G, TB = args.shape.TB;
  const int nkv = packed_key_tiles(min(unit.left, TB), unit.off, unit.n, causal);
  const bool ragged = nkv * kBN > unit.n;  // the last tile ends behind the keys
  const int box = (D / 64) * TB * G * 128;  // bytes of a query tile

  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto sK = [&](int st) { return base + st * C::STAGE; };
  auto sV = [&](int st) { return base + st * C::STAGE + C::TILE; };
  uint8_t* sQ = sK(STAGES - 1);
  uint8_t* sDO = sV(STAGES - 1);
  uint8_t* sO = base + C::OFF_O;

  WaitCtl ctl{args.err, args.timeout_ns, &abort_flag};
  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(&bar_q, 1);
    mbar_init(&bar_qfree, kRowWarps);
    for (int st = 0; st < STAGES; ++st) {
      mbar_init(&bar_kv[st], 1);
      mbar_init(&bar_kvempty[st], 1);
    }
    mbar_init(&bar_s, 1);
    mbar_init(&bar_consumed, kRowWarps);
    mbar_init(&bar_dp, 1);
    mbar_init(&bar_ds[0], kRowWarps);
    mbar_init(&bar_ds[1], kRowWarps);
    mbar_init(&bar_done, 1);
    mbar_init(&bar_o, 1);
    mbar_init(&bar_last, 1);
    mbar_init(&bar_care, 1);
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

  if (warp == kProducer) {
    // ------------------------------------------------------------ producer
    if (lane == 0 && nkv > 0) {
      mbar_expect_tx(&bar_q, 2 * box);
      load_rows<D>(sQ, &tm_q, &bar_q, head * G, unit.row);
      load_rows<D>(sDO, &tm_do, &bar_q, head * G, unit.row);
      int issued = 0;
      bool o_issued = false;
      for (int t = 0; t < nkv; ++t) {
        const int st = t % STAGES;
        if (t >= STAGES) {
          if (!mbar_wait(&bar_kvempty[st], ((t / STAGES) - 1) & 1, ctl, kErrTimeoutMma)) break;
        } else if (st == STAGES - 1) {  // the slot still holds Q and dO until they are in TMEM
          if (!mbar_wait(&bar_qfree, 0, ctl, kErrTimeoutSoftmax)) break;
        }
        uint64_t* bar = ragged && t == nkv - 1 ? &bar_last : &bar_kv[st];
        mbar_expect_tx(bar, 2 * C::TILE);
        load_rows<D>(sK(st), &tm_k, bar, unit.krow + t * kBN, head);
        load_rows<D>(sV(st), &tm_v, bar, unit.krow + t * kBN, head);
        issued = t + 1;
        if (t == 0) {  // O for delta
          mbar_expect_tx(&bar_o, box);
          load_rows<D>(sO, &tm_o, &bar_o, head * G, unit.row);
          o_issued = true;
        }
      }
      int zero = 0;
      WaitCtl drain{args.err, args.timeout_ns, reinterpret_cast<volatile int*>(&zero)};
      mbar_wait(&bar_q, 0, drain, kErrTimeoutTma);
      if (o_issued) mbar_wait(&bar_o, 0, drain, kErrTimeoutTma);
      for (int t = issued - STAGES > 0 ? issued - STAGES : 0; t < issued; ++t) {
        if (ragged && t == nkv - 1) mbar_wait(&bar_last, 0, drain, kErrTimeoutTma);
        else mbar_wait(&bar_kv[t % STAGES], (t / STAGES) & 1, drain, kErrTimeoutTma);
      }
    }
  } else if (warp == kMma) {
    // ----------------------------------------------------------------- MMA
    if (nkv > 0) {
      constexpr uint32_t idesc_s = idesc_f16(kBM, kBN, BF, false, false);
      constexpr uint32_t idesc_g = idesc_f16(kBM, D, BF, false, true);
      auto kv_ready = [&](int t) {
        if (ragged && t == nkv - 1) return warp_wait(&bar_care, 0, ctl, kErrTimeoutOther);
        return warp_wait(&bar_kv[t % STAGES], (t / STAGES) & 1, ctl, kErrTimeoutTma);
      };
      bool ok = warp_wait(&bar_qfree, 0, ctl, kErrTimeoutSoftmax) && kv_ready(0);
      if (ok) {
        tc_fence_after();
        mma_tmem_abT<D>(tmem + C::COL_A, tmem + C::COL_QT, smem_u32(sK(0)), idesc_s);
        commit_el(&bar_s);
        mma_tmem_abT<D>(tmem + C::COL_B, tmem + C::COL_DOT, smem_u32(sV(0)), idesc_s);  // dP = dO V^T
        commit_el(&bar_dp);
      }
      for (int t = 0; ok && t < nkv; ++t) {
        const int st = t % STAGES;
        const int st1 = (t + 1) % STAGES;
        const bool next = t + 1 < nkv;
        if (next) {
          if (!(ok = warp_wait(&bar_consumed, t & 1, ctl, kErrTimeoutSoftmax))) break;
          if (!(ok = kv_ready(t + 1))) break;
          tc_fence_after();
          mma_tmem_abT<D>(tmem + C::COL_A, tmem + C::COL_QT, smem_u32(sK(st1)), idesc_s);
          commit_el(&bar_s);
        }
        if (!(ok = warp_wait(&bar_ds[0], t & 1, ctl, kErrTimeoutSoftmax))) break;
        tc_fence_after();
        mma_half_y<0>(tmem + C::COL_DQ, tmem + C::COL_B, smem_u32(sK(st)), idesc_g, t > 0);
        if (!(ok = warp_wait(&bar_ds[1], t & 1, ctl, kErrTimeoutSoftmax))) break;
        tc_fence_after();
        mma_half_y<1>(tmem + C::COL_DQ, tmem + C::COL_B, smem_u32(sK(st)), idesc_g, true);
        commit_el(&bar_kvempty[st]);
        if (next) {
          mma_tmem_abT<D>(tmem + C::COL_B, tmem + C::COL_DOT, smem_u32(sV(st1)), idesc_s);
          commit_el(&bar_dp);
        }
      }
      if (ok) commit_el(&bar_done);
    }
  } else if (warp == kCare) {
    if (nkv > 0 && ragged) {
      const int t = nkv - 1, st = t % STAGES;
      if (warp_wait(&bar_last, 0, ctl, kErrTimeoutTma)) {
        zero_tile_rows<D / 64>(sK(st), unit.n - t * kBN, lane);
        zero_tile_rows<D / 64>(sV(st), unit.n - t * kBN, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_care);
      }
    }
  } else {
    // --------------------------------------------- query-row softmax gradient
    const int hc = warp >> 2;  // key half of the tile: columns [64 hc, 64 hc + 64)
    const int cb = 64 * hc;
    const int r = threadIdx.x & 127;
    const int tok = static_cast<int>(args.g_div.div(r)), hq = r - tok * G;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const bool in = tok < min(unit.left, TB);
    const size_t g = (static_cast<size_t>(unit.row) + (in ? tok : 0)) * args.shape.Hq + head * G + (in ? hq : 0);
    const float neg_L2 = in ? -args.lse[g] * kLog2e : -INFINITY;
    const int sees = causal ? min(unit.n - 1, unit.off + tok) : unit.n - 1;
    const int t_part = causal ? min(unit.n / kBN, unit.off < 0 ? 0 : (unit.off + 1) / kBN) : unit.n / kBN;
    bool ok = true;
    if (nkv > 0) {  // group 0 copies Q, group 1 dO into TMEM
      ok = warp_wait(&bar_q, 0, ctl, kErrTimeoutTma);
      if (ok) {
        tile_row_to_tmem<D>(hc == 0 ? sQ : sDO, r, lane_addr + (hc == 0 ? C::COL_QT : C::COL_DOT));
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_qfree);
      }
    }
    // delta: each group half of every row's columns; a tile that sees no key has O = 0
    float dlt = 0.f;
    if (nkv > 0 && ok) {
      ok = warp_wait(&bar_qfree, 0, ctl, kErrTimeoutSoftmax) && warp_wait(&bar_o, 0, ctl, kErrTimeoutTma);
      if (ok) {
        tc_fence_after();
        dlt = half_dot<T, D>(lane_addr + C::COL_DOT, sO, r, hc);
      }
    }
    float* halves = reinterpret_cast<float*>(sO);
    named_bar_sync(1, kRowWarps * 32);
    halves[hc * kBM + r] = dlt;
    named_bar_sync(1, kRowWarps * 32);
    dlt = halves[r] + halves[kBM + r];
    if (hc == 0 && in) args.delta[g] = dlt;
    for (int t = 0; ok && t < nkv; ++t) {
      const int k0 = t * kBN;
      if (!(ok = warp_wait(&bar_s, t & 1, ctl, kErrTimeoutMma))) break;
      tc_fence_after();
      uint32_t sv[64];
      tmem_ld_x32(lane_addr + C::COL_A + cb, TB_CHUNK(sv, 0));
      tmem_ld_x32(lane_addr + C::COL_A + cb + 32, TB_CHUNK(sv, 1));
      tmem_ld_wait(TB_CHUNK(sv, 0));
      tmem_ld_wait(TB_CHUNK(sv, 1));
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_consumed);  // S buffer free for S(t + 1)
      float p[64];
#pragma unroll
      for (int c = 0; c < 64; c += 2) {
        const float2 y = ffma2(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])),
                               make_float2(args.scale_log2, args.scale_log2), make_float2(neg_L2, neg_L2));
        p[c] = ex2(y.x);
        p[c + 1] = ex2(y.y);
      }
      if (t >= t_part) {
        const int lim = sees - k0 - cb;
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c > lim) p[c] = 0.f;
      }
      if (!(ok = warp_wait(&bar_dp, t & 1, ctl, kErrTimeoutMma))) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t dp[32];
        tmem_ld_x32(lane_addr + C::COL_B + cb + 32 * c, dp);
        tmem_ld_wait(dp);
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int c0 = 32 * c + 2 * e;
          const float2 ds = fmul2(make_float2(p[c0], p[c0 + 1]),
                                  fadd2(make_float2(__uint_as_float(dp[2 * e]), __uint_as_float(dp[2 * e + 1])),
                                        make_float2(-dlt, -dlt)));
          pk[e] = pack2<BF>(ds.x, ds.y);
        }
        tmem_st_x16(lane_addr + C::COL_B + cb + 16 * c, pk);  // dS (16-bit) over dP
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_ds[c]);
      }
    }
    if (nkv > 0 && ok) ok = warp_wait(&bar_done, 0, ctl, kErrTimeoutMma);
    tc_fence_after();
    // dQ (x sm_scale) staged over the ring's first K slot (every MMA has finished)
    const bool live = ok && nkv > 0;
#pragma unroll
    for (int cc = 0; cc < D / 64; ++cc) {
      const int c = hc * (D / 64) + cc;
      uint32_t v[32];
      if (live) {
        tmem_ld_x32(lane_addr + C::COL_DQ + 32 * c, v);
        tmem_ld_wait(v);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = 0u;
      }
      stage_row_chunk_sw128<BF>(smem_u32(sK(0)), r, c, v, args.sm_scale);
    }
    fence_proxy_async_smem();
    named_bar_sync(1, kRowWarps * 32);
    if (unit.left >= TB) {
      if (warp == 0 && lane == 0) {
#pragma unroll
        for (int kb = 0; kb < D / 64; ++kb)
          tma_store_3d(&tm_dq, sK(0) + kb * (kBM * 128), kb * 64, head * G, unit.row);
        tma_store_commit_and_wait_read();
      }
    } else {
      T* dq = static_cast<T*>(args.dq);
      const int rows = unit.left * G;
      copy_tile_rows(sK(0), args.dg, threadIdx.x, kRowWarps * 32, [&](int i) -> void* {
        if (i >= rows) return nullptr;
        const int k = static_cast<int>(args.g_div.div(i));
        return dq + (static_cast<long long>(unit.row) + k) * args.dq_t + (head * G + i - k * G) * args.dq_h;
      });
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc(tmem, 512);
}

// ======================================================================
//                       dK, dV (key-stationary)
// ======================================================================
// Per query tile u:  S^T(u + 1) | dV(u) dK(u) | dP^T(u + 1), with P^T and dS^T
// (16 + 16 packed columns per 32-column chunk) written over dP^T.  Q has a ring
// of its own, a tile ahead of dO's; L and delta of a tile are fetched a tile
// ahead into a double buffer.  All shared memory is in the dynamic region (K, V,
// the Q and dO rings, L and delta, barriers).
template <int D>
struct PkvCfg {
  static constexpr int TILE = (D / 64) * kBM * 128;
  static constexpr int QST = D == 128 ? 3 : 4;
  static constexpr int OST = D == 128 ? 2 : 4;
  static constexpr int LD_OFF = (2 + QST + OST) * TILE;  // [buffer][half][L, delta][64] floats
  static constexpr int BAR_OFF = LD_OFF + 2 * 2 * 2 * 64 * 4;
  static constexpr int BAR_BYTES = 256;
  static constexpr int USED = BAR_OFF + BAR_BYTES;
  static constexpr int PAD = (kSmemMax - USED) < 1023 ? (kSmemMax - USED) : 1023;
  static constexpr int SMEM = USED + PAD;
  static constexpr uint32_t COL_A = 0, COL_B = 128, COL_DV = 256, COL_DK = 256 + D;
  static_assert(PAD >= 0 && SMEM <= kSmemMax, "tiles do not fit in shared memory");
  static_assert(BAR_BYTES >= 8 * (1 + 2 * QST + 2 * OST + 6 + 4 + 4) + 8, "barrier area too small");
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    packed_dkdv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                       const __grid_constant__ CUtensorMap tm_dk, const __grid_constant__ CUtensorMap tm_dv,
                       const PackedArgs args) {
  using C = PkvCfg<D>;
  constexpr bool BF = DT<T>::bf16;
  constexpr int QST = C::QST, OST = C::OST;

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  if (base - smem_raw > C::PAD) {  // uniform across the CTA: nothing has been touched yet
    if (threadIdx.x == 0 && args.err) atomicOr(args.err, kErrSmemLayout);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + C::BAR_OFF);
  uint64_t& bar_kv = bars[0];
  uint64_t* bar_qf = bars + 1;
  uint64_t* bar_qe = bar_qf + QST;
  uint64_t* bar_of = bar_qe + QST;
  uint64_t* bar_oe = bar_of + OST;
  uint64_t& bar_s = bar_oe[OST];
  uint64_t& bar_consumed = bar_oe[OST + 1];
  uint64_t& bar_dp = bar_oe[OST + 2];
  uint64_t* bar_ds = bar_oe + OST + 3;  // [chunk group]
  uint64_t& bar_done = bar_oe[OST + 5];
  uint64_t* bar_pub = bar_oe + OST + 6;  // [buffer * 2 + half]: L / delta of a tile stored
  uint64_t* bar_care = bar_pub + 4;      // [0]: the last Q tile's rows zeroed, [1]: dO's
  uint64_t* bar_last = bar_care + 2;     // the last Q and dO tile, where they end behind the tokens
  uint32_t& tmem_slot = *reinterpret_cast<uint32_t*>(bar_last + 2);
  int& abort_flag = *(reinterpret_cast<int*>(bar_last + 2) + 1);
  float* sLD = reinterpret_cast<float*>(base + C::LD_OFF);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const PackedList list = packed_list(args, kPackedDkdv);
  if (blockIdx.x >= list.items) return;
  const PackedUnit unit = packed_item(args, list, blockIdx.x);
  const int causal = unit.pad[0], head = unit.pad[1];
  const int G = args.shape.G, TB = args.shape.TB;
  const int nq = (unit.left + TB - 1) / TB;
  const int box = (D / 64) * TB * G * 128;
  const bool ragged = nq * TB > unit.left;

  uint8_t* sK = base;
  uint8_t* sV = base + C::TILE;
  auto sQ = [&](int i) { return base + (2 + i) * C::TILE; };
  auto sDO = [&](int i) { return base + (2 + QST + i) * C::TILE; };

  WaitCtl ctl{args.err, args.timeout_ns, &abort_flag};
  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(&bar_kv, 1);
    for (int i = 0; i < QST; ++i) {
      mbar_init(&bar_qf[i], 1);
      mbar_init(&bar_qe[i], 1);
    }
    for (int i = 0; i < OST; ++i) {
      mbar_init(&bar_of[i], 1);
      mbar_init(&bar_oe[i], 1);
    }
    mbar_init(&bar_s, 1);
    mbar_init(&bar_consumed, kRowWarps);
    mbar_init(&bar_dp, 1);
    mbar_init(&bar_ds[0], kRowWarps);
    mbar_init(&bar_ds[1], kRowWarps);
    mbar_init(&bar_done, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&bar_pub[i], kRowWarps / 2);
    mbar_init(&bar_care[0], 1);
    mbar_init(&bar_care[1], 1);
    mbar_init(&bar_last[0], 1);
    mbar_init(&bar_last[1], 1);
    fence_mbar_init();
  }
  if (TB * G < kBM) {  // rows that no box ever fills, in every slot
    for (int i = warp; i < QST + OST; i += kThreads / 32) zero_tile_rows<D / 64>(sQ(0) + i * C::TILE, TB * G, lane);
    fence_proxy_async_smem();
  }
  if (warp == kMma) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp == kProducer) {
    // ---------------------- producer: lane 0 K, V and the Q ring; lane 1 the dO ring
    if (lane < 2 && nq > 0) {
      const bool is_q = (lane == 0);
      const int depth = is_q ? QST : OST;
      uint64_t* full = is_q ? bar_qf : bar_of;
      uint64_t* empty = is_q ? bar_qe : bar_oe;
      const CUtensorMap* map = is_q ? &tm_q : &tm_do;
      if (is_q) {
        mbar_expect_tx(&bar_kv, 2 * C::TILE);
        load_rows<D>(sK, &tm_k, &bar_kv, unit.krow, head);
        load_rows<D>(sV, &tm_v, &bar_kv, unit.krow, head);
      }
      int issued = 0;
      for (int u = 0; u < nq; ++u) {
        const int st = u % depth;
        if (u >= depth && !mbar_wait(&empty[st], ((u / depth) - 1) & 1, ctl, kErrTimeoutMma)) break;
        uint64_t* bar = ragged && u == nq - 1 ? &bar_last[lane] : &full[st];
        mbar_expect_tx(bar, box);
        load_rows<D>(is_q ? sQ(st) : sDO(st), map, bar, head * G, unit.row + u * TB);
        issued = u + 1;
      }
      int zero = 0;
      WaitCtl drain{args.err, args.timeout_ns, reinterpret_cast<volatile int*>(&zero)};
      if (is_q) mbar_wait(&bar_kv, 0, drain, kErrTimeoutTma);
      for (int u = issued - depth > 0 ? issued - depth : 0; u < issued; ++u) {
        if (ragged && u == nq - 1) mbar_wait(&bar_last[lane], 0, drain, kErrTimeoutTma);
        else mbar_wait(&full[u % depth], (u / depth) & 1, drain, kErrTimeoutTma);
      }
    }
  } else if (warp == kMma) {
    // ----------------------------------------------------------------- MMA
    if (nq > 0) {
      constexpr uint32_t idesc_s = idesc_f16(kBN, kBM, BF, false, false);  // M = keys, N = query rows
      constexpr uint32_t idesc_g = idesc_f16(kBN, D, BF, false, true);     // M = keys, N = D
      auto q_ready = [&](int u) {
        if (ragged && u == nq - 1) return warp_wait(&bar_care[0], 0, ctl, kErrTimeoutOther);
        return warp_wait(&bar_qf[u % QST], (u / QST) & 1, ctl, kErrTimeoutTma);
      };
      auto o_ready = [&](int u) {
        if (ragged && u == nq - 1) return warp_wait(&bar_care[1], 0, ctl, kErrTimeoutOther);
        return warp_wait(&bar_of[u % OST], (u / OST) & 1, ctl, kErrTimeoutTma);
      };
      bool ok = warp_wait(&bar_kv, 0, ctl, kErrTimeoutTma) && q_ready(0) && o_ready(0);
      if (ok) {
        tc_fence_after();
        mma_abT<D>(tmem + C::COL_A, smem_u32(sK), smem_u32(sQ(0)), idesc_s);  // S^T = K Q^T
        commit_el(&bar_s);
        mma_abT<D>(tmem + C::COL_B, smem_u32(sV), smem_u32(sDO(0)), idesc_s);  // dP^T = V dO^T
        commit_el(&bar_dp);
      }
      for (int u = 0; ok && u < nq; ++u) {
        const int sq = u % QST, so = u % OST;
        const int sq1 = (u + 1) % QST, so1 = (u + 1) % OST;
        const bool next = u + 1 < nq;
        if (next) {
          if (!(ok = warp_wait(&bar_consumed, u & 1, ctl, kErrTimeoutSoftmax))) break;
          if (!(ok = q_ready(u + 1))) break;
          tc_fence_after();
          mma_abT<D>(tmem + C::COL_A, smem_u32(sK), smem_u32(sQ(sq1)), idesc_s);
          commit_el(&bar_s);
        }
        if (!(ok = warp_wait(&bar_ds[0], u & 1, ctl, kErrTimeoutSoftmax))) break;
        tc_fence_after();
        mma_tY_il_g<0>(tmem + C::COL_DV, tmem + C::COL_B, smem_u32(sDO(so)), idesc_g, u > 0);
        mma_tY_il_g<0>(tmem + C::COL_DK, tmem + C::COL_B + 16, smem_u32(sQ(sq)), idesc_g, u > 0);
        if (!(ok = warp_wait(&bar_ds[1], u & 1, ctl, kErrTimeoutSoftmax))) break;
        tc_fence_after();
        mma_tY_il_g<1>(tmem + C::COL_DV, tmem + C::COL_B, smem_u32(sDO(so)), idesc_g, true);
        commit_el(&bar_oe[so]);
        mma_tY_il_g<1>(tmem + C::COL_DK, tmem + C::COL_B + 16, smem_u32(sQ(sq)), idesc_g, true);
        commit_el(&bar_qe[sq]);
        if (next) {
          if (!(ok = o_ready(u + 1))) break;
          tc_fence_after();
          mma_abT<D>(tmem + C::COL_B, smem_u32(sV), smem_u32(sDO(so1)), idesc_s);
          commit_el(&bar_dp);
        }
      }
      if (ok) commit_el(&bar_done);
    }
  } else if (warp == kCare) {
    if (nq > 0 && ragged) {
      const int u = nq - 1, rows = (unit.left - u * TB) * G;
      bool ok = warp_wait(&bar_last[0], 0, ctl, kErrTimeoutTma);
      if (ok) {
        zero_tile_rows<D / 64>(sQ(u % QST), rows, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_care[0]);
        ok = warp_wait(&bar_last[1], 0, ctl, kErrTimeoutTma);
      }
      if (ok) {
        zero_tile_rows<D / 64>(sDO(u % OST), rows, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_care[1]);
      }
    }
  } else {
    // ------------------------------------------- key-row softmax gradient
    const int hc = warp >> 2;  // half of the query tile's rows: columns [64 hc, 64 hc + 64)
    const int cb = 64 * hc;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    // L and delta of the half's 64 rows, one value a thread; rows of no token read
    // L = +inf (P = 0) and delta = 0
    const int ld_arr = (threadIdx.x & 127) >> 6;  // 0: L, 1: delta
    const int ld_col = threadIdx.x & 63;
    const int ld_tok = static_cast<int>(args.g_div.div(cb + ld_col)), ld_head = cb + ld_col - ld_tok * G;
    auto ld_fetch = [&](int u) -> float {
      if (ld_tok >= TB || u * TB + ld_tok >= unit.left) return ld_arr ? 0.f : INFINITY;
      const size_t row = static_cast<size_t>(unit.row) + u * TB + ld_tok;
      return __ldg((ld_arr ? args.delta : args.lse) + row * args.shape.Hq + head * G + ld_head);
    };
    auto ld_slot = [&](int u) { return sLD + ((u & 1) * 2 + hc) * 128; };
    if (nq > 0) {
      ld_slot(0)[ld_arr * 64 + ld_col] = ld_fetch(0);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_pub[hc]);
    }
    const int m = lane & 3;
    const int kl = 32 * (warp & 3) + (lane >> 2);  // the thread's first key of the tile (then + 8, + 16, + 24)
    bool ok = true;
    for (int u = 0; u < nq; ++u) {
      const float pre = (u + 1 < nq) ? ld_fetch(u + 1) : 0.f;
      if (!(ok = warp_wait(&bar_s, u & 1, ctl, kErrTimeoutMma))) break;
      tc_fence_after();
      // 16-lane shapes: sv[32 g + 4 jj + e], e = {(k, q), (k, q + 1), (k + 8, q), (k + 8, q + 1)} with
      // k = kl + 16 g and q = cb + 8 jj + 2 m
      uint32_t sv[64];
      tmem_ld_16x256b_x8(lane_addr + C::COL_A + cb, TB_CHUNK(sv, 0));
      tmem_ld_16x256b_x8(lane_addr + (16u << 16) + C::COL_A + cb, TB_CHUNK(sv, 1));
      tmem_ld_wait(TB_CHUNK(sv, 0));
      tmem_ld_wait(TB_CHUNK(sv, 1));
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_consumed);  // score buffer free for S^T(u + 1)
      if (!(ok = warp_wait(&bar_pub[(u & 1) * 2 + hc], (u >> 1) & 1, ctl, kErrTimeoutSoftmax))) break;
      const float* sL = ld_slot(u) + 2 * m;
      const float* sD = sL + 64;
      const float2 sc2 = make_float2(args.scale_log2, args.scale_log2);
      float p[64];
#pragma unroll
      for (int jj = 0; jj < 8; ++jj) {
        const float2 l2 = *reinterpret_cast<const float2*>(sL + 8 * jj);
        const float2 nl = fmul2(l2, make_float2(-kLog2e, -kLog2e));
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int i = 32 * g + 4 * jj;
          const float2 y0 = ffma2(make_float2(__uint_as_float(sv[i]), __uint_as_float(sv[i + 1])), sc2, nl);
          const float2 y1 = ffma2(make_float2(__uint_as_float(sv[i + 2]), __uint_as_float(sv[i + 3])), sc2, nl);
          p[i + 0] = ex2(y0.x);
          p[i + 1] = ex2(y0.y);
          p[i + 2] = ex2(y1.x);
          p[i + 3] = ex2(y1.y);
        }
      }
      // key k of the tile is seen from token off + k on: column q (token u TB + q / G)
      // is masked iff q < (off + k - u TB) G
      if (causal && unit.off + kBN - 1 > u * TB) {
        int lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = unit.off + kl + 8 * i - u * TB;
          lo[i] = min(max(x, 0), kBM) * G - cb - 2 * m;  // (past the tile's end: everything)
        }
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int jj = 0; jj < 8; ++jj)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (8 * jj + (e & 1) < lo[2 * g + (e >> 1)]) p[32 * g + 4 * jj + e] = 0.f;
      }
      if (!(ok = warp_wait(&bar_dp, u & 1, ctl, kErrTimeoutMma))) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        // chunk c (32 rows): read dP^T, write P^T and dS^T back into the same 32 columns
        uint32_t dp[32];  // [g][16]
        tmem_ld_16x256b_x4(lane_addr + C::COL_B + cb + 32 * c, TB_CHUNK16(dp, 0));
        tmem_ld_16x256b_x4(lane_addr + (16u << 16) + C::COL_B + cb + 32 * c, TB_CHUNK16(dp, 1));
        tmem_ld_wait(TB_CHUNK16(dp, 0));
        tmem_ld_wait(TB_CHUNK16(dp, 1));
        float2 nd2[4];  // -delta of the thread's query pairs
#pragma unroll
        for (int jq = 0; jq < 4; ++jq) {
          const float2 d2 = *reinterpret_cast<const float2*>(sD + 8 * (4 * c + jq));
          nd2[jq] = make_float2(-d2.x, -d2.y);
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t pp[8], pd[8];
#pragma unroll
          for (int jq = 0; jq < 4; ++jq) {
            const int i = 32 * g + 4 * (4 * c + jq);
            const int di = 16 * g + 4 * jq;
            pp[2 * jq] = pack2<BF>(p[i], p[i + 1]);
            pp[2 * jq + 1] = pack2<BF>(p[i + 2], p[i + 3]);
            const float2 s0 = fmul2(make_float2(p[i], p[i + 1]),
                                    fadd2(make_float2(__uint_as_float(dp[di]), __uint_as_float(dp[di + 1])), nd2[jq]));
            const float2 s1 = fmul2(make_float2(p[i + 2], p[i + 3]),
                                    fadd2(make_float2(__uint_as_float(dp[di + 2]), __uint_as_float(dp[di + 3])), nd2[jq]));
            pd[2 * jq] = pack2<BF>(s0.x, s0.y);
            pd[2 * jq + 1] = pack2<BF>(s1.x, s1.y);
          }
          const uint32_t ga = lane_addr + (static_cast<uint32_t>(16 * g) << 16) + C::COL_B + cb + 32 * c;
          tmem_st_16x128b_x4(ga, pp);
          tmem_st_16x128b_x4(ga + 16, pd);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_ds[c]);
      }
      if (u + 1 < nq) {  // every warp of the half is past tile u - 1, the buffer's previous tile
        ld_slot(u + 1)[ld_arr * 64 + ld_col] = pre;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_pub[((u + 1) & 1) * 2 + hc]);
      }
    }
    // ------------------------------------------------------------ epilogue
    if (nq > 0 && ok) ok = warp_wait(&bar_done, 0, ctl, kErrTimeoutMma);
    tc_fence_after();
    // dV staged over K, dK (x sm_scale) over V (every MMA has finished)
    const int r = threadIdx.x & 127;
    const bool live = ok && nq > 0;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
#pragma unroll
      for (int cc = 0; cc < D / 64; ++cc) {
        const int c = hc * (D / 64) + cc;
        uint32_t v[32];
        if (live) {
          tmem_ld_x32(lane_addr + (a == 0 ? C::COL_DV : C::COL_DK) + 32 * c, v);
          tmem_ld_wait(v);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0u;
        }
        stage_row_chunk_sw128<BF>(smem_u32(a == 0 ? sK : sV), r, c, v, a ? args.sm_scale : 1.f);
      }
    }
    fence_proxy_async_smem();
    named_bar_sync(1, kRowWarps * 32);
    if (unit.n >= kBN) {
      if (warp == 0 && lane == 0) {
#pragma unroll
        for (int kb = 0; kb < D / 64; ++kb) {
          tma_store_3d(&tm_dv, sK + kb * (kBM * 128), kb * 64, unit.krow, head);
          tma_store_3d(&tm_dk, sV + kb * (kBM * 128), kb * 64, unit.krow, head);
        }
        tma_store_commit_and_wait_read();
      }
    } else {  // the rows behind the keys are another sequence's
      auto copy = [&](const uint8_t* tile, void* to, long long st, long long sh) {
        T* p = static_cast<T*>(to) + head * sh + static_cast<long long>(unit.krow) * st;
        copy_tile_rows(tile, args.dg, threadIdx.x, kRowWarps * 32,
                       [&](int i) -> void* { return i < unit.n ? p + i * st : nullptr; });
      };
      copy(sK, args.dv, args.dv_t, args.dv_h);
      copy(sV, args.dk, args.dk_t, args.dk_h);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc(tmem, 512);
}

template <typename T, int D>
cudaError_t run_dq(const PackedMaps& m, const PackedArgs& a, cudaStream_t s) {
  using C = PdqCfg<D>;
  auto kern = packed_dq_kernel<T, D>;
  static std::atomic<bool> attr[kMaxDevices];
  cudaError_t e = smem_attr_once(kern, C::SMEM, attr);
  if (e != cudaSuccess) return e;
  const long long blocks = a.shape.bound(kPackedDq) * a.shape.Hkv;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  kern<<<static_cast<unsigned>(blocks), kThreads, C::SMEM, s>>>(m.q, m.k, m.v, m.dO, m.dq, m.o, a);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t run_dkdv(const PackedMaps& m, const PackedArgs& a, cudaStream_t s) {
  using C = PkvCfg<D>;
  auto kern = packed_dkdv_kernel<T, D>;
  static std::atomic<bool> attr[kMaxDevices];
  cudaError_t e = smem_attr_once(kern, C::SMEM, attr);
  if (e != cudaSuccess) return e;
  const long long blocks = a.shape.bound(kPackedDkdv) * a.shape.Hkv;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  kern<<<static_cast<unsigned>(blocks), kThreads, C::SMEM, s>>>(m.q, m.k, m.v, m.dO, m.dk, m.dv, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_packed_dq(bool bf16, int D, const PackedMaps& m, const PackedArgs& a, cudaStream_t s) {
  if (D == 64) return bf16 ? run_dq<__nv_bfloat16, 64>(m, a, s) : run_dq<__half, 64>(m, a, s);
  if (D == 128) return bf16 ? run_dq<__nv_bfloat16, 128>(m, a, s) : run_dq<__half, 128>(m, a, s);
  return cudaErrorInvalidValue;
}

cudaError_t launch_packed_dkdv(bool bf16, int D, const PackedMaps& m, const PackedArgs& a, cudaStream_t s) {
  if (D == 64) return bf16 ? run_dkdv<__nv_bfloat16, 64>(m, a, s) : run_dkdv<__half, 64>(m, a, s);
  if (D == 128) return bf16 ? run_dkdv<__nv_bfloat16, 128>(m, a, s) : run_dkdv<__half, 128>(m, a, s);
  return cudaErrorInvalidValue;
}

}  // namespace ta

TA_GUARD_ACCESSOR(packed_bwd)
