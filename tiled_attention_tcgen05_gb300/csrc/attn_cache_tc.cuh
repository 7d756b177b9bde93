// Attention of new tokens over a paged key/value cache on the tensor cores
// (tcgen05), for many query rows per key head: drafts' trees, prompts' chunks.
//
// A block works through its piece of the line (attn_cache.cuh) with the roles
//   warps 0-3, 4-7  two softmax groups, a thread per query row (= TMEM lane);
//   warps 8-11      bring Q into shared memory and look through tiles with new
//                   tokens; 8 bits: turn the keys' codes into fp16, and four
//                   warps more the values';
//   a warp          issues the MMAs: S = Q K^T, O += P V with P in TMEM;
//   two warps       fetch keys and values by TMA;
// and the registers handed to the softmax groups (setmaxnreg).  The groups
// alternate on the tensor core:  S0 S1 | PV0 S0' | PV1 S1' | ...  Units of more
// than 128 rows give each group a row tile of its own and both the same keys;
// units of up to 128 rows give both groups the same rows and every other
// key tile, and join the two states at the end: the softmax of one tile
// then runs beside the other's MMAs in either case.
//
// Tiles are gathered by TMA in boxes of 8, 16 or 32 rows (the largest that
// divides a page), a lane per box.  Boxes behind the sequence's end or of pages
// that do not exist are fetched from outside the map and so read as zeros.
// 16-bit rows go straight into the 128-byte-swizzled layout that the MMA
// descriptors read.  8-bit codes go into staging rings, one of keys (with the
// scales) and one of values, and the eight helpers turn them into fp16 as they
// are, which is exact.  As in attn_cache_rows.cuh a key's scale multiplies its
// finished scores, a value's is part of the weight's exponent, and the sum takes
// it out again: whatever the scales' range, weights are rounded relative to the
// row's largest contribution, and a value that a row does not see cannot cost
// it anything.  (Values multiplied out to fp16 by one power of two for all of
// them lost the small ones beside a large one that no row used, and took 124 us
// where this takes 119: 16 sequences of 8192, 8 key heads of 128, 64 rows, e4m3.  That is
// 34 % of the copy rate; over int8 122 us.  What bounds it are the hand-overs between the
// roles: of the 138 us it took over int8 when conversions still multiplied,
// 108 were left without the conversions' arithmetic, the softmax's first pass, the
// exponentials and the fetches.)
//
// A box may bring rows behind the sequence's end, whose memory may hold
// anything, and a draft's values may hold infinities and NaN that some rows
// must not see: 0 * NaN would reach every row.  Tiles of values with new
// tokens are looked through before they are handed on: dead rows are cleared
// and the new tokens' non-finite values taken out; the rows that do see such a
// value get it added to their result.  Older tokens' values stay: every row
// sees them.
#pragma once
#include "attn_cache.cuh"
#include "bwd_common.cuh"
#include "common.cuh"
#include "launch.h"

namespace ta {
namespace {

constexpr int kTcBlocks = 152;    // one per SM

template <int CT, int DP>
struct TcCfg {
  static constexpr bool Q8 = CT != kCache16;
  static constexpr int TILE = DP / 64 * (kBM * 128);
  static constexpr int QT = Q8 ? 1 : 2;                  // query tiles
  static constexpr int ROWS = QT * kBM;                  // rows per unit
  static constexpr int KST = Q8 ? (DP == 128 ? 2 : 3) : (DP == 128 ? 3 : 4);
  static constexpr int VST = Q8 ? KST : (DP == 128 ? 2 : 4);
  static constexpr int OPB = Q8 ? 64 * DP : 0;           // codes of half a tile
  static constexpr int SR = Q8 ? (DP == 128 ? 3 : 6) : 0;  // staging rings, of keys and of values
  static constexpr int SSLOT = OPB + 1024;               // keys': and both scales of the whole tile's keys
  static constexpr int SCS = KST + 2;                    // tiles whose scales the softmax may need
  static constexpr int SCALES = Q8 ? SCS * 1536 : 0;     // their ring: keys' scales, values' log2, sum's factors
  static constexpr int HELPERS = Q8 ? 8 : 4;             // warps 8 .. 8 + HELPERS - 1
  static constexpr int MMA = 8 + HELPERS;                // warp; the fetching warps follow it
  static constexpr int THREADS = 32 * (MMA + 4);         // whole register groups of four warps
  static constexpr int REG_LAUNCH = 65536 / THREADS / 8 * 8;
  static constexpr int REG_SOFTMAX = Q8 ? 152 : 176, REG_COPY = Q8 ? 64 : 80, REG_MMA = Q8 ? 48 : 80;
  static_assert(256 * REG_SOFTMAX + 32 * HELPERS * REG_COPY + 128 * REG_MMA <= THREADS * REG_LAUNCH,
                "the groups' registers come out of the launch's");
  // Where a one-tile unit's groups join: the second query tile (D = 128, 16
  // bits), memory of its own (D = 64), or the query tile itself, which then
  // is free for the next piece only after that.
  static constexpr bool XOWN = DP == 64, XQ = DP == 128 && Q8;
  static constexpr int XCH = DP == 64 ? 16 : TILE / 2048;  // float4 columns of 128 rows a round
  static constexpr int SMEM = 1024 + (QT + KST + VST) * TILE + (Q8 ? SR * (SSLOT + OPB) + SCALES : 0) + (XOWN ? 32768 : 0);
  static_assert(SMEM + 2048 <= kSmemMax, "tiles do not fit in shared memory");
};
template <int CT, int DP>
constexpr int tc_part_floats() {
  return TcCfg<CT, DP>::ROWS * (DP + 2);
}

__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds_u4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts_f32(uint32_t a, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

// Address of 16-byte chunk j (8 elements) of row r in a tile.
__device__ __forceinline__ uint32_t tile_at(uint32_t tile, int r, int j) {
  return tile + (j >> 3) * (kBM * 128) + r * 128 + (((j & 7) ^ (r & 7)) << 4);
}

// TMA load of a box of a map without a swizzle: the destination needs 128 bytes
// of alignment only (tma_load_3d's check asks for a swizzle atom's).
__device__ __forceinline__ void tma_load_rows(void* dst, const CUtensorMap* map, uint64_t* bar, int c1, int c2) {
  if (!TA_CHECK_V((smem_u32(dst) & 127u) == 0u && guard_in_dyn_smem(smem_u32(dst)) && c1 >= 0 && c2 >= 0,
                  smem_u32(dst)))
    return;
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(c1), "r"(c2)
      : "memory");
}

// Arrives at bar when the thread's copies so far have landed.
__device__ __forceinline__ void cp_async_signal(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// d (+)= P V: P 128 x 128 (16-bit, packed in tensor memory), V 128 rows of D,
// read as an MN-major B operand.
template <int D>
__device__ __forceinline__ void mma_weights(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_smem, uint32_t idesc,
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

// Adds the infinities and NaN among the values of the draft's tokens that
// `tok` sees, positions [lo, hi), to the row's result: out (T, dg elements) or
// part (float4 columns `stride` floats apart).
template <typename T>
__device__ __forceinline__ void add_non_finite(const CacheArgs& c, const CacheAttnArgs& a, int b, int h, int tok, int past,
                                            int lo, int hi, int dg, T* out, float* part, int stride) {
  for (int n = max(lo, past); n < hi; ++n) {
    const int d = n - past;
    const bool see = a.tree ? __ldg(a.tree + b * a.tree_b + tok * a.tree_t + d) != 0 : d <= tok;
    if (!see) continue;
    int r;
    const int id = cache_page_id(c, b, n, &r);
    const int row = cache_row(c, h, id, r);
    if (row < 0) continue;
    const T* v = static_cast<const T*>(c.v) + static_cast<size_t>(row) * dg;
    for (int e = 0; e < dg; ++e) {
      const float x = static_cast<float>(v[e]);
      if ((__float_as_uint(x) & 0x7f800000u) != 0x7f800000u) continue;
      if (out) out[e] = static_cast<T>(static_cast<float>(out[e]) + x);
      else part[(e >> 2) * stride + (e & 3)] += x;
    }
  }
}

template <typename T, int CT, int DP>
__global__ void __launch_bounds__(TcCfg<CT, DP>::THREADS, 1)
    attn_cache_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, CacheArgs c,
                         CacheAttnArgs a, int dg) {
  using F = TcCfg<CT, DP>;
  using Ln = Line<F::ROWS, kBN>;
  constexpr bool BF = DT<T>::bf16;
  constexpr bool MBF = BF && !F::Q8;
  constexpr int KST = F::KST, VST = F::VST;
  extern __shared__ uint8_t smem_raw[];
  __shared__ typename Ln::Shared line;
  __shared__ __align__(8) uint64_t bar_q, bar_qfree, bar_k[KST], bar_kempty[KST], bar_v[VST], bar_vempty[VST];
  __shared__ __align__(8) uint64_t bar_s[2], bar_p[2], bar_o[2], bar_ofinal, bar_xfull, bar_xempty;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ int odd[4];  // piece + 1 (mod 4 slots) whose draft holds non-finite values
  __shared__ float xm[kBM], xl[kBM];
  __shared__ float qfac[F::Q8 && BF ? kBM : 1];  // 8 bits: the rows' factors of the scores
  __shared__ __align__(8) uint64_t bar_scan[VST];  // values that have to be looked through have landed
  __shared__ __align__(8) uint64_t bar_stage[2][F::Q8 ? F::SR : 1], bar_sempty[2][F::Q8 ? F::SR : 1];  // 8 bits: keys', values'

  // (a shuffle from lane 0: a value the compiler knows to be the same in the
  // whole warp lives in uniform registers, which is where the MMAs take their
  // operands from)
  auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  let_dependents_launch();
  long long mine, before;
  const long long len = Ln::template length<F::THREADS>(c, a, line, &mine, &before);
  const long long x0 = cut<kTcBlocks>(len, blockIdx.x), x1 = cut<kTcBlocks>(len, blockIdx.x + 1);
  CutUnit* const cuts =
      reinterpret_cast<CutUnit*>(a.ws + static_cast<size_t>(kTcBlocks) * 2 * tc_part_floats<CT, DP>());
  if (x0 >= x1) {
    if (threadIdx.x == 0) write_cut<kTcBlocks, typename Ln::Cursor>(cuts, len, blockIdx.x, x0, x1, nullptr);
    return;
  }
  typename Ln::Cursor u;
  Ln::template find<F::THREADS>(c, a, line, x0, mine, before, u);

  uint8_t* const base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sQ = smem_u32(base);
  auto sK = [&](int st) { return sQ + (F::QT + st) * F::TILE; };
  auto sV = [&](int st) { return sQ + (F::QT + KST + st) * F::TILE; };
  const uint32_t sStage = sQ + (F::QT + KST + VST) * F::TILE;
  const uint32_t sScale = sStage + F::SR * (F::SSLOT + F::OPB);
  const uint32_t sX = F::XOWN ? sScale + F::SCALES : F::XQ ? sQ : sQ + F::TILE;

  WaitCtl ctl{c.err, a.timeout_ns, &abort_flag};
  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(&bar_q, 4);
    mbar_init(&bar_qfree, 8);
    for (int s = 0; s < KST; ++s) {
      mbar_init(&bar_k[s], F::Q8 ? 4 : 1);
      mbar_init(&bar_kempty[s], 1);
    }
    for (int s = 0; s < VST; ++s) {
      mbar_init(&bar_v[s], 4);
      mbar_init(&bar_vempty[s], 1);
      mbar_init(&bar_scan[s], 1);
    }
    if constexpr (F::Q8) {
      for (int s = 0; s < 2 * F::SR; ++s) {
        mbar_init(&bar_stage[0][0] + s, s < F::SR ? 1 + 32 : 1);  // the codes' fetch; keys': a warp's copies of scales
        mbar_init(&bar_sempty[0][0] + s, 4);
      }
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&bar_s[w], 1);
      mbar_init(&bar_p[w], 4);
      mbar_init(&bar_o[w], 1);
    }
    mbar_init(&bar_ofinal, 1);
    mbar_init(&bar_xfull, 4);
    mbar_init(&bar_xempty, 4);
    for (int i = 0; i < 4; ++i) odd[i] = 0;
    fence_mbar_init();
  }
  if (warp == F::MMA) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(tmem_slot);
  if (warp == F::MMA + 3 && lane == 0) write_cut<kTcBlocks>(cuts, len, blockIdx.x, x0, x1, &u);
  const uint32_t col_s[2] = {0u, 128u};
  const uint32_t col_o[2] = {256u, 256u + DP};

  // Pieces of this block: nt tiles from tile u.t of unit u.  `two`: two row
  // tiles that share the keys, else one row tile whose keys the groups share.
  auto piece_tiles = [&](const typename Ln::Cursor& p, long long x) {
    return static_cast<int>(min(static_cast<long long>(p.ntiles - p.t), x1 - x));
  };
  auto piece_two = [&](const typename Ln::Cursor& p) { return !F::Q8 && p.s.q * a.G - p.rt * F::ROWS > kBM; };

  if (warp >= 8 && warp < F::MMA) {
    // ------------------------------------------------------------- helpers
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(F::REG_COPY));
    const int pw = warp & 3, tid = threadIdx.x & 127;
    const bool keys = warp < 12;  // 8 bits: warps 8-11 convert keys, 12-15 values
    // query row i of tile w as an offset into q; false: no such row
    auto q_row = [&](const typename Ln::Cursor& p, int w, int i, long long* off) -> bool {
      const int rr = p.rt * F::ROWS + w * kBM + i;
      if (rr >= p.s.q * a.G) return false;
      const int t = static_cast<int>(a.g_div.div(rr));
      *off = p.b * a.qs[0] + static_cast<long long>(p.h * a.G + (rr - t * a.G)) * a.qs[1] + t * a.qs[2];
      return true;
    };
    // the next piece's query rows towards L2, while this piece runs
    auto prefetch_q = [&](const typename Ln::Cursor& p) {
      for (int w = 0; w < F::QT; ++w) {
        long long off = 0;
        if (!q_row(p, w, tid, &off)) continue;
        const char* at = reinterpret_cast<const char*>(static_cast<const T*>(a.q) + off);
        for (int k = 0; k < dg * 2; k += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + k));
      }
    };
    auto signal = [&](uint64_t* bar) {  // this warp's writes to shared memory, to the MMAs
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    int kt = 0;  // tiles before this piece
    bool ok = true;
    long long x = x0;
    [[maybe_unused]] uint32_t scan_par = 0;  // phase of each stage's bar_scan
    for (int piece = 0; ok && x < x1; ++piece) {
      const int nt = piece_tiles(u, x);
      if constexpr (!F::Q8) {
        constexpr int CH = DP / 8;  // 16-byte chunks per row
        const int ntile = piece_two(u) ? 2 : 1, dch = dg / 8;
        long long offs[2] = {0, 0};
        bool rows[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) rows[w] = q_row(u, w, pw * 32 + lane, &offs[w]);
        if (piece > 0 && !(ok = warp_wait(&bar_qfree, (piece - 1) & 1, ctl, kErrTimeoutMma))) break;
        for (int w = 0; w < ntile; ++w) {
          const long long off = w ? offs[1] : offs[0];
          const bool has = w ? rows[1] : rows[0];
#pragma unroll 8
          for (int k = 0; k < CH; ++k) {
            const int idx = k * 32 + lane, r = idx / CH, j = idx % CH;
            const long long o = __shfl_sync(0xffffffffu, off, r);
            const bool real = __shfl_sync(0xffffffffu, has, r) && j < dch;
            cp_async16(tile_at(sQ + w * F::TILE, pw * 32 + r, j), static_cast<const T*>(a.q) + (real ? o + j * 8 : 0),
                       real);
          }
        }
        cp_async_commit();
        cp_async_wait<0>();
        signal(&bar_q);
        if (x + nt < x1) {
          typename Ln::Cursor n = u;
          Ln::next_unit(c, a, n);
          prefetch_q(n);
        }
        // tiles of values with new tokens
        for (int i = max(0, (u.s.kv - u.s.q) / kBN - u.t); ok && i < nt; ++i) {
          const int vs = (kt + i) % VST;
          const uint32_t tile = sV(vs);
          if (!(ok = warp_wait(&bar_scan[vs], (scan_par >> vs) & 1, ctl, kErrTimeoutTma))) break;
          scan_par ^= 1u << vs;
          constexpr uint32_t EXP = BF ? 0x7f80u : 0x7c00u;
#pragma unroll 4
          for (int k = 0; k < CH; ++k) {
            const int idx = k * 32 + lane, r = pw * 32 + idx / CH;
            const uint32_t at = tile_at(tile, r, idx % CH);
            const uint4 v = lds_u4(at);
            uint32_t wd[4] = {v.x, v.y, v.z, v.w};
            bool hit = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if ((wd[e] & EXP) == EXP) hit = true, wd[e] &= 0xffff0000u;
              if (((wd[e] >> 16) & EXP) == EXP) hit = true, wd[e] &= 0x0000ffffu;
            }
            const int n = (u.t + i) * kBN + r;
            if (n >= u.s.kv) {
              sts_v4(at, 0u, 0u, 0u, 0u);
            } else if (hit && n >= u.s.kv - u.s.q) {  // a new token's
              sts_v4(at, wd[0], wd[1], wd[2], wd[3]);
              odd[piece & 3] = piece + 1;
            }
          }
          signal(&bar_v[vs]);
        }
      } else {
        constexpr int CH = DP / 16;  // 16-byte chunks per row of codes
        if (keys) {  // the piece's queries, a row per thread, in fp16
          long long off = 0;
          const bool has = q_row(u, 0, tid, &off);
          const uint4* p = reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + off);
          // bf16 rows: the row's largest magnitude to [1, 2) by a power of two, so
          // that an element is off by at most 2^-25 of that; the scores of the row
          // get the power back.  (Its exponent, biased, is kept finite for rows of
          // zeros and of infinities.)
          float up = 1.f;
          [[maybe_unused]] float back = 1.f;
          if constexpr (BF) {
            uint32_t top = 0;
#pragma unroll 8
            for (int j = 0; j < DP / 8; ++j) {
              const uint4 v = has && j < dg / 8 ? __ldg(p + j) : make_uint4(0u, 0u, 0u, 0u);
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) top = max(top, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
            }
            const uint32_t ex = min(max(top >> 7, 1u), 253u);
            up = __uint_as_float((254u - ex) << 23);
            back = a.scale_log2 * __uint_as_float(ex << 23);
          }
          uint4 first[8];  // half of the row (D = 128) is here before its place is free
#pragma unroll
          for (int j = 0; j < 8; ++j) first[j] = has && j < dg / 8 ? __ldg(p + j) : make_uint4(0u, 0u, 0u, 0u);
          if (piece > 0 && !(ok = warp_wait(&bar_qfree, (piece - 1) & 1, ctl, kErrTimeoutMma))) break;
          if constexpr (BF) qfac[tid] = back;
#pragma unroll
          for (int j = 0; j < DP / 8; ++j) {
            const uint4 v = j < 8 ? first[j & 7] : has && j < dg / 8 ? __ldg(p + j) : make_uint4(0u, 0u, 0u, 0u);
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
            if constexpr (BF) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = pack2<false>(__uint_as_float(w[k] << 16) * up, __uint_as_float(w[k] & 0xffff0000u) * up);
            }
            sts_v4(tile_at(sQ, tid, j), w[0], w[1], w[2], w[3]);
          }
          signal(&bar_q);
        }
        if (keys && x + nt < x1) {
          typename Ln::Cursor n = u;
          Ln::next_unit(c, a, n);
          prefetch_q(n);
        }
        // A tile's codes, of its half n & 1 -> fp16 in the tile; rows at and
        // behind `end` are zeros.  A warp converts rows pw * 16 .. + 15 of a half.
        const uint32_t ring = sStage + (keys ? 0 : F::SR * F::SSLOT);
        const int pitch = keys ? F::SSLOT : F::OPB;
        auto convert = [&](int n, uint32_t tile, int end) -> bool {
          const int slot = n % F::SR;
          const uint32_t st = ring + slot * pitch;
          if (!warp_wait(&bar_stage[keys ? 0 : 1][slot], (n / F::SR) & 1, ctl, kErrTimeoutTma)) return false;
          if (keys && !(n & 1)) {  // the whole tile's scales have come with its first half
            const uint32_t sc = st + F::OPB, to = sScale + ((n >> 1) % F::SCS) * 1536;
            const int key = (lane >> 4) * 64 + pw * 16 + (lane & 15);  // this lane's of the warp's
            float kx, vscale;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(kx) : "r"(sc + key * 4) : "memory");
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vscale) : "r"(sc + 512 + key * 4) : "memory");
            // A value whose scale is not a number, or negative: through its key's
            // scores it makes the rows that see it NaN, and does not reach the
            // others.  No scale stands for a value of zero.
            if (!(vscale >= 0.f && vscale < INFINITY)) kx = __uint_as_float(0x7fc00000u), vscale = 1.f;
            if (key >= end) kx = 0.f, vscale = 1.f;  // whatever the memory holds there
            const float lsv = lg2(fmaxf(vscale, kMinScale));
            sts_f32(to + key * 4, kx);
            sts_f32(to + 512 + key * 4, lsv);
            sts_f32(to + 1024 + key * 4, ex2(0.5f * (kSumUp - lsv)));
          }
          // Chunk of 16 codes -> two of 8 fp16.  Eight neighbouring lanes take
          // four chunks of a row and the other four of the next one (D = 128),
          // or two rows (D = 64): their loads and their stores then cover all
          // banks once.
          const int row0 = (n & 1) * 64;
          auto place = [&](int i, int* r, int* j) {  // row of the half, chunk
            if constexpr (CH == 8) {
              *r = pw * 16 + 2 * ((i >> 1) * 4 + (lane >> 3)) + ((lane >> 2) & 1);
              *j = (lane & 3) + 4 * (((lane >> 2) & 1) ^ (i & 1));
            } else {
              *r = pw * 16 + i * 8 + (lane >> 2);
              *j = lane & 3;
            }
          };
          // (all loads first: a load must not wait for the stores before it)
          uint4 codes[CH / 2];
#pragma unroll
          for (int i = 0; i < CH / 2; ++i) {
            int r, j;
            place(i, &r, &j);
            codes[i] = lds_u4(st + r * DP + j * 16);
          }
#pragma unroll
          for (int i = 0; i < CH / 2; ++i) {
            int r, j;
            place(i, &r, &j);
            r += row0;
            uint4 v = codes[i];
            if (r >= end) v = make_uint4(0u, 0u, 0u, 0u);
            uint32_t h[8];
            code4_to_f16<CT>(v.x, h[0], h[1]);
            code4_to_f16<CT>(v.y, h[2], h[3]);
            code4_to_f16<CT>(v.z, h[4], h[5]);
            code4_to_f16<CT>(v.w, h[6], h[7]);
            sts_v4(tile_at(tile, r, 2 * j), h[0], h[1], h[2], h[3]);
            sts_v4(tile_at(tile, r, 2 * j + 1), h[4], h[5], h[6], h[7]);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_sempty[keys ? 0 : 1][slot]);
          return true;
        };
        for (int i = 0; i < nt; ++i) {
          const int t = kt + i, ks = t % KST, vs = t % VST, end = u.s.kv - (u.t + i) * kBN;
          uint64_t* const empty = keys ? &bar_kempty[ks] : &bar_vempty[vs];
          static_assert(KST == VST, "one test for both rings");
          if (t >= KST && !(ok = warp_wait(empty, (t / KST - 1) & 1, ctl, kErrTimeoutMma))) break;
#pragma unroll 1
          for (int half = 0; ok && half < 2; ++half) ok = convert(2 * t + half, keys ? sK(ks) : sV(vs), end);
          if (!ok) break;
          signal(keys ? &bar_k[ks] : &bar_v[vs]);
        }
      }
      kt += nt;
      x += nt;
      if (x < x1) Ln::next_unit(c, a, u);
    }
  } else if (warp >= F::MMA) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(F::REG_MMA));
    if (warp == F::MMA) {
      // ------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_qk = idesc_f16(kBM, kBN, MBF, false, false);
      constexpr uint32_t idesc_pv = idesc_f16(kBM, DP, MBF, false, true);
      // The tiles' stages and phases are counted on, not divided out: this
      // warp shares its issue slots with the softmax, and what it issues
      // between two products is time the tensor core waits.
      int ks = 0, vs = 0;                     // stages of the next tiles
      uint32_t kp = 0, vp = 0, pp0 = 0, pp1 = 0;  // phases: of those stages, of the groups' P
      bool ok = true;
      long long x = x0;
      for (int piece = 0; ok; ++piece) {
        const int nt = uniform(piece_tiles(u, x));
        const bool two = uniform(piece_two(u)) != 0;
        auto next_k = [&]() {
          commit_el(&bar_kempty[ks]);
          if (++ks == KST) ks = 0, kp ^= 1;
        };
        auto next_v = [&]() {
          commit_el(&bar_vempty[vs]);
          if (++vs == VST) vs = 0, vp ^= 1;
        };
        // S of group w with the next key tile, which `first` waits for and `last` releases
        auto issue_s = [&](int w, bool first, bool last) -> bool {
          if (first && !warp_wait(&bar_k[ks], kp, ctl, kErrTimeoutTma)) return false;
          tc_fence_after();
          mma_abT<DP>(tmem + col_s[w], sQ + (two ? w * F::TILE : 0), sK(ks), idesc_qk);
          commit_el(&bar_s[w]);
          if (last) next_k();
          return true;
        };
        auto issue_pv = [&](int w, bool first, bool last, bool add) -> bool {
          if (first && !warp_wait(&bar_v[vs], vp, ctl, kErrTimeoutTma)) return false;
          if (!warp_wait(&bar_p[w], w ? pp1 : pp0, ctl, kErrTimeoutSoftmax)) return false;
          if (w) pp1 ^= 1;
          else pp0 ^= 1;
          tc_fence_after();
          mma_weights<DP>(tmem + col_o[w], tmem + col_s[w], sV(vs), idesc_pv, add);
          commit_el(&bar_o[w]);
          if (last) next_v();
          return true;
        };
        ok = warp_wait(&bar_q, piece & 1, ctl, kErrTimeoutTma);
        if (two) {
          ok = ok && issue_s(0, true, false) && issue_s(1, false, true);
          for (int i = 0; ok && i < nt; ++i) {
            const bool more = i + 1 < nt;
            ok = issue_pv(0, true, false, i > 0);
            if (ok && more) ok = issue_s(0, true, false);
            ok = ok && issue_pv(1, false, true, i > 0);
            if (ok && more) ok = issue_s(1, false, true);
          }
        } else {  // tile i with group i & 1
          ok = ok && issue_s(0, true, true);
          if (ok && nt > 1) ok = issue_s(1, true, true);
          for (int i = 0; ok && i < nt; i += 2) {
            ok = issue_pv(0, true, true, i > 0);
            if (ok && i + 2 < nt) ok = issue_s(0, true, true);
            if (ok && i + 1 < nt) {
              ok = issue_pv(1, true, true, i > 0);
              if (ok && i + 3 < nt) ok = issue_s(1, true, true);
            }
          }
        }
        if (ok) commit_el(&bar_ofinal);
        x += nt;
        if (uniform(x >= x1)) break;
        Ln::next_unit(c, a, u);
      }
    }
    if (warp == F::MMA + 1 || warp == F::MMA + 2) {
      // ------------------------------------------------------- TMA fetches
      const bool is_k = warp == F::MMA + 1;
      const int box = a.box_rows, nbox = kBN / box;
      const int outside = c.num_pages * c.Hkv;  // past the maps: reads as zeros
      // this lane's box of tile t: the table's entry and the first row (-1: none)
      auto look_up = [&](const typename Ln::Cursor& p, int t, int* r) -> int {
        const int n = t * kBN + lane * box;
        *r = -1;
        return lane >= nbox || n >= p.s.kv ? 0 : cache_page_id(c, p.b, n, r);
      };
      // the same a tile later, when the entry is there: page (-1: none) and row
      auto take = [&](int id, int* row) -> int {
        if (*row >= 0) {
          if (static_cast<unsigned>(id) < static_cast<unsigned>(c.num_pages)) return id;
          cache_error(c.err);
        }
        *row = 0;
        return -1;
      };
      if (lane == 0) tma_prefetch_desc(is_k ? &tm_k : &tm_v);
      int never = 0;
      WaitCtl drain{c.err, a.timeout_ns, &never};  // for copies in flight, also after a time-out elsewhere
      bool ok = true;
      int kt = 0;
      long long x = x0;
      int r, id = look_up(u, u.t, &r);  // of the next tile
      if constexpr (!F::Q8) {
        const int depth = is_k ? KST : VST;
        uint64_t* const full = is_k ? bar_k : bar_v;
        uint64_t* const empty = is_k ? bar_kempty : bar_vempty;
        uint32_t scanned = 0, scan_par = 0;  // stages whose last tile went to bar_scan; its phase
        for (; ok && x < x1; ++x, ++kt) {
          const int st = kt % depth;
          int row = r;
          const int page = take(id, &row), head = page < 0 ? outside : page * c.Hkv + u.h;
          const bool scan = !is_k && (u.t + 1) * kBN > u.s.kv - u.s.q;
          if (x + 1 < x1) {
            Ln::next_tile(c, a, u);
            id = look_up(u, u.t, &r);
          }
          if (kt >= depth && !(ok = warp_wait(&empty[st], (kt / depth - 1) & 1, ctl, kErrTimeoutMma))) break;
          uint64_t* const bar = scan ? &bar_scan[st] : &full[st];
          scanned = scan ? scanned | (1u << st) : scanned & ~(1u << st);
          scan_par ^= scan ? 1u << st : 0u;
          if (lane == 0) mbar_expect_tx(bar, F::TILE);
          else if (!is_k && !scan && lane < 4) mbar_arrive(bar);  // in place of the four helpers
          __syncwarp();
          if (lane < nbox) {
            const uint32_t dst = (is_k ? sK(st) : sV(st)) + lane * box * 128;
#pragma unroll
            for (int kb = 0; kb < DP / 64; ++kb)
              tma_load_3d(base + (dst - sQ) + kb * (kBM * 128), is_k ? &tm_k : &tm_v, bar, kb * 64, row, head);
          }
        }
        if (lane == 0) {
          for (int t = max(0, kt - depth); t < kt; ++t) {
            const int st = t % depth;
            if ((scanned >> st) & 1u) mbar_wait(&bar_scan[st], ~(scan_par >> st) & 1, drain, kErrTimeoutTma);
            else mbar_wait(&full[st], (t / depth) & 1, drain, kErrTimeoutTma);
          }
        }
      } else {
        // A warp and a ring each for keys and values, in halves of a tile: the
        // rings are short beside a fetch's 1.2 us.
        const uint32_t ring = sStage + (is_k ? 0 : F::SR * F::SSLOT);
        const int pitch = is_k ? F::SSLOT : F::OPB;
        uint64_t* const full = bar_stage[is_k ? 0 : 1];
        uint64_t* const empty = bar_sempty[is_k ? 0 : 1];
        int n = 0;
        for (; ok && x < x1; ++x) {
          int row = r;
          const int h = u.h, page = take(id, &row);
          if (x + 1 < x1) {
            Ln::next_tile(c, a, u);
            id = look_up(u, u.t, &r);
          }
          for (int half = 0; half < 2; ++half, ++n) {
            const int slot = n % F::SR;
            if (n >= F::SR && !(ok = warp_wait(&empty[slot], (n / F::SR - 1) & 1, ctl, kErrTimeoutMma))) break;
            const uint32_t st = ring + slot * pitch;
            if (lane == 0) mbar_expect_tx(&full[slot], F::OPB);
            __syncwarp();
            const int first = half * (nbox >> 1);
            if (lane >= first && lane < first + (nbox >> 1))
              tma_load_rows(base + (st - sQ) + (lane - first) * box * DP, is_k ? &tm_k : &tm_v, &full[slot], row,
                            page >= 0 ? page * c.Hkv + h : outside);
            if (!is_k) continue;
            if (half == 0) {  // both scales of the tile's keys, four keys' a lane, zeros for none
              const int b = lane * 4 / box;
              const int pg = __shfl_sync(0xffffffffu, page, b);
              const int rw = __shfl_sync(0xffffffffu, row, b) + lane * 4 % box;
              const size_t at = pg < 0 ? 0 : static_cast<size_t>((pg * c.Hkv + h) * static_cast<int>(c.page.d) + rw);
              cp_async16(st + F::OPB + lane * 16, c.ks + at, pg >= 0);
              cp_async16(st + F::OPB + 512 + lane * 16, c.vs + at, pg >= 0);
            }
            cp_async_signal(&full[slot]);
          }
        }
        if (lane == 0)
          for (int t = max(0, n - F::SR); t < n; ++t)
            mbar_wait(&full[t % F::SR], (t / F::SR) & 1, drain, kErrTimeoutTma);
      }
    }
  } else {
    // ---------------------------------- softmax, correction, epilogue (group w)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(F::REG_SOFTMAX));
    const int w = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_addr = lane_addr + col_s[w], o_addr = lane_addr + col_o[w];
    int ns = 0;   // tiles of this group so far
    int kt0 = 0;  // tiles of the block before this piece
    int nx = 0;   // hand-overs between the groups so far
    bool ok = true;
    long long x = x0;
    for (int piece = 0; ok && x < x1; ++piece) {
      const int nt = piece_tiles(u, x);
      const bool two = piece_two(u);
      const int n = two ? nt : (nt + 1 - w) >> 1;
      const int rr = u.rt * F::ROWS + (two ? w * kBM : 0) + r;
      const int tok = rr < u.s.q * a.G ? static_cast<int>(a.g_div.div(rr)) : -1;
      const int past = u.s.kv - u.s.q;
      // Which of the keys k0 .. k0 + 127 the row sees (bit j of the 128: key
      // k0 + j): those before the new tokens, and of these by the tree or, without
      // one, those up to its own.
      auto see_keys = [&](int k0, uint32_t (&vis)[4]) {
        if (!a.tree) {
          const int lim = min(u.s.kv - 1, past + tok) - k0;  // tok -1: rows that do not exist
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int bits = lim + 1 - 32 * k;
            vis[k] = bits <= 0 ? 0u : bits >= 32 ? 0xffffffffu : (1u << bits) - 1u;
          }
          return;
        }
        // The warp's tokens, eight at a time: a load brings 32 keys' bytes of a
        // token, all 32 loads are in flight together.
        const int d0 = k0 - past;
#pragma unroll
        for (int k = 0; k < 4; ++k) vis[k] = 0u;
        const int lo = __shfl_sync(0xffffffffu, tok, 0);
        const int hi = __reduce_max_sync(0xffffffffu, tok);
        const uint8_t* const rows = a.tree + u.b * a.tree_b;
#pragma unroll 1
        for (int t0 = lo; t0 >= 0 && t0 <= hi; t0 += 8) {
          uint32_t byte[4][8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int d = d0 + 32 * k + lane;
            const bool in = d >= 0 && d < u.s.q;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              byte[k][e] = in ? __ldg(rows + min(t0 + e, hi) * a.tree_t + d) : d < 0 ? 1u : 0u;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t word = __ballot_sync(0xffffffffu, byte[k][e] != 0u);
              if (tok == t0 + e) vis[k] = word;
            }
          }
        }
      };
      // The group's first tile with new tokens, looked up while the piece's
      // first scores are under way.
      uint32_t vis[4] = {0u, 0u, 0u, 0u};
      int vis_t = max(0, past / kBN - u.t);
      if (!two) vis_t = vis_t <= w ? 0 : (vis_t - w + 1) >> 1;
      float m_ref = -INFINITY, l = 0.f;
      [[maybe_unused]] float row_f = a.scale_log2;  // 8 bits: the row's factor of the scores
      for (int t = 0; t < n; ++t, ++ns) {
        const int ti = two ? t : 2 * t + w;       // tile of the piece
        const int k0 = (u.t + ti) * kBN;
        const bool masked = k0 + kBN > past;
        if (t == 0 ? vis_t < n : masked && t != vis_t)
          see_keys(t == 0 ? (u.t + (two ? vis_t : 2 * vis_t + w)) * kBN : k0, vis);
        if (!(ok = warp_wait(&bar_s[w], ns & 1, ctl, kErrTimeoutMma))) break;
        tc_fence_after();
        if constexpr (F::Q8 && BF) {
          if (t == 0) row_f = const_cast<volatile float*>(qfac)[r];
        }
        const float f = F::Q8 ? 1.f : a.scale_log2;  // of the scores (8 bits: row_f, in them already)
        [[maybe_unused]] const uint32_t scales = sScale + ((kt0 + ti) % F::SCS) * 1536;
        // 16 bits: the row's 128 scores in registers.  8 bits: two passes over S
        // in tensor memory, XC columns at a time (scales, mask and maximum;
        // weights): the loops of the softmax, the conversions and the MMA warp
        // then stay in the instruction cache together (with the row in registers
        // a third of all stalls were missing instructions: 212 us against 140 at
        // 128 rows of D = 128, e4m3, when that was changed; alone, beside idle
        // helpers, one pass is faster: 377 us against 496 for 16 bits' chunk of
        // 2048 over 16384).
        constexpr int XC = F::Q8 ? 32 : 128;
        float y[XC];
        auto load = [&](int c0, bool first) {  // 8 bits: the first pass leaves what the second takes
          uint32_t s[XC];
#pragma unroll
          for (int k = 0; k < XC / 32; ++k) tmem_ld_x32(s_addr + c0 + 32 * k, TB_CHUNK(s, k));
#pragma unroll
          for (int k = 0; k < XC / 32; ++k) tmem_ld_wait(TB_CHUNK(s, k));
#pragma unroll
          for (int j = 0; j < XC; ++j) y[j] = __uint_as_float(s[j]);
          if constexpr (F::Q8) {
            if (!first) return;
#pragma unroll
            for (int j = 0; j < XC; j += 4) {
              const float4 kx = lds_f4(scales + (c0 + j) * 4), vx = lds_f4(scales + 512 + (c0 + j) * 4);
              const float2 f2 = make_float2(row_f, row_f);
              // (the two factors first: a large key's with a small query's)
              const float2 p = ffma2(make_float2(y[j], y[j + 1]), fmul2(make_float2(kx.x, kx.y), f2), make_float2(vx.x, vx.y));
              const float2 q = ffma2(make_float2(y[j + 2], y[j + 3]), fmul2(make_float2(kx.z, kx.w), f2), make_float2(vx.z, vx.w));
              y[j] = p.x, y[j + 1] = p.y, y[j + 2] = q.x, y[j + 3] = q.y;
            }
          }
          if (masked) {
#pragma unroll
            for (int k = 0; k < XC / 32; ++k) {
              uint32_t seen = vis[k];
              if constexpr (XC < 128) {
                const int at = c0 / 32 + k;
                seen = at == 0 ? vis[0] : at == 1 ? vis[1] : at == 2 ? vis[2] : vis[3];
              }
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!((seen >> j) & 1u)) y[32 * k + j] = -INFINITY;
            }
          }
          if constexpr (F::Q8) {
#pragma unroll
            for (int j = 0; j < XC; ++j) s[j] = __float_as_uint(y[j]);
#pragma unroll
            for (int k = 0; k < XC / 32; ++k) tmem_st_x32(s_addr + c0 + 32 * k, TB_CHUNK(s, k));
          }
        };
        float mx = -INFINITY;
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += XC) {
          load(c0, true);
          constexpr int CHAINS = XC >= 64 ? 8 : 4;  // of three-input maxima
          float mc[CHAINS];
#pragma unroll
          for (int k = 0; k < CHAINS; ++k) {
            mc[k] = fmax3(y[k], y[CHAINS + k], y[2 * CHAINS + k]);
#pragma unroll
            for (int j = 3 * CHAINS; j + CHAINS < XC; j += 2 * CHAINS) mc[k] = fmax3(mc[k], y[j + k], y[j + CHAINS + k]);
            mc[k] = fmaxf(mc[k], y[XC - CHAINS + k]);
          }
#pragma unroll
          for (int k = 0; k < CHAINS; k += 2) mx = fmax3(mx, mc[k], mc[k + 1]);
        }
        if constexpr (F::Q8) tmem_st_wait();
        const float m_new = fmaxf(m_ref, mx * f);
        bool resc = false;
        float alpha = 1.f;
        if (t == 0) {
          m_ref = m_new;
        } else if (m_new > m_ref + kRescaleThreshold) {
          resc = true;
          alpha = ex2(m_ref - m_new);
          if constexpr (F::Q8) l = lower_sum(l, m_ref - m_new);
          m_ref = m_new;
        }
        const float neg_m = (m_ref == -INFINITY) ? 0.f : -m_ref;
        const float2 sc2 = make_float2(f, f);
        const float2 nm2 = make_float2(neg_m, neg_m);
        const float2 half2 = make_float2(0.5f, 0.5f), nmh2 = make_float2(0.5f * neg_m, 0.5f * neg_m);
        float2 rs2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += XC) {
          if constexpr (F::Q8) load(c0, false);
#pragma unroll
          for (int k = 0; k < XC / 16; ++k) {
            uint32_t pk[8];
            [[maybe_unused]] float4 root;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 y2 = make_float2(y[16 * k + 2 * e], y[16 * k + 2 * e + 1]);
              const float2 t2 = F::Q8 ? ffma2(y2, half2, nmh2) : ffma2(y2, sc2, nm2);
              float2 p2 = make_float2(ex2(t2.x), ex2(t2.y));
              if constexpr (F::Q8) {  // the weight's root (attn_cache.cuh)
                if (e % 2 == 0) root = lds_f4(scales + 1024 + (c0 + 16 * k + 2 * e) * 4);
                const float2 x = fmul2(p2, e % 2 ? make_float2(root.z, root.w) : make_float2(root.x, root.y));
                rs2[e & 3] = ffma2(x, x, rs2[e & 3]);
                p2 = fmul2(p2, p2);
              } else {
                rs2[e & 3] = fadd2(rs2[e & 3], p2);
              }
              pk[e] = pack2<MBF>(p2.x, p2.y);
            }
            tmem_st_x8(s_addr + c0 / 2 + 8 * k, pk);  // over columns that are read
          }
        }
        const float2 rsa = fadd2(fadd2(rs2[0], rs2[1]), fadd2(rs2[2], rs2[3]));
        l = (F::Q8 ? l : l * alpha) + (rsa.x + rsa.y);
        if (t > 0 && __any_sync(0xffffffffu, resc)) {
          if (!(ok = warp_wait(&bar_o[w], (ns - 1) & 1, ctl, kErrTimeoutMma))) break;
          tc_fence_after();
          const float o_alpha = keep_infinite(alpha);
#pragma unroll
          for (int k = 0; k < DP / 32; ++k) {
            uint32_t ov[32];
            tmem_ld_x32(o_addr + 32 * k, ov);
            tmem_ld_wait(ov);
#pragma unroll
            for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * o_alpha);
            tmem_st_x32(o_addr + 32 * k, ov);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_p[w]);
      }
      // ---------------------------------------------------------- epilogue
      ok = __all_sync(0xffffffffu, ok) && warp_wait(&bar_ofinal, piece & 1, ctl, kErrTimeoutMma);
      if (!ok) break;
      tc_fence_after();
      const bool odd_values = !F::Q8 && *const_cast<volatile int*>(&odd[piece & 3]) == piece + 1;
      // Q's memory is free for the next piece now, or after the join where
      // that piece may write what the join uses
      const bool q_early = two || F::XOWN || (!F::XQ && u.s.q * a.G <= kBM && u.h + 1 < c.Hkv);
      if (q_early) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_qfree);
      }
      // one row tile: group 1 hands its state over in rounds of XCH columns
      constexpr int NCH = DP / 4;                                  // float4 columns
      constexpr int XCH = F::XCH, XR = NCH / XCH;
      float f0 = 1.f, f1 = 0.f;
      const bool whole = u.t == 0 && nt == u.ntiles;
      float* const part = a.ws + (static_cast<size_t>(blockIdx.x) * 2 + (x > x0 ? 1 : 0)) * tc_part_floats<CT, DP>();
      const int prow = (two ? w * kBM : 0) + r;
      const int hq = u.h * a.G + (tok >= 0 ? rr - tok * a.G : 0);
      T* const out = static_cast<T*>(a.o) + (tok >= 0 ? u.b * a.os[0] + hq * a.os[1] + tok * a.os[2] : 0);
      if (!two && w == 1) {
        xm[r] = m_ref;
        xl[r] = l;
      }
#pragma unroll 1
      for (int round = 0; round < XR; ++round) {
        if (!two && w == 1) {
          if (nx > 0 && !(ok = warp_wait(&bar_xempty, (nx - 1) & 1, ctl, kErrTimeoutSoftmax))) break;
          // (round 0 of a later piece: group 0 has read the last one's rows)
#pragma unroll 1
          for (int k = 0; k < XCH; k += 8) {
            uint32_t ov[32];
            if (n > 0) {
              tmem_ld_x32(o_addr + (round * XCH + k) * 4, ov);
              tmem_ld_wait(ov);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) ov[j] = 0u;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
              sts_v4(sX + ((k + j) * kBM + r) * 16, ov[4 * j], ov[4 * j + 1], ov[4 * j + 2], ov[4 * j + 3]);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_xfull);
          ++nx;
          continue;
        }
        if (!two) {
          if (!(ok = warp_wait(&bar_xfull, nx & 1, ctl, kErrTimeoutSoftmax))) break;
          ++nx;
          if (round == 0) {
            const float m1 = xm[r], l1 = xl[r];
            const float mm = fmaxf(m_ref, m1);
            f0 = m_ref == -INFINITY ? 0.f : ex2(m_ref - mm);
            f1 = m1 == -INFINITY ? 0.f : ex2(m1 - mm);
            l = mm == -INFINITY ? l + l1  // NaN stays
                : F::Q8         ? lower_sum(l, m_ref - mm) + lower_sum(l1, m1 - mm)
                                : l * f0 + l1 * f1;
            f0 = keep_infinite(f0), f1 = keep_infinite(f1);
            m_ref = mm;
          }
        }
        const float norm = whole ? sum_norm<CT>(l) : 1.f;
#pragma unroll 1
        for (int k = 0; k < XCH; k += 8) {
          const int ch0 = round * XCH + k;
          uint32_t ov[32];
          tmem_ld_x32(o_addr + ch0 * 4, ov);
          tmem_ld_wait(ov);
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(ov[j]);
          if (!two) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 y = lds_f4(sX + ((k + j) * kBM + r) * 16);
              v[4 * j] = fmaf(v[4 * j], f0, y.x * f1);
              v[4 * j + 1] = fmaf(v[4 * j + 1], f0, y.y * f1);
              v[4 * j + 2] = fmaf(v[4 * j + 2], f0, y.z * f1);
              v[4 * j + 3] = fmaf(v[4 * j + 3], f0, y.w * f1);
            }
          }
          if (whole) {
            if (tok >= 0) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint4 o;
                o.x = pack2<BF>(v[8 * j] * norm, v[8 * j + 1] * norm);
                o.y = pack2<BF>(v[8 * j + 2] * norm, v[8 * j + 3] * norm);
                o.z = pack2<BF>(v[8 * j + 4] * norm, v[8 * j + 5] * norm);
                o.w = pack2<BF>(v[8 * j + 6] * norm, v[8 * j + 7] * norm);
                if (ch0 * 4 + 8 * j < dg) *reinterpret_cast<uint4*>(out + ch0 * 4 + 8 * j) = o;
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if ((ch0 + j) * 4 < dg)
                reinterpret_cast<float4*>(part)[(ch0 + j) * F::ROWS + prow] =
                    make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          }
        }
        if (!two) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_xempty);
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (two || w == 0) {
        if (!whole) {
          part[F::ROWS * DP + prow] = m_ref;
          part[F::ROWS * (DP + 1) + prow] = l;
        } else if (tok >= 0) {
          a.lse[(static_cast<long long>(u.b) * a.Hq + hq) * c.T + tok] = row_lse<CT>(m_ref, l);
        }
        if constexpr (!F::Q8) {
          if (odd_values && tok >= 0)
            add_non_finite<T>(c, a, u.b, u.h, tok, past, u.t * kBN, min(u.s.kv, (u.t + nt) * kBN), dg,
                              whole ? out : nullptr, part + prow * 4, F::ROWS * 4);
        }
      }
      tc_fence_before();
      if (!q_early) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_qfree);
      }
      kt0 += nt;
      x += nt;
      if (x < x1) Ln::next_unit(c, a, u);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == F::MMA) tmem_dealloc(tmem, 512);
}

// Joins the partial states of the units that block borders cut: block (i, y)
// joins rows 32 y .. 32 y + 31 of the unit that border i + 1 is the first to
// cut, a row per lane, every eighth group of four columns per warp.
template <typename T, int CT, int DP>
__global__ void __launch_bounds__(256) attn_cache_tc_join_kernel(CacheArgs c, CacheAttnArgs a, int dg) {
  using F = TcCfg<CT, DP>;
  constexpr bool BF = DT<T>::bf16;
  constexpr int NC = DP / 32;  // float4 columns per thread
  __shared__ int slots[kTcBlocks];
  __shared__ float fs[kTcBlocks][32];
  __shared__ float red[8][32];
  wait_for_main_kernel();  // every block: the next kernel in the stream may start when this one has ended
  const CutUnit u =
      reinterpret_cast<const CutUnit*>(a.ws + static_cast<size_t>(kTcBlocks) * 2 * tc_part_floats<CT, DP>())[blockIdx.x + 1];
  const int parts = u.parts, rows = u.q * a.G;
  if (parts == 0 || u.rt * F::ROWS + static_cast<int>(blockIdx.y) * 32 >= rows) return;
  for (int i = threadIdx.x; i < parts; i += 256) slots[i] = part_slot<kTcBlocks>(u, i);
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int prow = blockIdx.y * 32 + lane, rr = u.rt * F::ROWS + prow;
  auto part = [&](int i) { return a.ws + static_cast<size_t>(slots[i]) * tc_part_floats<CT, DP>(); };
  // every warp looks at every eighth part's maximum and sum
  float mm = -INFINITY;
  for (int i = warp; i < parts; i += 8)
    if (slots[i] >= 0) mm = fmaxf(mm, __ldcg(part(i) + F::ROWS * DP + prow));
  red[warp][lane] = mm;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) mm = fmaxf(mm, red[w][lane]);
  __syncthreads();
  float ll = 0.f;
  for (int i = warp; i < parts; i += 8) {
    float f = 0.f;
    if (slots[i] >= 0) {
      const float pm = __ldcg(part(i) + F::ROWS * DP + prow), pl = __ldcg(part(i) + F::ROWS * (DP + 1) + prow);
      f = pm == -INFINITY ? 0.f : ex2(pm - mm);
      // a NaN sum stays one where no score was a number
      ll += mm == -INFINITY ? pl : F::Q8 ? lower_sum(pl, pm - mm) : pl * f;
    }
    fs[i][lane] = keep_infinite(f);
  }
  red[warp][lane] = ll;
  __syncthreads();
  ll = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) ll += red[w][lane];
  float v[NC][4] = {};
#pragma unroll 4
  for (int i = 0; i < parts; ++i) {
    const float f = fs[i][lane];
    if (slots[i] < 0) continue;  // a block without a piece
    const float4* p = reinterpret_cast<const float4*>(part(i)) + prow;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int ch = warp + 8 * k;
      if (ch * 4 < dg) {
        const float4 y = __ldcg(p + ch * F::ROWS);
        v[k][0] = fmaf(y.x, f, v[k][0]);
        v[k][1] = fmaf(y.y, f, v[k][1]);
        v[k][2] = fmaf(y.z, f, v[k][2]);
        v[k][3] = fmaf(y.w, f, v[k][3]);
      }
    }
  }
  if (rr >= rows) return;
  const int t = static_cast<int>(a.g_div.div(rr)), hq = u.h * a.G + (rr - t * a.G);
  const float norm = sum_norm<CT>(ll);
  T* const out = static_cast<T*>(a.o) + u.b * a.os[0] + hq * a.os[1] + t * a.os[2];
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int ch = warp + 8 * k;
    if (ch * 4 < dg) {
      uint2 o;
      o.x = pack2<BF>(v[k][0] * norm, v[k][1] * norm);
      o.y = pack2<BF>(v[k][2] * norm, v[k][3] * norm);
      *reinterpret_cast<uint2*>(out + ch * 4) = o;
    }
  }
  if (warp == 0) a.lse[(static_cast<long long>(u.b) * a.Hq + hq) * c.T + t] = row_lse<CT>(mm, ll);
}

template <typename T, int CT, int DP>
cudaError_t run_tc(int dg, const PageMaps& m, const CacheArgs& c, const CacheAttnArgs& a, cudaStream_t s) {
  static std::atomic<bool> done[kMaxDevices];
  auto* kern = attn_cache_tc_kernel<T, CT, DP>;
  constexpr int smem = TcCfg<CT, DP>::SMEM;
  cudaError_t e = smem_attr_once(kern, smem, done);
  if (e != cudaSuccess) return e;
  prof_begin("attn_cache_tc", s);
  kern<<<kTcBlocks, TcCfg<CT, DP>::THREADS, smem, s>>>(m.k, m.v, c, a, dg);
  prof_end(s);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  prof_begin("attn_cache_tc_join", s);
  e = launch_join(attn_cache_tc_join_kernel<T, CT, DP>, dim3(kTcBlocks - 1, TcCfg<CT, DP>::ROWS / 32), 256, s, c, a, dg);
  prof_end(s);
  return e;
}
template <int CT>
size_t tc_ws_bytes(int D) {
  const int f = D <= 64 ? tc_part_floats<CT, 64>() : tc_part_floats<CT, 128>();
  return static_cast<size_t>(kTcBlocks) * (2 * f * sizeof(float) + sizeof(CutUnit));
}

}  // namespace
}  // namespace ta
