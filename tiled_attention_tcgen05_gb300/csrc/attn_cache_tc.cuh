// Attention of new tokens over a paged key/value cache on the tensor cores
// (tcgen05), for many query rows per key head: drafts' trees, prompts' chunks.
//
// A block works through its piece of the line (attn_cache.cuh) with the roles
//   warps 0-3, 4-7  two softmax groups, a thread per query row (= TMEM lane);
//   warps 8-11      copy Q and the key and value tiles into shared memory;
//   warp 12         issues the MMAs: S = Q K^T, O += P V with P in TMEM;
// and the registers handed to the softmax groups (setmaxnreg).  The groups
// alternate on the tensor core:  S0 S1 | PV0 S0' | PV1 S1' | ...  Units of more
// than 128 rows give each group a row tile of its own and both the same keys;
// units of up to 128 rows give both groups the same rows and every other
// key tile, and join the two states at the end: the softmax of one tile
// then runs beside the other's MMAs in either case.
//
// Pages can have any size, so tiles are gathered row by row with 16-byte
// cp.async into the 128-byte-swizzled layout that the MMA descriptors read.
// 8-bit codes are gathered into a staging ring several tiles ahead and turned
// into fp16 codes (exact) by the threads that copied them; scores take their
// key's scale and the value's scale goes into the exponent as in
// attn_cache.cu.
//
// Infinities and NaN among a draft's values would reach rows that must not
// see them (0 * NaN): the copying warps take them out of the tile, and the
// rows that do see them get them added to their result.
#pragma once
#include "attn_cache.cuh"
#include "common.cuh"
#include "fwd_mma.cuh"
#include "launch.h"

namespace ta {
namespace {

constexpr int kTcBlocks = 152;    // one per SM
constexpr int kTcThreads = 512;   // 16 warps; 13 to 15 only fill their register group
constexpr int kTcRegsSoftmax = 184, kTcRegsCopy = 96, kTcRegsMma = 48;
static_assert(256 * kTcRegsSoftmax + 128 * kTcRegsCopy + 128 * kTcRegsMma <= kTcThreads * 128,
              "the groups' registers come out of the launch's");

template <int CT, int DP>
struct TcCfg {
  static constexpr bool Q8 = CT != kCache16;
  static constexpr int TILE = DP / 64 * (kBM * 128);
  static constexpr int QT = Q8 ? 1 : 2;                  // query tiles
  static constexpr int ROWS = QT * kBM;                  // rows per unit
  static constexpr int KST = Q8 ? (DP == 128 ? 2 : 3) : (DP == 128 ? 3 : 4);
  static constexpr int VST = Q8 ? KST : (DP == 128 ? 2 : 4);
  static constexpr int OPB = Q8 ? 128 * DP : 0;          // codes of one tile
  static constexpr int SR = Q8 ? (DP == 128 ? 3 : 6) : 0;  // staging ring
  static constexpr int SSLOT = OPB + 1024;               // and their scales (K tiles)
  static constexpr int SCS = KST + 2;                    // ring of scales for the softmax
  static constexpr int SCB = 128 * 12;                   // K scale, log2 and 1 / of the V scale
  static constexpr int SMEM = 1024 + (QT + KST + VST) * TILE + (Q8 ? SR * SSLOT + SCS * SCB : 0);
  static constexpr int XCH = QT * TILE / 2048;           // float4 columns of 128 rows that fit over Q
  static_assert(SMEM + 2048 <= kSmemMax, "tiles do not fit in shared memory");
};
template <int CT, int DP>
constexpr int tc_part_floats() {
  return TcCfg<CT, DP>::ROWS * (DP + 2);
}

__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(ok)
               : "r"(smem_u32(bar)), "r"(parity)
               : "memory");
  return ok != 0;
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
__global__ void __launch_bounds__(kTcThreads, 1) attn_cache_tc_kernel(CacheArgs c, CacheAttnArgs a, int dg) {
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
  __shared__ float qfac[F::Q8 ? kBM : 1];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long mine, before;
  const long long len = Ln::template length<kTcThreads>(c, a, line, &mine, &before);
  const long long x0 = cut(len, gridDim.x, blockIdx.x), x1 = cut(len, gridDim.x, blockIdx.x + 1);
  if (x0 >= x1) return;
  typename Ln::Cursor u;
  Ln::template find<kTcThreads>(c, a, line, x0, mine, before, u);

  uint8_t* const base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sQ = smem_u32(base);
  auto sK = [&](int st) { return sQ + (F::QT + st) * F::TILE; };
  auto sV = [&](int st) { return sQ + (F::QT + KST + st) * F::TILE; };
  const uint32_t sStage = sQ + (F::QT + KST + VST) * F::TILE;
  const uint32_t sScale = sStage + F::SR * F::SSLOT;

  WaitCtl ctl{c.err, a.timeout_ns, &abort_flag};
  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(&bar_q, 4);
    mbar_init(&bar_qfree, 8);
    for (int s = 0; s < KST; ++s) {
      mbar_init(&bar_k[s], 4);
      mbar_init(&bar_kempty[s], 1);
    }
    for (int s = 0; s < VST; ++s) {
      mbar_init(&bar_v[s], 4);
      mbar_init(&bar_vempty[s], 1);
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
  if (warp == 12) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint32_t col_s[2] = {0u, 128u};
  const uint32_t col_o[2] = {256u, 256u + DP};

  // Pieces of this block: nt tiles from tile u.t of unit u.  `two`: two row
  // tiles that share the keys, else one row tile whose keys the groups share.
  auto piece_tiles = [&](const typename Ln::Cursor& p, long long x) {
    return static_cast<int>(min(static_cast<long long>(p.ntiles - p.t), x1 - x));
  };
  auto piece_two = [&](const typename Ln::Cursor& p) { return !F::Q8 && p.s.q * a.G - p.rt * F::ROWS > kBM; };

  if (warp >= 8 && warp < 12) {
    // ------------------------------------------------------------- copies
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTcRegsCopy));
    const int pw = warp - 8, tid = threadIdx.x - 256;
    // row of the cache that holds this lane's key of tile t (-1: none)
    auto look_up = [&](const typename Ln::Cursor& p, int t) -> int {
      const int n = t * kBN + pw * 32 + lane;
      if (n >= p.s.kv) return -1;
      int r;
      const int id = cache_page_id(c, p.b, n, &r);
      return cache_row(c, p.h, id, r);
    };
    // query row i of tile w as an offset into q; false: no such row
    auto q_row = [&](const typename Ln::Cursor& p, int w, int i, long long* off) -> bool {
      const int rr = p.rt * F::ROWS + w * kBM + i;
      if (rr >= p.s.q * a.G) return false;
      const int t = static_cast<int>(a.g_div.div(rr));
      *off = p.b * a.qs[0] + static_cast<long long>(p.h * a.G + (rr - t * a.G)) * a.qs[1] + t * a.qs[2];
      return true;
    };

    if constexpr (!F::Q8) {
      constexpr int CH = DP / 8;  // 16-byte chunks per row
      const int dch = dg / 8;
      // Copies in flight, oldest first: the barrier to signal and, for a
      // tile with new tokens' values, the tile to look through.  At most
      // three wait behind the one being issued.
      uint64_t* fb0 = nullptr;
      uint64_t* fb1 = nullptr;
      uint64_t* fb2 = nullptr;
      uint32_t fs0 = 0, fs1 = 0, fs2 = 0;
      int fp0 = 0, fp1 = 0, fp2 = 0;
      auto signal = [&](uint64_t* bar, uint32_t scan, int piece) {
        if (scan) {
          constexpr uint32_t EXP = BF ? 0x7f80u : 0x7c00u;
#pragma unroll 4
          for (int i = 0; i < CH; ++i) {  // the chunks this thread has copied
            const int idx = i * 32 + lane;
            const uint32_t at = tile_at(scan, pw * 32 + idx / CH, idx % CH);
            const uint4 v = lds_u4(at);
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
            bool hit = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if ((w[k] & EXP) == EXP) hit = true, w[k] &= 0xffff0000u;
              if (((w[k] >> 16) & EXP) == EXP) hit = true, w[k] &= 0x0000ffffu;
            }
            if (hit) {
              sts_v4(at, w[0], w[1], w[2], w[3]);
              odd[piece & 3] = piece + 1;
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
      };
      auto drain = [&]() {
        cp_async_wait<0>();
        if (fb0) signal(fb0, fs0, fp0);
        if (fb1) signal(fb1, fs1, fp1);
        if (fb2) signal(fb2, fs2, fp2);
        fb0 = fb1 = fb2 = nullptr;
      };
      auto push = [&](uint64_t* bar, uint32_t scan, int piece) {
        cp_async_commit();
        if (fb2) {
          cp_async_wait<3>();
          signal(fb0, fs0, fp0);
          fb0 = fb1, fs0 = fs1, fp0 = fp1;
          fb1 = fb2, fs1 = fs2, fp1 = fp2;
          fb2 = bar, fs2 = scan, fp2 = piece;
        } else if (fb1) {
          fb2 = bar, fs2 = scan, fp2 = piece;
        } else if (fb0) {
          fb1 = bar, fs1 = scan, fp1 = piece;
        } else {
          fb0 = bar, fs0 = scan, fp0 = piece;
        }
      };
      // A wait that would block signals everything in flight first: what it
      // waits for may depend on it.
      auto acquire = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
        drain();
        return warp_wait(bar, parity, ctl, kErrTimeoutMma);
      };
      auto copy = [&](const void* src, uint32_t tile, int rid) {
        const uint8_t* p = static_cast<const uint8_t*>(src);
#pragma unroll 4
        for (int i = 0; i < CH; ++i) {
          const int idx = i * 32 + lane, r = idx / CH, j = idx % CH;
          const int row = __shfl_sync(0xffffffffu, rid, r);
          const bool real = row >= 0 && j < dch;
          const size_t off = real ? static_cast<size_t>(row) * (dg * 2) + j * 16 : 0;
          cp_async16(tile_at(tile, pw * 32 + r, j), p + off, real);
        }
      };
      int kt = 0;  // tiles so far
      bool ok = true;
      long long x = x0;
      for (int piece = 0; ok && x < x1; ++piece) {
        const int nt = piece_tiles(u, x);
        const int past = u.s.kv - u.s.q;
        int rid = look_up(u, u.t);
        for (int i = 0; i < nt; ++i, ++kt) {
          const int next = i + 1 < nt ? look_up(u, u.t + i + 1) : -1;
          const int ks = kt % KST, vs = kt % VST;
          if (kt >= KST && !(ok = acquire(&bar_kempty[ks], (kt / KST - 1) & 1))) break;
          copy(c.k, sK(ks), rid);
          push(&bar_k[ks], 0, piece);
          if (kt >= VST && !(ok = acquire(&bar_vempty[vs], (kt / VST - 1) & 1))) break;
          copy(c.v, sV(vs), rid);
          push(&bar_v[vs], (u.t + i + 1) * kBN > past ? sV(vs) : 0u, piece);
          rid = next;
          if (i == 0) {  // the piece's queries, behind its first tile
            if (piece > 0 && !(ok = acquire(&bar_qfree, (piece - 1) & 1))) break;
            const int ntile = piece_two(u) ? 2 : 1;
            for (int w = 0; w < ntile; ++w) {
              long long off = 0;
              const bool has = q_row(u, w, pw * 32 + lane, &off);
#pragma unroll 4
              for (int k = 0; k < CH; ++k) {
                const int idx = k * 32 + lane, r = idx / CH, j = idx % CH;
                const long long o = __shfl_sync(0xffffffffu, off, r);
                const bool real = __shfl_sync(0xffffffffu, has, r) && j < dch;
                cp_async16(tile_at(sQ + w * F::TILE, pw * 32 + r, j),
                           static_cast<const T*>(a.q) + (real ? o + j * 8 : 0), real);
              }
            }
            push(&bar_q, 0, piece);
          }
        }
        x += nt;
        if (x < x1) Ln::next_unit(c, a, u);
      }
      drain();
    } else {
      constexpr int CH = DP / 16;  // 16-byte chunks per row of codes
      const int dch = dg / 16;
      // copy side: op n is K (even) or V (odd) of a tile, SR - 1 ahead of the
      // conversions
      typename Ln::Cursor q = u;
      long long xq = x0;
      int nq = 0, rid = -1;
      auto copy_next = [&]() {
        if (xq < x1) {
          const uint32_t st = sStage + (nq % F::SR) * F::SSLOT;
          const bool is_k = (nq & 1) == 0;
          if (is_k) {
            rid = look_up(q, q.t);
            const size_t off = static_cast<size_t>(rid < 0 ? 0 : rid);
            cp_async4(st + F::OPB + tid * 8, c.ks + off, rid >= 0);
            cp_async4(st + F::OPB + tid * 8 + 4, c.vs + off, rid >= 0);
          }
          const uint8_t* p = static_cast<const uint8_t*>(is_k ? c.k : c.v);
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            const int idx = i * 32 + lane, r = idx / CH, j = idx % CH;
            const int row = __shfl_sync(0xffffffffu, rid, r);
            const bool real = row >= 0 && j < dch;
            const size_t off = real ? static_cast<size_t>(row) * dg + j * 16 : 0;
            cp_async16(st + (i * 128 + tid) * 16, p + off, real);
          }
          ++nq;
          if (!is_k && ++xq < x1) Ln::next_tile(c, a, q);
        }
        cp_async_commit();
      };
      auto convert = [&](uint32_t st, uint32_t tile) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int idx = i * 32 + lane, r = idx / CH, j = idx % CH;
          const uint4 v = lds_u4(st + (i * 128 + tid) * 16);
          uint32_t h[8];
          code4_to_f16<CT>(v.x, h[0], h[1]);
          code4_to_f16<CT>(v.y, h[2], h[3]);
          code4_to_f16<CT>(v.z, h[4], h[5]);
          code4_to_f16<CT>(v.w, h[6], h[7]);
          // the two halves in an order that spreads a quarter warp over the banks
          const bool swap = DP == 128 && (j & 4);
          const uint32_t a0 = tile_at(tile, pw * 32 + r, 2 * j), a1 = tile_at(tile, pw * 32 + r, 2 * j + 1);
          if (swap) {
            sts_v4(a1, h[4], h[5], h[6], h[7]);
            sts_v4(a0, h[0], h[1], h[2], h[3]);
          } else {
            sts_v4(a0, h[0], h[1], h[2], h[3]);
            sts_v4(a1, h[4], h[5], h[6], h[7]);
          }
        }
      };
      auto signal = [&](uint64_t* bar) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
      };
#pragma unroll 1
      for (int i = 0; i < F::SR - 1; ++i) copy_next();
      int kt = 0;
      bool ok = true;
      long long x = x0;
      for (int piece = 0; ok && x < x1; ++piece) {
        const int nt = piece_tiles(u, x);
        for (int i = 0; i < nt; ++i, ++kt) {
          const int ks = kt % KST, vs = kt % VST;
          copy_next();
          cp_async_wait<F::SR - 1>();
          if (kt >= KST && !(ok = warp_wait(&bar_kempty[ks], (kt / KST - 1) & 1, ctl, kErrTimeoutMma))) break;
          uint32_t st = sStage + (2 * kt % F::SR) * F::SSLOT;
          convert(st, sK(ks));
          {
            float ksc, vsc;
            asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ksc), "=f"(vsc) : "r"(st + F::OPB + tid * 8) : "memory");
            // no scale (a row past the end or of a missing page): a value of zero
            if (vsc == 0.f) vsc = kMinScale;
            const uint32_t sc = sScale + (kt % F::SCS) * F::SCB + tid * 4;
            sts_f32(sc, ksc);
            sts_f32(sc + 512, lg2(vsc));
            // a NaN row's scores are NaN; its 1 / scale must not reach the sums of rows that do not see it
            sts_f32(sc + 1024, vsc == vsc ? 1.f / vsc : 0.f);
          }
          signal(&bar_k[ks]);
          copy_next();
          cp_async_wait<F::SR - 1>();
          if (kt >= VST && !(ok = warp_wait(&bar_vempty[vs], (kt / VST - 1) & 1, ctl, kErrTimeoutMma))) break;
          st = sStage + ((2 * kt + 1) % F::SR) * F::SSLOT;
          convert(st, sV(vs));
          signal(&bar_v[vs]);
          if (i == 0) {  // the piece's queries, a row per thread, in fp16
            if (piece > 0 && !(ok = warp_wait(&bar_qfree, (piece - 1) & 1, ctl, kErrTimeoutMma))) break;
            long long off = 0;
            const bool has = q_row(u, 0, tid, &off);
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + off);
            uint32_t top = 0;
            if constexpr (BF) {
#pragma unroll 4
              for (int j = 0; j < DP / 8; ++j) {
                const uint4 v = has && j < dg / 8 ? __ldg(p + j) : make_uint4(0u, 0u, 0u, 0u);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) top = max(top, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
              }
            }
            // bf16 rows: the largest magnitude to [1, 2) by a power of two
            int ex = static_cast<int>(top >> 7);
            ex = ex < 1 ? 1 : (ex > 253 ? 253 : ex);
            const float up = __uint_as_float(static_cast<uint32_t>(254 - ex) << 23);
            qfac[tid] = BF ? __uint_as_float(static_cast<uint32_t>(ex) << 23) : 1.f;
#pragma unroll 4
            for (int j = 0; j < DP / 8; ++j) {
              const uint4 v = has && j < dg / 8 ? __ldg(p + j) : make_uint4(0u, 0u, 0u, 0u);
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
        }
        x += nt;
        if (x < x1) Ln::next_unit(c, a, u);
      }
      cp_async_wait<0>();
    }
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTcRegsMma));
    if (warp == 12) {
      // ------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_qk = idesc_f16(kBM, kBN, MBF, false, false);
      constexpr uint32_t idesc_pv = idesc_f16(kBM, DP, MBF, false, true);
      int kt0 = 0;                  // tiles before this piece
      int np0 = 0, np1 = 0;         // products with V so far, per group
      bool ok = true;
      long long x = x0;
      for (int piece = 0; ok && x < x1; ++piece) {
        const int nt = piece_tiles(u, x);
        const bool two = piece_two(u);
        // item i: group i & 1 with its (i >> 1)-th tile
        const int ni = two ? 2 * nt : nt;
        auto issue_s = [&](int i) -> bool {
          const int kt = kt0 + (two ? i >> 1 : i), st = kt % KST, w = i & 1;
          if ((!two || w == 0) && !warp_wait(&bar_k[st], (kt / KST) & 1, ctl, kErrTimeoutTma)) return false;
          tc_fence_after();
          mma_qk<DP>(tmem + col_s[w], sQ + (two ? w * F::TILE : 0), sK(st), idesc_qk, false);
          commit_el(&bar_s[w]);
          if (!two || w == 1) commit_el(&bar_kempty[st]);
          return true;
        };
        ok = warp_wait(&bar_q, piece & 1, ctl, kErrTimeoutTma);
        if (ok) ok = issue_s(0);
        if (ok && ni > 1) ok = issue_s(1);
        for (int i = 0; ok && i < ni; ++i) {
          const int kt = kt0 + (two ? i >> 1 : i), st = kt % VST, w = i & 1;
          if ((!two || w == 0) && !(ok = warp_wait(&bar_v[st], (kt / VST) & 1, ctl, kErrTimeoutTma))) break;
          if (!(ok = warp_wait(&bar_p[w], (w ? np1 : np0) & 1, ctl, kErrTimeoutSoftmax))) break;
          if (w) ++np1;
          else ++np0;
          tc_fence_after();
          mma_pv<DP>(tmem + col_o[w], tmem + col_s[w], sV(st), idesc_pv, i > 1);
          commit_el(&bar_o[w]);
          if (!two || w == 1) commit_el(&bar_vempty[st]);
          if (i + 2 < ni) ok = issue_s(i + 2);
        }
        if (ok) commit_el(&bar_ofinal);
        kt0 += nt;
        x += nt;
        if (x < x1) Ln::next_unit(c, a, u);
      }
    }
  } else {
    // ---------------------------------- softmax, correction, epilogue (group w)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTcRegsSoftmax));
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
      float m_ref = -INFINITY, l = 0.f;
      for (int t = 0; t < n; ++t, ++ns) {
        if (!(ok = warp_wait(&bar_s[w], ns & 1, ctl, kErrTimeoutMma))) break;
        tc_fence_after();
        const int ti = two ? t : 2 * t + w;       // tile of the piece
        const int k0 = (u.t + ti) * kBN;
        const uint32_t sc = sScale + ((kt0 + ti) % F::SCS) * F::SCB;
        uint32_t s[128];
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld_x32(s_addr + 32 * k, TA_CHUNK(s, k));
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld_wait(TA_CHUNK(s, k));
        float y[128];
#pragma unroll
        for (int j = 0; j < 128; ++j) y[j] = __uint_as_float(s[j]);
        if constexpr (F::Q8) {
          const float f = a.scale_log2 * qfac[r];
          const float2 f2 = make_float2(f, f);
#pragma unroll
          for (int j = 0; j < 128; j += 4) {
            const float4 kx = lds_f4(sc + j * 4), vx = lds_f4(sc + 512 + j * 4);
            const float2 p = ffma2(make_float2(y[j], y[j + 1]), fmul2(f2, make_float2(kx.x, kx.y)), make_float2(vx.x, vx.y));
            const float2 q = ffma2(make_float2(y[j + 2], y[j + 3]), fmul2(f2, make_float2(kx.z, kx.w)), make_float2(vx.z, vx.w));
            y[j] = p.x, y[j + 1] = p.y, y[j + 2] = q.x, y[j + 3] = q.y;
          }
        }
        if (k0 + kBN > past) {  // keys behind the end, and new tokens
          if (!a.tree) {
            const int lim = min(u.s.kv - 1, past + tok) - k0;  // tok -1: rows that do not exist
#pragma unroll
            for (int j = 0; j < 128; ++j)
              if (j > lim) y[j] = -INFINITY;
          } else {
            // the warp's tokens one after the other: 32 keys' bytes a load
            uint32_t vis[4] = {0u, 0u, 0u, 0u};
            const int lo = __shfl_sync(0xffffffffu, tok, 0);
            int hi = tok;
#pragma unroll
            for (int k = 16; k > 0; k >>= 1) hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, k));
            for (int tt = lo; tt >= 0 && tt <= hi; ++tt) {
              const uint8_t* row = a.tree + u.b * a.tree_b + tt * a.tree_t;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int d = k0 + 32 * k + lane - past;
                const bool see = d < 0 || (d < u.s.q && __ldg(row + d) != 0);
                const uint32_t word = __ballot_sync(0xffffffffu, see);
                if (tok == tt) vis[k] = word;
              }
            }
#pragma unroll
            for (int j = 0; j < 128; ++j)
              if (!((vis[j >> 5] >> (j & 31)) & 1u)) y[j] = -INFINITY;
          }
        }
        float mx8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          mx8[k] = fmax3(y[k], y[8 + k], y[16 + k]);
#pragma unroll
          for (int j = 24; j < 120; j += 16) mx8[k] = fmax3(mx8[k], y[j + k], y[j + 8 + k]);
          mx8[k] = fmaxf(mx8[k], y[120 + k]);
        }
        const float mx = fmaxf(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(fmax3(mx8[3], mx8[4], mx8[5]), mx8[6], mx8[7]));
        const float m_new = fmaxf(m_ref, F::Q8 ? mx : mx * a.scale_log2);
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
        const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
        const float2 nm2 = make_float2(neg_m, neg_m);
        float2 rs2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t pk[8];
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const int j = 16 * k + 2 * e;
            float2 ya = make_float2(y[j], y[j + 1]), yb = make_float2(y[j + 2], y[j + 3]);
            if constexpr (F::Q8) {
              ya = fadd2(ya, nm2);
              yb = fadd2(yb, nm2);
            } else {
              ya = ffma2(ya, sc2, nm2);
              yb = ffma2(yb, sc2, nm2);
            }
            const float2 pa = make_float2(ex2(ya.x), ex2(ya.y)), pb = make_float2(ex2(yb.x), ex2(yb.y));
            if constexpr (F::Q8) {
              const float4 iv = lds_f4(sc + 1024 + j * 4);
              rs2[e & 2] = ffma2(pa, make_float2(iv.x, iv.y), rs2[e & 2]);
              rs2[(e & 2) + 1] = ffma2(pb, make_float2(iv.z, iv.w), rs2[(e & 2) + 1]);
            } else {
              rs2[e & 2] = fadd2(rs2[e & 2], pa);
              rs2[(e & 2) + 1] = fadd2(rs2[(e & 2) + 1], pb);
            }
            pk[e] = pack2<MBF>(pa.x, pa.y);
            pk[e + 1] = pack2<MBF>(pb.x, pb.y);
          }
          tmem_st_x8(s_addr + 8 * k, pk);
        }
        const float2 rsa = fadd2(fadd2(rs2[0], rs2[1]), fadd2(rs2[2], rs2[3]));
        l = l * alpha + (rsa.x + rsa.y);
        if (t > 0 && __any_sync(0xffffffffu, resc)) {
          if (!(ok = warp_wait(&bar_o[w], (ns - 1) & 1, ctl, kErrTimeoutMma))) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < DP / 32; ++k) {
            uint32_t ov[32];
            tmem_ld_x32(o_addr + 32 * k, ov);
            tmem_ld_wait(ov);
#pragma unroll
            for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * alpha);
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
      if (two) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_qfree);
      }
      // one row tile: group 1 hands its state over through Q's memory, in
      // rounds of as many columns as fit
      constexpr int NCH = DP / 4;                                  // float4 columns
      constexpr int XCH = F::XCH < NCH ? F::XCH : NCH, XR = NCH / XCH;
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
              sts_v4(sQ + ((k + j) * kBM + r) * 16, ov[4 * j], ov[4 * j + 1], ov[4 * j + 2], ov[4 * j + 3]);
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
            l = mm == -INFINITY ? l + l1 : l * f0 + l1 * f1;
            m_ref = mm;
          }
        }
        const float norm = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
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
              const float4 y = lds_f4(sQ + ((k + j) * kBM + r) * 16);
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
          a.lse[(static_cast<long long>(u.b) * a.Hq + hq) * c.T + tok] =
              l == 0.f ? -INFINITY : (m_ref == -INFINITY ? l : (m_ref + lg2(l)) * kLn2);
        }
        if constexpr (!F::Q8) {
          if (odd_values && tok >= 0)
            add_non_finite<T>(c, a, u.b, u.h, tok, past, u.t * kBN, min(u.s.kv, (u.t + nt) * kBN), dg,
                              whole ? out : nullptr, part + prow * 4, F::ROWS * 4);
        }
      }
      tc_fence_before();
      if (!two) {
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
  if (warp == 12) tmem_dealloc(tmem, 512);
}

// Joins the partial states of the units that block borders cut: block (i, y)
// looks at border i + 1 and, where it is the first inside its unit, joins rows
// 32 y .. 32 y + 31, a row per lane, every eighth group of four columns per warp.
template <typename T, int CT, int DP>
__global__ void __launch_bounds__(256) attn_cache_tc_join_kernel(CacheArgs c, CacheAttnArgs a, int dg, int nblocks) {
  using F = TcCfg<CT, DP>;
  using Ln = Line<F::ROWS, kBN>;
  constexpr bool BF = DT<T>::bf16;
  constexpr int NC = DP / 32;  // float4 columns per thread
  __shared__ typename Ln::Shared line;
  long long mine, before;
  const long long len = Ln::template length<256>(c, a, line, &mine, &before);
  const int i = blockIdx.x + 1;
  const long long x = cut(len, nblocks, i);
  if (x >= len) return;
  typename Ln::Cursor u;
  Ln::template find<256>(c, a, line, x, mine, before, u);
  const long long u0 = x - u.t, u1 = u0 + u.ntiles;
  if (u.t == 0 || cut(len, nblocks, i - 1) > u0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int prow = blockIdx.y * 32 + lane, rr = u.rt * F::ROWS + prow;
  const int rows = u.s.q * a.G;
  if (u.rt * F::ROWS + static_cast<int>(blockIdx.y) * 32 >= rows) return;
  const int b1 = block_of(len, nblocks, u1 - 1);
  auto state = [&](int b) -> const float* {
    const long long s = cut(len, nblocks, b);
    if (s == cut(len, nblocks, b + 1)) return nullptr;  // an empty piece
    return a.ws + (static_cast<size_t>(b) * 2 + (s < u0 ? 1 : 0)) * tc_part_floats<CT, DP>();
  };
  float mm = -INFINITY;
  for (int b = i - 1; b <= b1; ++b) {
    const float* p = state(b);
    if (p) mm = fmaxf(mm, __ldcg(p + F::ROWS * DP + prow));
  }
  float ll = 0.f;
  float v[NC][4] = {};
#pragma unroll 2
  for (int b = i - 1; b <= b1; ++b) {
    const float* p = state(b);
    if (!p) continue;
    const float pm = __ldcg(p + F::ROWS * DP + prow), pl = __ldcg(p + F::ROWS * (DP + 1) + prow);
    const float f = pm == -INFINITY ? 0.f : ex2(pm - mm);
    ll += mm == -INFINITY ? pl : pl * f;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int ch = warp + 8 * k;
      if (ch * 4 < dg) {
        const float4 y = __ldcg(reinterpret_cast<const float4*>(p) + ch * F::ROWS + prow);
        v[k][0] = fmaf(y.x, f, v[k][0]);
        v[k][1] = fmaf(y.y, f, v[k][1]);
        v[k][2] = fmaf(y.z, f, v[k][2]);
        v[k][3] = fmaf(y.w, f, v[k][3]);
      }
    }
  }
  if (rr >= rows) return;
  const int t = static_cast<int>(a.g_div.div(rr)), hq = u.h * a.G + (rr - t * a.G);
  const float norm = ll == 0.f ? 0.f : 1.f / ll;
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
  if (warp == 0)
    a.lse[(static_cast<long long>(u.b) * a.Hq + hq) * c.T + t] =
        ll == 0.f ? -INFINITY : (mm == -INFINITY ? ll : (mm + lg2(ll)) * kLn2);
}

template <typename T, int CT, int DP>
cudaError_t run_tc(int dg, const CacheArgs& c, const CacheAttnArgs& a, cudaStream_t s) {
  static std::atomic<bool> done[kMaxDevices];
  auto* kern = attn_cache_tc_kernel<T, CT, DP>;
  constexpr int smem = TcCfg<CT, DP>::SMEM;
  cudaError_t e = smem_attr_once(kern, smem, done);
  if (e != cudaSuccess) return e;
  prof_begin("attn_cache_tc", s);
  kern<<<kTcBlocks, kTcThreads, smem, s>>>(c, a, dg);
  prof_end(s);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  prof_begin("attn_cache_tc_join", s);
  attn_cache_tc_join_kernel<T, CT, DP>
      <<<dim3(kTcBlocks - 1, TcCfg<CT, DP>::ROWS / 32), 256, 0, s>>>(c, a, dg, kTcBlocks);
  prof_end(s);
  return cudaGetLastError();
}
template <int CT>
size_t tc_ws_bytes(int D) {
  const int f = D <= 64 ? tc_part_floats<CT, 64>() : tc_part_floats<CT, 128>();
  return static_cast<size_t>(kTcBlocks) * 2 * f * sizeof(float);
}

}  // namespace
}  // namespace ta
