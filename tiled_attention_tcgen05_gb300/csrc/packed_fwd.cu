// Forward attention of packed sequences with shared key heads (sm_103a).
//
//   O_i = sum_j p_ij V_j / sum_j p_ij,  p_ij = exp(c q_i . k_j - m_i),  L_i = m_i + ln sum_j p_ij
//
// over the keys j of the query's own sequence, causal ones up to i + n_k - n_q.
//
// One CTA owns two 128-row query tiles of one key head (packed.cuh: TB tokens x G
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
// They work on a V tile between its arrival and its product, beside the tiles
// before it, and only on the last tiles of a CTA (up to three).
#include <cstdio>

#include "launch.h"
#include "packed.cuh"

namespace ta {

namespace {

constexpr int kThreads = 384;
constexpr int kProducer = 8, kMma = 9, kCare = 10;  // warps; kCare and the one behind it
// Key tiles that some row of a CTA sees in part, at most: its tokens' last keys
// lie within 256 of each other.  Each has a pair of barriers of its own, used
// once, so that the two warps need not follow the V ring's phases.
constexpr int kPart = 3;

template <int D>
struct PfCfg {
  static constexpr int TILE = (D / 64) * kBM * 128;
  static constexpr int KST = D == 128 ? 3 : 4;  // K ring depth
  static constexpr int VST = D == 128 ? 2 : 4;  // V ring depth
  static constexpr int SMEM = (2 + KST + VST) * TILE + 1024;
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

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    packed_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                      const PackedArgs args) {
  using C = PfCfg<D>;
  constexpr bool BF = DT<T>::bf16;
  constexpr int KST = C::KST, VST = C::VST;

  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_q;
  __shared__ __align__(8) uint64_t bar_k[KST], bar_kempty[KST], bar_v[VST], bar_vempty[VST];
  __shared__ __align__(8) uint64_t bar_part[kPart], bar_care[kPart];
  __shared__ __align__(8) uint64_t bar_s[2], bar_p[2], bar_o[2], bar_ofinal;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag, odd_values;  // odd_values: a non-finite value was taken out of a tile

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  PackedUnit unit;
  int head;  // key head
  if (!packed_unit(args, kPackedFwd, &unit, &head)) return;
  const int causal = unit.pad[0];
  const int G = args.shape.G, TB = args.shape.TB;
  // tile w: tokens left, last key its first token sees, key tiles
  int left[2], off[2], n_t[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    left[w] = unit.left - w * TB;
    off[w] = unit.off + w * TB;
    n_t[w] = packed_key_tiles(min(left[w], TB), off[w], unit.n, causal);
  }
  const int nt = max(n_t[0], n_t[1]);
  // key tiles from here on are seen in part by some row, or end behind the keys
  int t_part = unit.n / kBN;
  if (causal) t_part = min(t_part, unit.off < 0 ? 0 : (unit.off + 1) / kBN);

  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = base;
  auto sK = [&](int st) { return base + (2 + st) * C::TILE; };
  auto sV = [&](int st) { return base + (2 + KST + st) * C::TILE; };

  WaitCtl ctl{args.err, args.timeout_ns, &abort_flag};
  if (threadIdx.x == 0) {
    abort_flag = 0;
    odd_values = 0;
    mbar_init(&bar_q, 1);
    for (int s = 0; s < KST; ++s) {
      mbar_init(&bar_k[s], 1);
      mbar_init(&bar_kempty[s], 1);
    }
    for (int s = 0; s < VST; ++s) {
      mbar_init(&bar_v[s], 1);
      mbar_init(&bar_vempty[s], 1);
    }
    for (int i = 0; i < kPart; ++i) {
      mbar_init(&bar_part[i], 1);
      mbar_init(&bar_care[i], 2);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&bar_s[w], 1);
      mbar_init(&bar_p[w], 4);
      mbar_init(&bar_o[w], 1);
    }
    mbar_init(&bar_ofinal, 1);
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

  if (warp == kProducer) {
    // ------------------------- TMA producer: lane 0 Q and the K ring, lane 1 the V ring
    if (lane < 2 && nt > 0) {
      const bool is_k = (lane == 0);
      const int depth = is_k ? KST : VST;
      uint64_t* full = is_k ? bar_k : bar_v;
      uint64_t* empty = is_k ? bar_kempty : bar_vempty;
      const CUtensorMap* map = is_k ? &tm_k : &tm_v;
      if (is_k) {
        const int tiles = left[1] > 0 ? 2 : 1;
        mbar_expect_tx(&bar_q, tiles * (D / 64) * TB * G * 128);  // rows past a tile's TB x G are not loaded
        for (int w = 0; w < tiles; ++w) load_rows<D>(sQ + w * C::TILE, &tm_q, &bar_q, head * G, unit.row + w * TB);
      }
      int issued = 0;
      for (int t = 0; t < nt; ++t) {
        const int st = t % depth;
        if (t >= depth && !mbar_wait(&empty[st], ((t / depth) - 1) & 1, ctl, kErrTimeoutMma)) break;
        uint64_t* bar = !is_k && t >= t_part ? &bar_part[t - t_part] : &full[st];
        mbar_expect_tx(bar, C::TILE);
        load_rows<D>(is_k ? sK(st) : sV(st), map, bar, unit.krow + t * kBN, head);
        issued = t + 1;
      }
      int zero = 0;
      WaitCtl drain{args.err, args.timeout_ns, reinterpret_cast<volatile int*>(&zero)};
      if (is_k) mbar_wait(&bar_q, 0, drain, kErrTimeoutTma);
      for (int t = issued - depth > 0 ? issued - depth : 0; t < issued; ++t) {
        if (!is_k && t >= t_part) mbar_wait(&bar_part[t - t_part], 0, drain, kErrTimeoutTma);
        else mbar_wait(&full[t % depth], (t / depth) & 1, drain, kErrTimeoutTma);
      }
    }
  } else if (warp == kMma) {
    // --------------------------------------------------------- MMA issuer
    if (nt > 0) {
      constexpr uint32_t idesc_qk = idesc_f16(kBM, kBN, BF, false, false);
      constexpr uint32_t idesc_pv = idesc_f16(kBM, D, BF, false, true);
      const uint32_t aQ[2] = {smem_u32(sQ), smem_u32(sQ) + C::TILE};
      bool ok = warp_wait(&bar_q, 0, ctl, kErrTimeoutTma) && warp_wait(&bar_k[0], 0, ctl, kErrTimeoutTma);
      if (ok) {
        tc_fence_after();
        for (int w = 0; w < 2; ++w)
          if (n_t[w] > 0) {
            mma_abT<D>(tmem + col_s[w], aQ[w], smem_u32(sK(0)), idesc_qk);
            commit_el(&bar_s[w]);
          }
        commit_el(&bar_kempty[0]);
      }
      for (int t = 0; ok && t < nt; ++t) {
        const int sv = t % VST;
        const int sk1 = (t + 1) % KST;
        if (!(ok = t < t_part ? warp_wait(&bar_v[sv], (t / VST) & 1, ctl, kErrTimeoutTma)
                              : warp_wait(&bar_care[t - t_part], 0, ctl, kErrTimeoutOther)))
          break;
        const bool next = t + 1 < nt;
        if (next && !(ok = warp_wait(&bar_k[sk1], ((t + 1) / KST) & 1, ctl, kErrTimeoutTma))) break;
        for (int w = 0; w < 2; ++w) {
          if (t < n_t[w]) {
            if (!(ok = warp_wait(&bar_p[w], t & 1, ctl, kErrTimeoutSoftmax))) break;
            tc_fence_after();
            mma_pv<D>(tmem + col_o[w], tmem + col_s[w], smem_u32(sV(sv)), idesc_pv, t > 0);
            commit_el(&bar_o[w]);
          }
          if (next && t + 1 < n_t[w]) {
            mma_abT<D>(tmem + col_s[w], aQ[w], smem_u32(sK(sk1)), idesc_qk);
            commit_el(&bar_s[w]);
          }
        }
        if (!ok) break;
        commit_el(&bar_vempty[sv]);
        if (next) commit_el(&bar_kempty[sk1]);
      }
      if (ok) commit_el(&bar_ofinal);
    }
  } else if (warp >= kCare) {
    // ------------------------------- value tiles that some row sees in part
    const int r0 = (warp - kCare) * 64;  // each warp's half of the tile's rows
    for (int t = t_part; t < nt; ++t) {
      const int sv = t % VST;
      if (!warp_wait(&bar_part[t - t_part], 0, ctl, kErrTimeoutTma)) break;
      const int valid = min(kBN, unit.n - t * kBN);  // rows of the tile that are keys
      bool odd = false;
#pragma unroll
      for (int kb = 0; kb < D / 64; ++kb) {
        uint4* rows = reinterpret_cast<uint4*>(sV(sv) + kb * (kBM * 128) + r0 * 128);
        const int keys = min(max(valid - r0, 0), 64) * 8;  // 16-byte pieces
        for (int i = keys + lane; i < 64 * 8; i += 32) rows[i] = make_uint4(0u, 0u, 0u, 0u);
        if (causal) {
#pragma unroll 4
          for (int i = lane; i < keys; i += 32) {
            uint4 x = rows[i];
            const uint4 m = make_uint4(non_finite2<BF>(x.x), non_finite2<BF>(x.y), non_finite2<BF>(x.z),
                                       non_finite2<BF>(x.w));
            if (m.x | m.y | m.z | m.w) {
              odd = true;
              rows[i] = make_uint4(x.x & ~m.x, x.y & ~m.y, x.z & ~m.z, x.w & ~m.w);
            }
          }
        }
      }
      if (odd) odd_values = 1;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_care[t - t_part]);
    }
  } else {
    // ------------------------------- softmax / correction / epilogue (tile w)
    const int w = warp >> 2;
    const int r = threadIdx.x & 127;
    const int tok = static_cast<int>(args.g_div.div(r)), g = r - tok * G;  // of the tile
    const int n = n_t[w];
    const int sees = causal ? min(unit.n - 1, off[w] + tok) : unit.n - 1;  // last key of this row
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    float m_ref = -INFINITY, l = 0.f;
    bool ok = true;
    for (int t = 0; t < n; ++t) {
      if (!(ok = warp_wait(&bar_s[w], t & 1, ctl, kErrTimeoutMma))) break;
      tc_fence_after();
      const int k0 = t * kBN;
      uint32_t s[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld_x32(lane_addr + col_s[w] + 32 * c, TB_CHUNK(s, c));
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld_wait(TB_CHUNK(s, c));
      float x[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) x[j] = __uint_as_float(s[j]);
      if (t >= t_part) {
        const int lim = sees - k0;
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
        tmem_st_x8(lane_addr + col_s[w] + 8 * c, pk);
      }
      const float2 rsa = fadd2(fadd2(rs2[0], rs2[1]), fadd2(rs2[2], rs2[3]));
      l = l * alpha + (rsa.x + rsa.y);
      if (t > 0 && __any_sync(0xffffffffu, resc)) {
        if (!(ok = warp_wait(&bar_o[w], (t - 1) & 1, ctl, kErrTimeoutMma))) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          tmem_ld_x32(lane_addr + col_o[w] + 32 * c, ov);
          tmem_ld_wait(ov);
#pragma unroll
          for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * alpha);
          tmem_st_x32(lane_addr + col_o[w] + 32 * c, ov);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_p[w]);
    }
    // ------------------------------------------------------------ epilogue
    if (nt > 0) ok = warp_wait(&bar_ofinal, 0, ctl, kErrTimeoutMma) && __all_sync(0xffffffffu, ok);
    tc_fence_after();
    const bool live = ok && n > 0;
    const float inv_l = (live && l > 0.f) ? 1.f / l : (l == l ? 0.f : l);
    const bool stored = tok < min(left[w], TB);  // TB x G rows at most, and tokens of the sequence
    const size_t qrow = static_cast<size_t>(unit.row) + w * TB + tok;
    if (stored)
      args.lse[qrow * args.shape.Hq + head * G + g] =
          (live && l != 0.f) ? (m_ref + lg2(l)) * kLn2 : -INFINITY;
    // non-finite values that were taken out: of this row's keys in those tiles, added to O at the end
    bool odd = false;
    if (live && causal && t_part < nt) {
      for (int t = t_part; ok && t < nt; ++t)  // (done long since: the products waited for them)
        ok = warp_wait(&bar_care[t - t_part], 0, ctl, kErrTimeoutOther);
      odd = *reinterpret_cast<volatile int*>(&odd_values) != 0;
    }
    const uint32_t stage = smem_u32(sQ) + static_cast<uint32_t>(w * C::TILE);
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t ov[32];
      if (live) {
        tmem_ld_x32(lane_addr + col_o[w] + 32 * c, ov);
        tmem_ld_wait(ov);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) ov[j] = 0u;
      }
      float scale = inv_l;
      if (odd) {
        if (stored && l > 0.f) {
          const int ng = chunk_groups(args.dg, 32 * c);
#pragma unroll
          for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * inv_l);
          for (int k = t_part * kBN; k <= min(sees, n * kBN - 1); ++k) {
            const T* vrow = static_cast<const T*>(args.v) + (static_cast<long long>(unit.krow) + k) * args.vt +
                            head * args.vh + 32 * c;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (q >= ng) break;
              const uint4 x = __ldg(reinterpret_cast<const uint4*>(vrow) + q);
              const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
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
      }
      stage_row_chunk_sw128<BF>(stage, r, c, ov, scale);
    }
    fence_proxy_async_smem();
    named_bar_sync(1 + w, 4 * 32);  // the tile's four warps have staged their rows
    if (left[w] >= TB) {  // whole: a box
      if ((warp & 3) == 0 && lane == 0) {
#pragma unroll
        for (int kb = 0; kb < D / 64; ++kb)
          tma_store_3d(&tm_o, sQ + w * C::TILE + kb * (kBM * 128), kb * 64, head * G, unit.row + w * TB);
        tma_store_commit_and_wait_read();
      }
    } else if (left[w] > 0) {  // the rows behind it are another sequence's
      T* o = static_cast<T*>(args.o);
      const int rows = left[w] * G;
      copy_tile_rows(sQ + w * C::TILE, args.dg, r, 128, [&](int i) -> void* {
        if (i >= rows) return nullptr;
        const int k = static_cast<int>(args.g_div.div(i));
        return o + (static_cast<long long>(unit.row) + w * TB + k) * args.o_t + (head * G + i - k * G) * args.o_h;
      });
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
