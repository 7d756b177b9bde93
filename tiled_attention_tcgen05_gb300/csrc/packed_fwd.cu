// Forward attention of packed sequences with shared key heads (sm_103a).
//
//   O_i = sum_j p_ij V_j / sum_j p_ij,  p_ij = exp(c q_i . k_j - m_i),  L_i = m_i + ln sum_j p_ij
//
// over the keys j of the query's own sequence, causal ones up to i + n_k - n_q.
//
// A CTA works on two 128-row query tiles of one key head (packed.cuh: TB tokens x G
// heads each) that share every K/V tile: warps 0-3 and 4-7 run their softmax, one
// thread a row (and each group's first thread stores its O), warp 8
// feeds the K and V rings and Q by TMA, warp 9 issues the MMAs, alternating between the
// tiles so that one's softmax runs beside the other's products, and warps 10 and 11
// look after the key tiles that some row sees only in part:
//   * the rows behind the sequence's keys belong to another sequence or to
//     nobody, and a weight of zero times an infinity there would be NaN:
//     they become zeros;
//   * so would an infinity or a NaN in the value of a key that only some rows
//     see: such elements become zeros for the product, and the rows that see them
//     get them back from memory at the end.
// Such tiles are the last ones of a unit, three at most; they come in through
// barriers of their own.  The rings run on from one unit to the next (UnitRing);
// warp 11 asks for the units.
//
// Bound, for long sequences, by the MMAs: three prompts of up to 16384 tokens, 32 / 8 heads of 128, bf16,
// take 2.06 ms, 1693 TFLOP/s, 0.90 of the measured peak, in short runs (in runs of seconds the power limit lowers
// the clock, and they take 2.23).  Short ones are bound by the way
// from one role to the next and by fetching code that runs once a unit: 64 prompts of up to 250 tokens, 32 / 4
// heads of 64, take 34 us, some 3.4 us a unit of one or two key tiles, of which its memory and products need 1.3.
// For them there is an instance whose short units (kFewTiles) go through one copy of each
// product and through loops over 32 columns; with the long units' straight-line code they took 40 us. The
// other way round the loops cost long units 13 % (products) and 8 % (scores).
// Measured and not taken: scores of the tile after next before a tile's product with V (long 2.44 ms), two
// more softmax groups (2.78 ms).
#include "launch.h"
#include "packed.cuh"

namespace ta {

namespace {

constexpr int kThreads = 384;
constexpr int kProducer = 8, kMma = 9, kCare = 10;  // warps; kCare and the one behind it
// registers: 384 x 168 at launch = 256 x 200 (softmax) + 128 x 104
// Key tiles of a short unit.  3 and 5 instead of 2 gain up to 5 % (400 tokens, 16 / 16 heads of 128) and lose up to
// 10 (400 tokens, 16 / 16 of 64); sequences of up to 256 take the same.
constexpr int kFewTiles = 2;
constexpr int kPart = 3;  // tiles that some row sees in part: its tokens' last keys lie within 256 of each other

template <int D>
struct PfCfg {
  static constexpr int TILE = (D / 64) * kBM * 128;
  static constexpr int KST = D == 128 ? 3 : 4;  // K ring depth
  static constexpr int VST = D == 128 ? 2 : 4;  // V ring depth
  static constexpr int QB = D == 128 ? 1 : 2;   // Q tiles of each group (their memory takes O on its way out)
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
// Bit 15 of a half is set where it is one: an exponent of ones carries into it.
template <bool BF>
__device__ __forceinline__ uint32_t non_finite_bits(uint32_t w) {
  constexpr uint32_t E = BF ? 0x7f807f80u : 0x7c007c00u, ONE = BF ? 0x00800080u : 0x04000400u;
  return (w & E) + ONE;
}

// What the roles need of a unit, made by the asking thread.
struct Pair {
  int row, krow, n, off;            // first token's row, first key's row, keys, last key the first token sees
  int left, n0, n1, head;           // tokens to the sequence's end, key tiles of the two tiles, key head
  int t_part, causal;               // from t_part on some row sees a tile in part, or it ends behind the keys
  __device__ __forceinline__ Pair(const UnitRing* r, int i) {
    const int4 a = ring_words(r, i, 0), b = ring_words(r, i, 1), c = ring_words(r, i, 2);
    row = a.x;
    krow = a.y;
    n = a.z;
    off = a.w;
    left = b.x;
    n0 = b.y;
    n1 = b.z;
    head = b.w;
    t_part = c.x;
    causal = c.y;
  }
  __device__ __forceinline__ int nt() const { return max(n0, n1); }
  __device__ __forceinline__ int n_t(int w) const { return w ? n1 : n0; }
};
__device__ __forceinline__ void make_pair(const PackedUnit& u, int TB, int4 (&words)[4]) {
  const int causal = u.pad[0];
  const int n0 = packed_key_tiles(min(u.left, TB), u.off, u.n, causal);
  const int n1 = packed_key_tiles(min(u.left - TB, TB), u.off + TB, u.n, causal);
  int t_part = u.n / kBN;
  if (causal) t_part = min(t_part, u.off < 0 ? 0 : (u.off + 1) / kBN);
  words[0] = make_int4(u.row, u.krow, u.n, u.off);
  words[1] = make_int4(u.left, n0, n1, u.pad[1]);
  words[2] = make_int4(t_part, causal, 0, 0);
}
// A ring's next slot and the parity of its phase.
template <int N>
struct RingAt {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void step() {
    if (++st == N) {
      st = 0;
      ph ^= 1u;
    }
  }
};

template <typename T, int D, bool SHORT>
__global__ void __launch_bounds__(kThreads, 1)
    packed_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                      const PackedArgs args) {
  using C = PfCfg<D>;
  constexpr bool BF = DT<T>::bf16;
  constexpr int KST = C::KST, VST = C::VST, QB = C::QB;

  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) UnitRing ring;
  __shared__ __align__(8) uint64_t bar_k[KST], bar_kempty[KST], bar_v[VST], bar_vempty[VST];
  __shared__ __align__(8) uint64_t bar_part[2][kPart], bar_care[2][kPart];  // [unit % 2]: such a tile is in, is seen to
  __shared__ __align__(8) uint64_t bar_q[2][QB], bar_s[2], bar_p[2], bar_o[2], bar_ofinal[2];  // [group]
  __shared__ __align__(8) uint64_t bar_qfree[2];  // [group] (QB == 2) its other Q buffer can be loaded
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ int care_odd[2][kPart][2];  // the tile held non-finite values that only some rows see (by caring warp)
  __shared__ int unit_odd[2];            // [group]: any of its last unit's did

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const PackedList list = packed_list(args, kPackedFwd);
  if (blockIdx.x >= list.items) return;
  const int G = args.shape.G, TB = args.shape.TB;

  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto sQ = [&](int w, int qb) { return base + (w * QB + qb) * C::TILE; };
  auto sK = [&](int st) { return base + (2 * QB + st) * C::TILE; };
  auto sV = [&](int st) { return base + (2 * QB + KST + st) * C::TILE; };

  const bool asks = threadIdx.x == (kCare + 1) * 32;
  if (asks) {
    make_pair(packed_item(args, list, blockIdx.x), TB, ring.unit[0]);
    ring.unit[0][3].w = 1;
  }
  WaitCtl ctl{args.err, args.timeout_ns, &abort_flag};
  if (threadIdx.x == 0) {
    abort_flag = 0;
    ring_init(&ring, 8 + 1 + 2 + 1);  // softmax warps, MMA, two producing lanes, warp 10
    for (int s = 0; s < KST; ++s) {
      mbar_init(&bar_k[s], 1);
      mbar_init(&bar_kempty[s], 1);
    }
    for (int s = 0; s < VST; ++s) {
      mbar_init(&bar_v[s], 1);
      mbar_init(&bar_vempty[s], 1);
    }
    for (int w = 0; w < 2; ++w) {
      for (int j = 0; j < kPart; ++j) {
        mbar_init(&bar_part[w][j], 1);
        mbar_init(&bar_care[w][j], 2);
      }
      for (int q = 0; q < QB; ++q) mbar_init(&bar_q[w][q], 1);
      mbar_init(&bar_s[w], 1);
      mbar_init(&bar_p[w], 4);
      mbar_init(&bar_o[w], 1);
      mbar_init(&bar_ofinal[w], 2);
      mbar_init(&bar_qfree[w], 1);
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
  constexpr uint32_t kColS1 = 128, kColO0 = 256, kColO1 = 256 + D;

  int zero = 0;  // (an exit waits for its own copies whatever the abort flag says)
  const WaitCtl drain{args.err, args.timeout_ns, reinterpret_cast<volatile int*>(&zero)};
  const uint32_t qbytes = (D / 64) * TB * G * 128;  // of a Q tile: rows past its TB x G are not loaded
  // (on the way out) waits for the Q tiles of group w that are still on their way
  auto drain_q = [&](int w, uint32_t n) {
    for (uint32_t a = n > QB ? n - QB : 0; a < n; ++a)
      mbar_wait(&bar_q[w][a % QB], (a / QB) & 1, drain, kErrTimeoutTma);
  };
  if (warp == kProducer) {
    // ------ TMA producer: lane 0 the K ring and, where it has two buffers, Q; lane 1 the V ring
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (lane < 2) {
      const bool is_k = lane == 0;
      const int depth = is_k ? KST : VST;
      uint64_t* full = is_k ? bar_k : bar_v;
      uint64_t* empty = is_k ? bar_kempty : bar_vempty;
      const CUtensorMap* map = is_k ? &tm_k : &tm_v;
      int e = 0;             // tiles so far
      uint32_t own = 0;      // V slots whose last tile came through bar_part
      uint32_t part_ph = 0;  // parities of bar_part's phases (those armed so far are odd in number)
      uint32_t qs[2] = {0, 0};  // (lane 0) Q tiles asked for, by group
      bool ok = true;
      for (int i = 0; ok && ring_take(&ring, i, ctl); ++i) {
        const Pair p(&ring, i);
        const int nt = p.nt();
        for (int t = 0; t < nt; ++t, ++e) {
          const int st = e % depth;
          if (e >= depth && !(ok = mbar_wait(&empty[st], ((e / depth) - 1) & 1, ctl, kErrTimeoutMma))) break;
          uint64_t* bar = &full[st];
          if (!is_k && t >= p.t_part) {
            const int j = t - p.t_part;
            mbar_arrive(bar);  // (the ring's own phase passes on)
            bar = &bar_part[i & 1][j];
            part_ph ^= 1u << ((i & 1) * kPart + j);
            own |= 1u << st;
          } else {
            own &= ~(1u << st);
          }
          mbar_expect_tx(bar, C::TILE);
          load_rows<D>(is_k ? sK(st) : sV(st), map, bar, p.krow + t * kBN, p.head);
          if (QB == 2 && is_k && t == 0) {  // (the first K tile waits for no group)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              if (!ok || p.n_t(w) == 0) continue;
              if (qs[w] > 0 && !(ok = mbar_wait(&bar_qfree[w], (qs[w] - 1) & 1, ctl, kErrTimeoutSoftmax))) continue;
              uint64_t* qbar = &bar_q[w][qs[w] % QB];
              mbar_expect_tx(qbar, qbytes);
              load_rows<D>(sQ(w, qs[w] % QB), &tm_q, qbar, p.head * G, p.row + w * TB);
              ++qs[w];
            }
            if (!ok) {
              ++e;
              break;
            }
          }
        }
        if (!ok) break;
        if (is_k) mbar_arrive(&ring.near);
        mbar_arrive(&ring.left[i & 1]);
      }
      if (QB == 2 && is_k) {
        drain_q(0, qs[0]);
        drain_q(1, qs[1]);
      }
      for (int t = e - depth > 0 ? e - depth : 0; t < e; ++t)
        if (!(own >> (t % depth) & 1u)) mbar_wait(&full[t % depth], (t / depth) & 1, drain, kErrTimeoutTma);
      if (!is_k)  // (a phase that was never armed: the parity of the one before it, which has passed)
        for (int j = 0; j < 2 * kPart; ++j)
          mbar_wait(&bar_part[j / kPart][j % kPart], (part_ph >> j & 1u) ^ 1u, drain, kErrTimeoutTma);
    }
  } else if (warp == kMma) {
    // --------------------------------------------------------- MMA issuer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    constexpr uint32_t idesc_qk = idesc_f16(kBM, kBN, BF, false, false);
    constexpr uint32_t idesc_pv = idesc_f16(kBM, D, BF, false, true);
    RingAt<KST> k;
    RingAt<VST> v;
    uint32_t qs0 = 0, qs1 = 0;  // Q tiles of the groups so far
    uint32_t np0 = 0, np1 = 0;  // parities of the groups' tiles
    uint32_t part_ph = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      if (!__all_sync(0xffffffffu, ring_take(&ring, i, ctl))) break;
      int n0, n1, t_part;
      {
        const Pair p(&ring, i);
        n0 = p.n0;
        n1 = p.n1;
        t_part = p.t_part;
      }
      const int nt = max(n0, n1);
      int odd = 0;
      if (SHORT && nt <= kFewTiles) {
        // one copy of each product, for both groups and a unit's first tile, too: a short unit's
        // time is that of fetching this code
#pragma unroll 1
        for (int t = -1; t < nt; ++t) {
          const bool next = t + 1 < nt;
          if (t >= 0) {
            if (t < t_part) {
              ok = warp_wait(&bar_v[v.st], v.ph, ctl, kErrTimeoutTma);
            } else {
              const int j = t - t_part, bit = (i & 1) * kPart + j;
              ok = warp_wait(&bar_care[i & 1][j], part_ph >> bit & 1u, ctl, kErrTimeoutOther);
              part_ph ^= 1u << bit;
              if (ok) odd |= care_odd[i & 1][j][0] | care_odd[i & 1][j][1];
            }
            if (!ok) break;
          }
          if (next && !(ok = warp_wait(&bar_k[k.st], k.ph, ctl, kErrTimeoutTma))) break;
#pragma unroll 1
          for (int w = 0; w < 2; ++w) {
            const int n = w ? n1 : n0;
            if (t >= n) continue;
            const bool more = t + 1 < n;
            const uint32_t cs = tmem + (w ? kColS1 : 0u);
            const uint32_t qs = w ? qs1 : qs0;
            if (t < 0) {
              if (!more) continue;
              if (!(ok = warp_wait(&bar_q[w][qs % QB], (qs / QB) & 1u, ctl, kErrTimeoutTma))) break;
            } else {
              if (!(ok = warp_wait(&bar_p[w], w ? np1 : np0, ctl, kErrTimeoutSoftmax))) break;
              np0 ^= w ? 0u : 1u;
              np1 ^= w ? 1u : 0u;
              tc_fence_after();
              mma_pv<D>(tmem + (w ? kColO1 : kColO0), cs, smem_u32(sV(v.st)), idesc_pv, t > 0);
              commit_el(&bar_o[w]);
            }
            if (more) {
              tc_fence_after();
              mma_abT<D>(cs, smem_u32(sQ(w, qs % QB)), smem_u32(sK(k.st)), idesc_qk);
              commit_el(&bar_s[w]);
            } else {
              if (w) ++qs1;
              else ++qs0;
              commit_el(&bar_ofinal[w]);
              if (lane == 0) {
                unit_odd[w] = odd;
                mbar_arrive(&bar_ofinal[w]);  // (with the flag behind it)
              }
              __syncwarp();
            }
          }
          if (!ok) break;
          if (t >= 0) {
            commit_el(&bar_vempty[v.st]);
            v.step();
          }
          if (next) {
            commit_el(&bar_kempty[k.st]);
            k.step();
          }
        }
      } else if (nt > 0) {
        const uint32_t aQ0 = smem_u32(sQ(0, qs0 % QB)), aQ1 = smem_u32(sQ(1, qs1 % QB));
        ok = warp_wait(&bar_k[k.st], k.ph, ctl, kErrTimeoutTma);
        if (ok && n0 > 0) {
          ok = warp_wait(&bar_q[0][qs0 % QB], (qs0 / QB) & 1u, ctl, kErrTimeoutTma);
          if (ok) {
            ++qs0;
            tc_fence_after();
            mma_abT<D>(tmem, aQ0, smem_u32(sK(k.st)), idesc_qk);
            commit_el(&bar_s[0]);
          }
        }
        if (ok && n1 > 0) {
          ok = warp_wait(&bar_q[1][qs1 % QB], (qs1 / QB) & 1u, ctl, kErrTimeoutTma);
          if (ok) {
            ++qs1;
            tc_fence_after();
            mma_abT<D>(tmem + kColS1, aQ1, smem_u32(sK(k.st)), idesc_qk);
            commit_el(&bar_s[1]);
          }
        }
        if (!ok) break;
        commit_el(&bar_kempty[k.st]);
        k.step();
        for (int t = 0; t < nt; ++t) {
          if (t < t_part) {
            ok = warp_wait(&bar_v[v.st], v.ph, ctl, kErrTimeoutTma);
          } else {
            const int j = t - t_part, bit = (i & 1) * kPart + j;
            ok = warp_wait(&bar_care[i & 1][j], part_ph >> bit & 1u, ctl, kErrTimeoutOther);
            part_ph ^= 1u << bit;
            if (ok) odd |= care_odd[i & 1][j][0] | care_odd[i & 1][j][1];
          }
          if (!ok) break;
          const bool next = t + 1 < nt;
          if (next && !(ok = warp_wait(&bar_k[k.st], k.ph, ctl, kErrTimeoutTma))) break;
          if (t < n0) {
            if (!(ok = warp_wait(&bar_p[0], np0, ctl, kErrTimeoutSoftmax))) break;
            np0 ^= 1u;
            tc_fence_after();
            mma_pv<D>(tmem + kColO0, tmem, smem_u32(sV(v.st)), idesc_pv, t > 0);
            commit_el(&bar_o[0]);
            if (t + 1 < n0) {
              mma_abT<D>(tmem, aQ0, smem_u32(sK(k.st)), idesc_qk);
              commit_el(&bar_s[0]);
            } else {
              commit_el(&bar_ofinal[0]);
              if (lane == 0) {
                unit_odd[0] = odd;
                mbar_arrive(&bar_ofinal[0]);  // (with the flag behind it)
              }
              __syncwarp();
            }
          }
          if (t < n1) {
            if (!(ok = warp_wait(&bar_p[1], np1, ctl, kErrTimeoutSoftmax))) break;
            np1 ^= 1u;
            tc_fence_after();
            mma_pv<D>(tmem + kColO1, tmem + kColS1, smem_u32(sV(v.st)), idesc_pv, t > 0);
            commit_el(&bar_o[1]);
            if (t + 1 < n1) {
              mma_abT<D>(tmem + kColS1, aQ1, smem_u32(sK(k.st)), idesc_qk);
              commit_el(&bar_s[1]);
            } else {
              commit_el(&bar_ofinal[1]);
              if (lane == 0) {
                unit_odd[1] = odd;
                mbar_arrive(&bar_ofinal[1]);
              }
              __syncwarp();
            }
          }
          commit_el(&bar_vempty[v.st]);
          v.step();
          if (next) {
            commit_el(&bar_kempty[k.st]);
            k.step();
          }
        }
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&ring.left[i & 1]);
    }
  } else if (warp >= kCare) {
    // ------------------ value tiles that some row sees in part; warp 11: units ahead
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    const int half = warp - kCare;
    const int r0 = half * 64;  // each warp's half of the tile's rows
    RingAsker asker;
    int vst = 0;  // V slot of the unit's first tile
    uint32_t part_ph = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      if (!__all_sync(0xffffffffu, ring_take(&ring, i, ctl))) break;
      const Pair p(&ring, i);
      const int nt = p.nt();
      for (int t = p.t_part; t < nt; ++t) {
        const int j = t - p.t_part, bit = (i & 1) * kPart + j;
        if (!(ok = warp_wait(&bar_part[i & 1][j], part_ph >> bit & 1u, ctl, kErrTimeoutTma))) break;
        part_ph ^= 1u << bit;
        const int valid = min(kBN, p.n - t * kBN);  // rows of the tile that are keys
        const int keys = min(max(valid - r0, 0), 64) * 8;  // 16-byte pieces
        uint4* rows = reinterpret_cast<uint4*>(sV((vst + t) % VST) + r0 * 128);
        uint32_t bits = 0;
#pragma unroll
        for (int kb = 0; kb < D / 64; ++kb) {
          uint4* blk = rows + kb * (kBM * 8);
          for (int x = keys + lane; x < 64 * 8; x += 32) blk[x] = make_uint4(0u, 0u, 0u, 0u);
          if (p.causal) {
#pragma unroll 8
            for (int x = lane; x < keys; x += 32) {
              const uint4 y = blk[x];
              bits |= non_finite_bits<BF>(y.x) | non_finite_bits<BF>(y.y) | non_finite_bits<BF>(y.z) |
                      non_finite_bits<BF>(y.w);
            }
          }
        }
        const bool odd = __any_sync(0xffffffffu, (bits & 0x80008000u) != 0u);
        if (odd) {
          for (int kb = 0; kb < D / 64; ++kb)
            for (int x = lane; x < keys; x += 32) {
              uint4 y = rows[kb * (kBM * 8) + x];
              y.x &= ~non_finite2<BF>(y.x);
              y.y &= ~non_finite2<BF>(y.y);
              y.z &= ~non_finite2<BF>(y.z);
              y.w &= ~non_finite2<BF>(y.w);
              rows[kb * (kBM * 8) + x] = y;
            }
        }
        if (lane == 0) care_odd[i & 1][j][half] = odd;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_care[i & 1][j]);
      }
      vst = (vst + nt) % VST;
      __syncwarp();
      if (ok && half == 0 && lane == 0) mbar_arrive(&ring.left[i & 1]);
      if (ok && half == 1) {
        if (asks)
          ok = asker.pass(&ring, args, list, i, ctl,
                          [&](const PackedUnit& u, int4(&words)[4]) { make_pair(u, TB, words); });
        ok = __all_sync(0xffffffffu, ok);
      }
    }
    if (asks) asker.drain(&ring, drain);
  } else {
    // ------------------------------- softmax / correction / epilogue (tile w)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int w = warp >> 2;
    const int r = threadIdx.x & 127;
    const int tok = static_cast<int>(args.g_div.div(r)), g = r - tok * G;  // of the tile
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t scol = w ? kColS1 : 0u, ocol = w ? kColO1 : kColO0;
    const bool serves = r == 0;  // the group's thread that loads Q and stores O
    uint32_t np = 0, units = 0;  // parities of this group's tiles, and units with any
    RingAt<QB> q;                // Q of the unit at hand
    // QB == 1: the serving thread loads Q, and waits until it knows of the unit behind unit i.  That
    // needs nothing from this group any more.
    uint32_t q_armed = 0;
    auto load_q = [&](int i) {
      const Pair p(&ring, i);
      if (p.n_t(w) == 0) return;
      mbar_expect_tx(&bar_q[w][0], qbytes);
      load_rows<D>(sQ(w, 0), &tm_q, &bar_q[w][0], p.head * G, p.row + w * TB);
      ++q_armed;
    };
    auto load_next_q = [&](int i) {
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // O of the buffer's last unit is on its way
      if (ring_take(&ring, i + 1, ctl)) load_q(i + 1);
    };
    if (QB == 1 && serves) load_q(0);
    bool ok = true;
    for (int i = 0;; ++i) {
      if (!__all_sync(0xffffffffu, ring_take(&ring, i, ctl))) break;
      int n, sees, t_part;  // key tiles, last key of this row (the rest of the unit is read again behind the loop)
      {
        const Pair p(&ring, i);
        n = p.n_t(w);
        sees = p.causal ? min(p.n - 1, p.off + w * TB + tok) : p.n - 1;
        t_part = p.t_part;
      }
      float m_ref = -INFINITY, l = 0.f;
      if (SHORT && n <= kFewTiles) {
        // A short unit's time is that of fetching code that runs once in it: 32 columns at a time, as far as
        // a row of the warp sees, and twice over the scores.
#pragma unroll 1
        for (int t = 0; t < n; ++t, np ^= 1u) {
          if (!(ok = warp_wait(&bar_s[w], np, ctl, kErrTimeoutMma))) break;
          tc_fence_after();
          if (QB == 2 && t == 0 && serves) {  // O of the last unit has left the other buffer
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            mbar_arrive(&bar_qfree[w]);
          }
          const int lim = sees - t * kBN;
          // (rows' tokens ascend)
          const int near = __shfl_sync(0xffffffffu, lim, 0), far = __shfl_sync(0xffffffffu, lim, 31);
          const int chunks = min(max(far + 32, 0) >> 5, 4);
          float x[32];
          auto load = [&](int c) {
            uint32_t s[32];
            tmem_ld_x32(lane_addr + scol + 32 * c, s);
            tmem_ld_wait(s);
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(s[j]);
            if (32 * c + 31 > near) {
              const int v = lim - 32 * c;
              const uint32_t keep = v >= 31 ? 0xffffffffu : v < 0 ? 0u : (2u << v) - 1u;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!(keep >> j & 1u)) x[j] = -INFINITY;
            }
          };
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < chunks; ++c) {
            load(c);
            float m4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              m4[k] = fmax3(x[k], x[4 + k], x[8 + k]);
              m4[k] = fmax3(m4[k], x[12 + k], x[16 + k]);
              m4[k] = fmax3(m4[k], x[20 + k], x[24 + k]);
              m4[k] = fmaxf(m4[k], x[28 + k]);
            }
            mx = fmaxf(mx, fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]));
          }
          const float m_new = fmaxf(m_ref, mx * args.scale_log2);
          float alpha = 1.f;
          bool resc = false;
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
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
            if (c < chunks) {
              load(c);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float2 y = ffma2(make_float2(x[2 * e], x[2 * e + 1]), sc2, nm2);
                const float2 pr = make_float2(ex2(y.x), ex2(y.y));
                rs2[e & 3] = fadd2(rs2[e & 3], pr);
                pk[e] = pack2<BF>(pr.x, pr.y);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) pk[e] = 0u;
            }
            tmem_st_x16(lane_addr + scol + 16 * c, pk);
          }
          const float2 rsa = fadd2(fadd2(rs2[0], rs2[1]), fadd2(rs2[2], rs2[3]));
          l = l * alpha + (rsa.x + rsa.y);
          if (t > 0 && __any_sync(0xffffffffu, resc)) {
            if (!(ok = warp_wait(&bar_o[w], np ^ 1u, ctl, kErrTimeoutMma))) break;
            tc_fence_after();
#pragma unroll 1
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
      } else {
        for (int t = 0; t < n; ++t, np ^= 1u) {
          if (!(ok = warp_wait(&bar_s[w], np, ctl, kErrTimeoutMma))) break;
          tc_fence_after();
          if (QB == 2 && t == 0 && serves) {  // O of the last unit has left the other buffer
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            mbar_arrive(&bar_qfree[w]);
          }
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
            // (rows' tokens ascend)
            const int near = __shfl_sync(0xffffffffu, lim, 0), far = __shfl_sync(0xffffffffu, lim, 31);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (32 * c + 31 > near) {
                const int v = lim - 32 * c;
                const uint32_t keep = v >= 31 ? 0xffffffffu : v < 0 ? 0u : (2u << v) - 1u;
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (!(keep >> j & 1u)) x[32 * c + j] = -INFINITY;
              }
            }
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
            if (!(ok = warp_wait(&bar_o[w], np ^ 1u, ctl, kErrTimeoutMma))) break;
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
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      const Pair p(&ring, i);
      const int left = p.left - w * TB;
      const int tokens = min(left, TB);  // (none: the sequence ends before this tile)
      const long long qrow = static_cast<long long>(p.row) + w * TB;
      auto out_row = [&](int j) -> void* {
        const int k = static_cast<int>(args.g_div.div(j));
        return static_cast<T*>(args.o) + (qrow + k) * args.o_t + (p.head * G + j - k * G) * args.o_h;
      };
      if (n == 0) {  // rows that see nothing
        if (QB == 1 && serves) load_next_q(i);
        if (tok < tokens) args.lse[(qrow + tok) * args.shape.Hq + p.head * G + g] = -INFINITY;
        const int c = args.dg >> 3;
        for (int j = r; j < tokens * G * c; j += 128) {
          const int row = j / c;
          static_cast<uint4*>(out_row(row))[j - row * c] = make_uint4(0u, 0u, 0u, 0u);
        }
      } else {
        if (!(ok = warp_wait(&bar_ofinal[w], units, ctl, kErrTimeoutMma))) break;
        units ^= 1u;
        tc_fence_after();
        if (tok < tokens)
          args.lse[(qrow + tok) * args.shape.Hq + p.head * G + g] = l != 0.f ? (m_ref + lg2(l)) * kLn2 : -INFINITY;
        const float inv_l = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
        const uint32_t stage = smem_u32(sQ(w, q.st));  // (its products are done)
        // non-finite values that were taken out of this unit's tiles: this row's are added to O here
        if (p.causal && *reinterpret_cast<volatile int*>(&unit_odd[w]) != 0) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld_x32(lane_addr + ocol + 32 * c, ov);
            tmem_ld_wait(ov);
#pragma unroll
            for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * inv_l);
            if (tok < tokens && l > 0.f) {
              const int ng = chunk_groups(args.dg, 32 * c);
              for (int k = t_part * kBN; k <= min(sees, n * kBN - 1); ++k) {
                const T* vrow = static_cast<const T*>(args.v) + (static_cast<long long>(p.krow) + k) * args.vt +
                                p.head * args.vh + 32 * c;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  if (q >= ng) break;
                  const uint4 xv = __ldg(reinterpret_cast<const uint4*>(vrow) + q);
                  const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                  for (int k2 = 0; k2 < 4; ++k2) {
                    const uint32_t m = non_finite2<BF>(xs[k2]);
                    if (!m) continue;
                    const uint32_t y = xs[k2] & m;
                    const T* h = reinterpret_cast<const T*>(&y);
                    float *lo = reinterpret_cast<float*>(&ov[8 * q + 2 * k2]), *hi = lo + 1;
                    if (m & 0xffffu) *lo += static_cast<float>(h[0]);
                    if (m >> 16) *hi += static_cast<float>(h[1]);
                  }
                }
              }
            }
            stage_row_chunk_sw128<BF>(stage, r, c, ov, 1.f);
          }
        } else {
#pragma unroll(SHORT ? 1 : 4)
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld_x32(lane_addr + ocol + 32 * c, ov);
            tmem_ld_wait(ov);
            stage_row_chunk_sw128<BF>(stage, r, c, ov, inv_l);
          }
        }
        tc_fence_before();  // O's columns are free for the next unit
        fence_proxy_async_smem();
        named_bar_sync(1 + w, 4 * 32);  // the tile's four warps have staged their rows
        if (left >= TB) {  // whole: a box
          if (serves) {
#pragma unroll
            for (int kb = 0; kb < D / 64; ++kb)
              tma_store_3d(&tm_o, sQ(w, q.st) + kb * (kBM * 128), kb * 64, p.head * G, p.row + w * TB);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        } else {  // the rows behind it are another sequence's
          copy_tile_rows(sQ(w, q.st), args.dg, r, 128, tokens * G, out_row);
          named_bar_sync(1 + w, 4 * 32);
        }
        if (QB == 1 && serves) load_next_q(i);
        q.step();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.left[i & 1]);
    }
    if (serves) {
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      if (QB == 1) drain_q(w, q_armed);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc(tmem, 512);
}

template <typename T, int D, bool SHORT>
cudaError_t run_kernel(const PackedMaps& m, const PackedArgs& a, cudaStream_t s) {
  using C = PfCfg<D>;
  auto kern = packed_fwd_kernel<T, D, SHORT>;
  static std::atomic<bool> attr[kMaxDevices];
  cudaError_t e = smem_attr_once(kern, C::SMEM, attr);
  if (e != cudaSuccess) return e;
  const long long blocks = a.shape.bound(kPackedFwd) * a.shape.Hkv;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  kern<<<static_cast<unsigned>(blocks), kThreads, C::SMEM, s>>>(m.q, m.k, m.v, m.o, a);
  return cudaGetLastError();
}

// Sequences of up to 512 keys on average: most units have one or two key tiles.  With and without the instance for
// them, us, 32768 tokens (16384 from 512 on): 32 / 4 heads of 64, sequences of 100 tokens 114 / 153, 256 111 / 132,
// 400 138 / 147, 512 78 / 81, 1024 109 / 108, 2048 173 / 167; 32 / 8 of 128: 100 171 / 194, 256 168 / 171, 400 227 / 230,
// 1024 159 / 155.
template <typename T, int D>
cudaError_t run(const PackedMaps& m, const PackedArgs& a, cudaStream_t s) {
  const bool few = a.shape.total_k <= 512ll * a.shape.B;
  return few ? run_kernel<T, D, true>(m, a, s) : run_kernel<T, D, false>(m, a, s);
}

}  // namespace

cudaError_t launch_packed_fwd(bool bf16, int D, const PackedMaps& m, const PackedArgs& a, cudaStream_t s) {
  if (D == 64) return bf16 ? run<__nv_bfloat16, 64>(m, a, s) : run<__half, 64>(m, a, s);
  if (D == 128) return bf16 ? run<__nv_bfloat16, 128>(m, a, s) : run<__half, 128>(m, a, s);
  return cudaErrorInvalidValue;
}

}  // namespace ta

TA_GUARD_ACCESSOR(packed_fwd)
