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
// asks for units ahead (UnitRing) and zeroes the rows of a unit's last streamed tile
// that belong to no token of the sequence: their P and dS are zero, and a
// neighbour's infinity in a product with zero would be NaN.  Such tiles come in
// through barriers of their own.
//
// The rings run on from one unit to the next.  What leaves a block goes
// through a ring's slot, too: an entry behind the unit's tiles, which the storing
// thread hands back.
//
// Bound, for long sequences, by the MMAs: S and dP are made in both passes, seven products where
// five would do, and no dQ is summed in memory.  Three documents of 2000 to 8192 tokens, 32 / 8 heads of
// 128, bf16: 2.05 ms (0.84 + 1.20); seven products at the measured peak take 1.81, five 1.30.
// Short documents are bound by the way from one role to the next: 24 of up to 700 tokens, 16 heads
// of 64, 92 us (45 + 52 timed one by one) where memory would need 19.  The MMA warp's loops hold one copy of
// each product, a unit's first scores too (95 us with a copy of their own; the long case takes the same).
#include "launch.h"
#include "packed.cuh"

namespace ta {

namespace {

// Registers: 384 x 168 at launch = 256 x 200 (row warps) + 128 x 104; warp 11 only makes up the
// warpgroup.  With 168 a thread for all and units asked for one ahead, three documents of
// 2000 to 8192 tokens, 32 / 8 heads of 128, took 2185 us, so 2024 us.
constexpr int kThreads = 384;
constexpr int kProducer = 8, kMma = 9, kCare = 10;
constexpr int kRowWarps = 8;

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
// The row threads' (256) zeros into rows of an output.
template <typename F>
__device__ __forceinline__ void zero_rows(int rows, int dg, F row) {
  const int c = dg >> 3;
  for (int j = threadIdx.x; j < rows * c; j += kRowWarps * 32) {
    const int k = j / c;
    static_cast<uint4*>(row(k))[j - k * c] = make_uint4(0u, 0u, 0u, 0u);
  }
}

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

// Whether half of row r of a swizzled tile holds the numbers of a value's row of `dg` elements (zeros
// of either sign are one number).
template <int D>
__device__ __forceinline__ bool half_equal(const void* row, int dg, const uint8_t* b, int r, int half) {
  uint32_t eq = 0xffffffffu;
  auto both = [&](uint32_t u, uint32_t v) { eq &= __vcmpeq2(u, v) | __vcmpeq2((u | v) & 0x7fff7fffu, 0u); };
#pragma unroll 1
  for (int gc = half * (D / 16); gc < (half + 1) * (D / 16) && gc * 8 < dg; ++gc) {
    const uint4 x = __ldg(static_cast<const uint4*>(row) + gc);
    const uint4 y = *reinterpret_cast<const uint4*>(b + (gc >> 3) * (kBM * 128) + r * 128 + (((gc & 7) ^ (r & 7)) * 16));
    both(x.x, y.x);
    both(x.y, y.y);
    both(x.z, y.z);
    both(x.w, y.w);
  }
  return eq == 0xffffffffu;
}
// named_bar_sync that tells whether x held for all of its threads.
__device__ __forceinline__ bool named_bar_all(uint32_t id, uint32_t count, bool x) {
  uint32_t all = x;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %0, 0;\n barrier.cta.red.and.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "+r"(all)
      : "r"(id), "r"(count)
      : "memory");
  return all != 0u;
}

// ======================================================================
//                         dQ (query-stationary)
// ======================================================================
// Q and dO are the A operands of every score product and live in TMEM; they
// come through the ring as the entry in front of a unit's K/V tiles.  O has a tile
// of its own, and delta is formed while the first products run.  dQ leaves
// through the entry behind the tiles.
//
// A sequence's only key: where a row's O is that key's value, dS = P (<dO, V> - <dO, O>) = 0.  The
// product's sum and delta's are of the same numbers in different orders and would leave their rounding, so
// such rows' delta is the product's own dP, here and, through memory, in the other pass (whose product sums
// the same terms in the same order).  With O and L over more keys than this call's, O is another, and dS what it is.
// (The same for every row that sees one key, the first of each causal sequence among them, would cost
// short documents 2 us of 92: the value's row is fetched in the first unit of each.)
template <int D>
struct PdqCfg {
  static constexpr int TILE = (D / 64) * kBM * 128;
  static constexpr int STAGE = 2 * TILE;  // K, V
  static constexpr int ST_FIT = (kSmemMax - 2048 - TILE) / STAGE;
  static constexpr int STAGES = ST_FIT > 4 ? 4 : ST_FIT;
  static constexpr int OFF_O = STAGES * STAGE;  // O, then the halves of delta
  static constexpr int SMEM = OFF_O + TILE + 1024;
  static constexpr uint32_t COL_A = 0, COL_B = 128, COL_DQ = 256;
  static constexpr uint32_t COL_QT = 256 + D, COL_DOT = 256 + D + D / 2;
  static_assert(STAGES >= 3 && SMEM + 2048 <= kSmemMax, "shared memory");
  static_assert(COL_DOT + D / 2 <= 512, "TMEM");
};

struct DqUnit {
  int row, krow, n, off;         // first token's row, first key's row, keys, last key the first token sees
  int left, nkv, head, causal;   // tokens to the sequence's end, key tiles, key head
  __device__ __forceinline__ DqUnit(const UnitRing* r, int i) {
    const int4 a = ring_words(r, i, 0), b = ring_words(r, i, 1);
    row = a.x;
    krow = a.y;
    n = a.z;
    off = a.w;
    left = b.x;
    nkv = b.y;
    head = b.z;
    causal = b.w;
  }
  __device__ __forceinline__ bool ragged() const { return nkv * kBN > n; }  // the last tile ends behind the keys
};
__device__ __forceinline__ void make_dq_unit(const PackedUnit& u, int TB, int4 (&words)[4]) {
  words[0] = make_int4(u.row, u.krow, u.n, u.off);
  words[1] = make_int4(u.left, packed_key_tiles(min(u.left, TB), u.off, u.n, u.pad[0]), u.pad[1], u.pad[0]);
}

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
  __shared__ __align__(16) UnitRing ring;
  __shared__ __align__(8) uint64_t bar_qfree, bar_kv[STAGES], bar_kvempty[STAGES];
  __shared__ __align__(8) uint64_t bar_s, bar_consumed, bar_dp, bar_ds[2], bar_done, bar_o;
  __shared__ __align__(8) uint64_t bar_last[2], bar_care[2];  // [unit % 2]: a ragged last tile is in, is seen to
  __shared__ __align__(8) uint64_t bar_out[2];                // [live units so far % 2]: dQ's slot is free to write
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const PackedList list = packed_list(args, kPackedDq);
  if (blockIdx.x >= list.items) return;
  const int G = args.shape.G, TB = args.shape.TB;
  const int box = (D / 64) * TB * G * 128;  // bytes of a query tile

  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto sK = [&](int st) { return base + st * C::STAGE; };           // K | Q | dQ
  auto sV = [&](int st) { return base + st * C::STAGE + C::TILE; };  // V | dO
  uint8_t* sO = base + C::OFF_O;
  float* halves = reinterpret_cast<float*>(sO);

  const bool asks = threadIdx.x == kCare * 32;
  if (asks) {
    make_dq_unit(packed_item(args, list, blockIdx.x), TB, ring.unit[0]);
    ring.unit[0][3].w = 1;
  }
  WaitCtl ctl{args.err, args.timeout_ns, &abort_flag};
  if (threadIdx.x == 0) {
    abort_flag = 0;
    ring_init(&ring, kRowWarps + 2);  // row warps, MMA, producer
    mbar_init(&bar_qfree, kRowWarps);
    for (int st = 0; st < STAGES; ++st) {
      mbar_init(&bar_kv[st], 1);
      mbar_init(&bar_kvempty[st], 1);
    }
    mbar_init(&bar_s, 1);
    mbar_init(&bar_consumed, kRowWarps);
    mbar_init(&bar_dp, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_ds[i], kRowWarps);
      mbar_init(&bar_last[i], 1);
      mbar_init(&bar_care[i], 1);
      mbar_init(&bar_out[i], 1);
    }
    mbar_init(&bar_done, 1);
    mbar_init(&bar_o, 1);
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
  int zero = 0;  // (an exit waits for its own copies whatever the abort flag says)
  const WaitCtl drain{args.err, args.timeout_ns, reinterpret_cast<volatile int*>(&zero)};

  if (warp == kProducer) {
    // ------------------------------------------------------------ producer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (lane == 0) {
      RingAt<STAGES> k;
      int e = 0;              // entries so far
      uint32_t own = 0;       // slots whose last entry did not come through bar_kv
      uint32_t last_ph = 0;   // bit i: bar_last[i] has been armed an odd number of times
      uint32_t outs = 0;
      bool ok = true;
      auto slot = [&] { return e < STAGES || mbar_wait(&bar_kvempty[k.st], k.ph ^ 1u, ctl, kErrTimeoutMma); };
      for (int i = 0; ok && ring_take(&ring, i, ctl); ++i) {
        const DqUnit p(&ring, i);
        if (p.nkv == 0) mbar_arrive(&ring.near);
        for (int t = -1; p.nkv > 0 && t <= p.nkv; ++t, ++e) {
          if (t == p.nkv) mbar_arrive(&ring.near);
          if (!(ok = slot())) break;
          own &= ~(1u << k.st);
          if (t < 0) {
            mbar_expect_tx(&bar_kv[k.st], 2 * box);
            load_rows<D>(sK(k.st), &tm_q, &bar_kv[k.st], p.head * G, p.row);
            load_rows<D>(sV(k.st), &tm_do, &bar_kv[k.st], p.head * G, p.row);
          } else if (t < p.nkv) {
            uint64_t* bar = &bar_kv[k.st];
            if (t == p.nkv - 1 && p.ragged()) {
              mbar_arrive(bar);  // (the ring's own phase passes on)
              bar = &bar_last[i & 1];
              last_ph ^= 1u << (i & 1);
              own |= 1u << k.st;
            }
            mbar_expect_tx(bar, 2 * C::TILE);
            load_rows<D>(sK(k.st), &tm_k, bar, p.krow + t * kBN, p.head);
            load_rows<D>(sV(k.st), &tm_v, bar, p.krow + t * kBN, p.head);
          } else {
            mbar_arrive(&bar_kv[k.st]);
            mbar_arrive(&bar_out[outs & 1]);
            ++outs;
            own |= 1u << k.st;
          }
          k.step();
        }
        if (ok) mbar_arrive(&ring.left[i & 1]);
      }
      for (int t = e - STAGES > 0 ? e - STAGES : 0; t < e; ++t)
        if (!(own >> (t % STAGES) & 1u)) mbar_wait(&bar_kv[t % STAGES], (t / STAGES) & 1, drain, kErrTimeoutTma);
      for (int j = 0; j < 2; ++j) mbar_wait(&bar_last[j], (last_ph >> j & 1u) ^ 1u, drain, kErrTimeoutTma);
    }
  } else if (warp == kMma) {
    // ----------------------------------------------------------------- MMA
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    constexpr uint32_t idesc_s = idesc_f16(kBM, kBN, BF, false, false);
    constexpr uint32_t idesc_g = idesc_f16(kBM, D, BF, false, true);
    RingAt<STAGES> k;
    uint32_t units = 0, tiles = 0, nc = 0, care_ph = 0;  // parities
    bool any = false, ok = true;
    for (int i = 0; ok; ++i) {
      if (!__all_sync(0xffffffffu, ring_take(&ring, i, ctl))) break;
      int nkv;
      bool ragged;
      {
        const DqUnit p(&ring, i);
        nkv = p.nkv;
        ragged = p.ragged();
      }
      if (nkv > 0) {
        auto kv_ready = [&](int t) {
          if (ragged && t == nkv - 1) {
            const uint32_t ph = care_ph >> (i & 1) & 1u;
            care_ph ^= 1u << (i & 1);
            return warp_wait(&bar_care[i & 1], ph, ctl, kErrTimeoutOther);
          }
          return warp_wait(&bar_kv[k.st], k.ph, ctl, kErrTimeoutTma);
        };
        // Q and dO are in TMEM: their slot is free, and the last unit's S has been read
        ok = warp_wait(&bar_qfree, units, ctl, kErrTimeoutSoftmax);
        units ^= 1u;
        if (!ok) break;
        commit_el(&bar_kvempty[k.st]);
        k.step();
#pragma unroll 1
        for (int t = -1; t < nkv; ++t) {
          const int st = k.st;
          const bool next = t + 1 < nkv;
          if (t >= 0) k.step();
          if (next) {
            if (any && !(ok = warp_wait(&bar_consumed, nc, ctl, kErrTimeoutSoftmax))) break;
            nc ^= any ? 1u : 0u;
            any = true;
            if (!(ok = kv_ready(t + 1))) break;
            tc_fence_after();
            mma_tmem_abT<D>(tmem + C::COL_A, tmem + C::COL_QT, smem_u32(sK(k.st)), idesc_s);
            commit_el(&bar_s);
          }
          if (t >= 0) {
            if (!(ok = warp_wait(&bar_ds[0], tiles, ctl, kErrTimeoutSoftmax))) break;
            tc_fence_after();
            mma_half_y<0>(tmem + C::COL_DQ, tmem + C::COL_B, smem_u32(sK(st)), idesc_g, t > 0);
            if (!(ok = warp_wait(&bar_ds[1], tiles, ctl, kErrTimeoutSoftmax))) break;
            tiles ^= 1u;
            tc_fence_after();
            mma_half_y<1>(tmem + C::COL_DQ, tmem + C::COL_B, smem_u32(sK(st)), idesc_g, true);
            commit_el(&bar_kvempty[st]);
          }
          if (next) {
            mma_tmem_abT<D>(tmem + C::COL_B, tmem + C::COL_DOT, smem_u32(sV(k.st)), idesc_s);  // dP = dO V^T
            commit_el(&bar_dp);
          }
        }
        if (!ok) break;
        commit_el(&bar_done);
        k.step();  // dQ's entry
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.left[i & 1]);
    }
  } else if (warp >= kCare) {
    // --------------------------------- units ahead; rows behind the keys
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == kCare) {
      RingAsker asker;
      int st = 0;  // slot of the unit's first entry
      uint32_t ph = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        if (!__all_sync(0xffffffffu, ring_take(&ring, i, ctl))) break;
        const DqUnit p(&ring, i);
        if (p.nkv > 0) {
          if (p.ragged()) {
            if (!(ok = warp_wait(&bar_last[i & 1], ph >> (i & 1) & 1u, ctl, kErrTimeoutTma))) break;
            ph ^= 1u << (i & 1);
            const int at = (st + p.nkv) % STAGES, first = p.n - (p.nkv - 1) * kBN;
            zero_tile_rows<D / 64>(sK(at), first, lane);
            zero_tile_rows<D / 64>(sV(at), first, lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_care[i & 1]);
          }
          st = (st + p.nkv + 2) % STAGES;
        }
        if (asks)
          ok = asker.pass(&ring, args, list, i, ctl,
                          [&](const PackedUnit& u, int4(&words)[4]) { make_dq_unit(u, TB, words); });
        ok = __all_sync(0xffffffffu, ok);
      }
      if (asks) asker.drain(&ring, drain);
    }
  } else {
    // --------------------------------------------- query-row softmax gradient
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int hc = warp >> 2;  // key half of the tile: columns [64 hc, 64 hc + 64)
    const int cb = 64 * hc;
    const int r = threadIdx.x & 127;
    const int tok = static_cast<int>(args.g_div.div(r)), hq = r - tok * G;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const bool serves = threadIdx.x == 0;  // loads O, stores dQ
    RingAt<STAGES> k;
    uint32_t units = 0, tiles = 0, outs = 0, os = 0;  // os: (serving thread) O tiles asked for
    int lent = -1;                                    // slot that a store still reads
    auto load_o = [&](int i) {
      const DqUnit p(&ring, i);
      if (p.nkv == 0) return;
      mbar_expect_tx(&bar_o, box);
      load_rows<D>(sO, &tm_o, &bar_o, p.head * G, p.row);
      ++os;
    };
    auto give_back = [&] {
      if (lent >= 0) {
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        mbar_arrive(&bar_kvempty[lent]);
        lent = -1;
      }
    };
    if (serves) load_o(0);
    bool ok = true;
    for (int i = 0; ok; ++i) {
      if (!__all_sync(0xffffffffu, ring_take(&ring, i, ctl))) break;
      const DqUnit p(&ring, i);
      const int nkv = p.nkv;
      const bool in = tok < min(p.left, TB);
      const size_t g = (static_cast<size_t>(p.row) + (in ? tok : 0)) * args.shape.Hq + p.head * G + (in ? hq : 0);
      T* const dq = static_cast<T*>(args.dq) + static_cast<long long>(p.row) * args.dq_t + p.head * G * args.dq_h;
      auto out_row = [&](int j) -> void* {
        const int tk = static_cast<int>(args.g_div.div(j));
        return dq + tk * args.dq_t + (j - tk * G) * args.dq_h;
      };
      if (nkv == 0) {  // rows that see nothing: O = 0
        if (hc == 0 && in) args.delta[g] = 0.f;
        zero_rows(min(p.left, TB) * G, args.dg, out_row);
        if (serves) {
          give_back();
          if (ring_take(&ring, i + 1, ctl)) load_o(i + 1);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ring.left[i & 1]);
        continue;
      }
      const float neg_L2 = in ? -args.lse[g] * kLog2e : -INFINITY;
      const int sees = p.causal ? min(p.n - 1, p.off + tok) : p.n - 1;
      const int t_part = p.causal ? min(p.n / kBN, p.off < 0 ? 0 : (p.off + 1) / kBN) : p.n / kBN;
      // group 0 copies Q, group 1 dO into TMEM (the last unit's products are done)
      if (!(ok = warp_wait(&bar_kv[k.st], k.ph, ctl, kErrTimeoutTma))) break;
      tile_row_to_tmem<D>(hc == 0 ? sK(k.st) : sV(k.st), r, lane_addr + (hc == 0 ? C::COL_QT : C::COL_DOT));
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_qfree);
      k.step();
      if (serves) give_back();
      // delta: each group half of every row's columns
      if (!(ok = warp_wait(&bar_qfree, units, ctl, kErrTimeoutSoftmax) && warp_wait(&bar_o, units, ctl, kErrTimeoutTma)))
        break;
      tc_fence_after();
      float dlt = half_dot<T, D>(lane_addr + C::COL_DOT, sO, r, hc);
      const bool lone = p.n == 1 && in && sees == 0;
      const bool same = !lone || half_equal<D>(static_cast<const T*>(args.v) + static_cast<long long>(p.krow) * args.vt +
                                                   p.head * args.vh,
                                               args.dg, sO, r, hc);
      named_bar_sync(1, kRowWarps * 32);  // the halves go over O
      halves[hc * kBM + r] = dlt;
      // the tile in which delta becomes the lone key's dP (-1: none)
      const int t_lone = named_bar_all(1, kRowWarps * 32, same) && lone && hc == 0 ? 0 : -1;
      dlt = halves[r] + halves[kBM + r];
      fence_proxy_async_smem();
      for (int t = 0; t < nkv; ++t, tiles ^= 1u) {
        const int k0 = t * kBN;
        if (!(ok = warp_wait(&bar_s, tiles, ctl, kErrTimeoutMma))) break;
        tc_fence_after();
        uint32_t sv[64];
        tmem_ld_x32(lane_addr + C::COL_A + cb, TB_CHUNK(sv, 0));
        tmem_ld_x32(lane_addr + C::COL_A + cb + 32, TB_CHUNK(sv, 1));
        tmem_ld_wait(TB_CHUNK(sv, 0));
        tmem_ld_wait(TB_CHUNK(sv, 1));
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_consumed);  // S buffer free for S(t + 1)
        float pr[64];
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const float2 y = ffma2(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])),
                                 make_float2(args.scale_log2, args.scale_log2), make_float2(neg_L2, neg_L2));
          pr[c] = ex2(y.x);
          pr[c + 1] = ex2(y.y);
        }
        if (t >= t_part) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int lim = sees - k0 - cb - 32 * h;
            const uint32_t keep = lim >= 31 ? 0xffffffffu : lim < 0 ? 0u : (2u << lim) - 1u;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(keep >> c & 1u)) pr[32 * h + c] = 0.f;
          }
        }
        if (!(ok = warp_wait(&bar_dp, tiles, ctl, kErrTimeoutMma))) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t dp[32];
          tmem_ld_x32(lane_addr + C::COL_B + cb + 32 * c, dp);
          tmem_ld_wait(dp);
          if (c == 0 && t == t_lone) dlt = __uint_as_float(dp[0]);
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int c0 = 32 * c + 2 * e;
            const float2 ds = fmul2(make_float2(pr[c0], pr[c0 + 1]),
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
        k.step();
      }
      if (!ok) break;
      if (hc == 0 && in) args.delta[g] = dlt;
      if (!(ok = warp_wait(&bar_done, units, ctl, kErrTimeoutMma) &&
                 warp_wait(&bar_out[outs & 1], (outs >> 1) & 1, ctl, kErrTimeoutMma)))
        break;
      units ^= 1u;
      ++outs;
      tc_fence_after();
      // (every warp has handed in its last dS, and so has read O and delta)
      if (serves && ring_take(&ring, i + 1, ctl)) load_o(i + 1);
      __syncwarp();
      // dQ (x sm_scale) staged in its slot
#pragma unroll
      for (int cc = 0; cc < D / 64; ++cc) {
        const int c = hc * (D / 64) + cc;
        uint32_t v[32];
        tmem_ld_x32(lane_addr + C::COL_DQ + 32 * c, v);
        tmem_ld_wait(v);
        stage_row_chunk_sw128<BF>(smem_u32(sK(k.st)), r, c, v, args.sm_scale);
      }
      tc_fence_before();
      fence_proxy_async_smem();
      named_bar_sync(1, kRowWarps * 32);
      if (p.left >= TB) {
        if (serves) {
#pragma unroll
          for (int kb = 0; kb < D / 64; ++kb)
            tma_store_3d(&tm_dq, sK(k.st) + kb * (kBM * 128), kb * 64, p.head * G, p.row);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          lent = k.st;
        }
      } else {  // the rows behind it are another sequence's
        copy_tile_rows(sK(k.st), args.dg, threadIdx.x, kRowWarps * 32, p.left * G, out_row);
        named_bar_sync(1, kRowWarps * 32);
        if (serves) mbar_arrive(&bar_kvempty[k.st]);
      }
      k.step();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.left[i & 1]);
    }
    if (serves) {
      give_back();
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      if (os > 0) mbar_wait(&bar_o, (os - 1) & 1, drain, kErrTimeoutTma);
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
// ahead into a double buffer.  K and V are free for the next unit's once the last
// S^T and dP^T are done; dK leaves through the Q ring, dV through dO's.  All
// shared memory is in the dynamic region (K, V, the rings, L and delta, barriers).
template <int D>
struct PkvCfg {
  static constexpr int TILE = (D / 64) * kBM * 128;
  static constexpr int QST = D == 128 ? 3 : 4;
  static constexpr int OST = D == 128 ? 2 : 4;
  static constexpr int LD_OFF = (2 + QST + OST) * TILE;  // [buffer][half][L, delta][64] floats
  static constexpr int BAR_OFF = LD_OFF + 2 * 2 * 2 * 64 * 4;
  static constexpr int BAR_BYTES = 576;
  static constexpr int USED = BAR_OFF + BAR_BYTES;
  static constexpr int PAD = (kSmemMax - USED) < 1023 ? (kSmemMax - USED) : 1023;
  static constexpr int SMEM = USED + PAD;
  static constexpr uint32_t COL_A = 0, COL_B = 128, COL_DV = 256, COL_DK = 256 + D;
  static_assert(PAD >= 0 && SMEM <= kSmemMax, "tiles do not fit in shared memory");
  static_assert(BAR_BYTES >= static_cast<int>(sizeof(UnitRing)) + 8 * (2 + 2 * QST + 2 * OST + 6 + 4 + 8 + 4) + 8, "barrier area too small");
};

struct KvUnit {
  int krow, n, row, left, off;  // first key's row, keys from it on, first token that sees any, tokens from it on; see PackedUnit
  int nq, head, causal;         // query tiles, key head
  int ragged;                   // the last tile ends behind the tokens
  __device__ __forceinline__ KvUnit(const UnitRing* r, int i) {
    const int4 a = ring_words(r, i, 0), b = ring_words(r, i, 1), c = ring_words(r, i, 2);
    krow = a.x;
    n = a.y;
    row = a.z;
    left = a.w;
    off = b.x;
    nq = b.y;
    head = b.z;
    causal = b.w;
    ragged = c.x;
  }
};
__device__ __forceinline__ void make_kv_unit(const PackedUnit& u, int TB, int4 (&words)[4]) {
  const int nq = (u.left + TB - 1) / TB;
  words[0] = make_int4(u.krow, u.n, u.row, u.left);
  words[1] = make_int4(u.off, nq, u.pad[1], u.pad[0]);
  words[2] = make_int4(nq * TB > u.left, 0, 0, 0);
}

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
  UnitRing& ring = *reinterpret_cast<UnitRing*>(base + C::BAR_OFF);
  uint64_t* bars = reinterpret_cast<uint64_t*>(&ring + 1);
  uint64_t& bar_kv = bars[0];
  uint64_t& bar_kvfree = bars[1];
  uint64_t* bar_qf = bars + 2;
  uint64_t* bar_qe = bar_qf + QST;
  uint64_t* bar_of = bar_qe + QST;
  uint64_t* bar_oe = bar_of + OST;
  uint64_t& bar_s = bar_oe[OST];
  uint64_t& bar_consumed = bar_oe[OST + 1];
  uint64_t& bar_dp = bar_oe[OST + 2];
  uint64_t* bar_ds = bar_oe + OST + 3;  // [chunk group]
  uint64_t& bar_done = bar_oe[OST + 5];
  uint64_t* bar_pub = bar_oe + OST + 6;  // [buffer * 2 + half]: L / delta of a tile stored
  uint64_t* bar_care = bar_pub + 4;      // [unit % 2 * 2 + (0: Q, 1: dO)]: a ragged last tile's rows zeroed
  uint64_t* bar_last = bar_care + 4;     // the same: it is in
  uint64_t* bar_out = bar_last + 4;      // [live units % 2 * 2 + (0: Q ring, 1: dO ring)]: a slot is free to write
  uint32_t& tmem_slot = *reinterpret_cast<uint32_t*>(bar_out + 4);
  int& abort_flag = *(reinterpret_cast<int*>(bar_out + 4) + 1);
  float* sLD = reinterpret_cast<float*>(base + C::LD_OFF);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const PackedList list = packed_list(args, kPackedDkdv);
  if (blockIdx.x >= list.items) return;
  const int G = args.shape.G, TB = args.shape.TB;
  const int box = (D / 64) * TB * G * 128;

  uint8_t* sK = base;
  uint8_t* sV = base + C::TILE;
  auto sQ = [&](int i) { return base + (2 + i) * C::TILE; };
  auto sDO = [&](int i) { return base + (2 + QST + i) * C::TILE; };

  const bool asks = threadIdx.x == kCare * 32;
  if (asks) {
    make_kv_unit(packed_item(args, list, blockIdx.x), TB, ring.unit[0]);
    ring.unit[0][3].w = 1;
  }
  WaitCtl ctl{args.err, args.timeout_ns, &abort_flag};
  if (threadIdx.x == 0) {
    abort_flag = 0;
    ring_init(&ring, kRowWarps + 3);  // row warps, MMA, two producing lanes
    mbar_init(&bar_kv, 1);
    mbar_init(&bar_kvfree, 1);
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
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar_pub[i], kRowWarps / 2);
      mbar_init(&bar_care[i], 1);
      mbar_init(&bar_last[i], 1);
      mbar_init(&bar_out[i], 1);
    }
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
  int zero = 0;  // (an exit waits for its own copies whatever the abort flag says)
  const WaitCtl drain{args.err, args.timeout_ns, reinterpret_cast<volatile int*>(&zero)};

  if (warp == kProducer) {
    // ---------------------- producer: lane 0 K, V and the Q ring; lane 1 the dO ring
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (lane < 2) {
      const bool is_q = lane == 0;
      const int depth = is_q ? QST : OST;
      uint64_t* full = is_q ? bar_qf : bar_of;
      uint64_t* empty = is_q ? bar_qe : bar_oe;
      const CUtensorMap* map = is_q ? &tm_q : &tm_do;
      int e = 0;                     // entries so far
      uint32_t own = 0, last_ph = 0, units = 0;
      bool ok = true;
      for (int i = 0; ok && ring_take(&ring, i, ctl); ++i) {
        const KvUnit p(&ring, i);
        if (p.nq > 0 && is_q) {
          if (units > 0 && !(ok = mbar_wait(&bar_kvfree, (units - 1) & 1, ctl, kErrTimeoutMma))) break;
          mbar_expect_tx(&bar_kv, 2 * C::TILE);
          load_rows<D>(sK, &tm_k, &bar_kv, p.krow, p.head);
          load_rows<D>(sV, &tm_v, &bar_kv, p.krow, p.head);
        }
        if (p.nq == 0 && is_q) mbar_arrive(&ring.near);
        for (int u = 0; p.nq > 0 && u <= p.nq; ++u, ++e) {
          if (u == p.nq && is_q) mbar_arrive(&ring.near);
          const int st = e % depth;
          if (e >= depth && !(ok = mbar_wait(&empty[st], ((e / depth) - 1) & 1, ctl, kErrTimeoutMma))) break;
          own &= ~(1u << st);
          if (u == p.nq) {  // the way out
            mbar_arrive(&full[st]);
            mbar_arrive(&bar_out[(units & 1) * 2 + lane]);
            own |= 1u << st;
            continue;
          }
          uint64_t* bar = &full[st];
          if (p.ragged && u == p.nq - 1) {
            mbar_arrive(bar);  // (the ring's own phase passes on)
            bar = &bar_last[(i & 1) * 2 + lane];
            last_ph ^= 1u << (i & 1);
            own |= 1u << st;
          }
          mbar_expect_tx(bar, box);
          load_rows<D>(is_q ? sQ(st) : sDO(st), map, bar, p.head * G, p.row + u * TB);
        }
        if (p.nq > 0) ++units;
        if (ok) mbar_arrive(&ring.left[i & 1]);
      }
      if (is_q && units > 0) mbar_wait(&bar_kv, (units - 1) & 1, drain, kErrTimeoutTma);
      for (int u = e - depth > 0 ? e - depth : 0; u < e; ++u)
        if (!(own >> (u % depth) & 1u)) mbar_wait(&full[u % depth], (u / depth) & 1, drain, kErrTimeoutTma);
      for (int j = 0; j < 2; ++j) mbar_wait(&bar_last[j * 2 + lane], (last_ph >> j & 1u) ^ 1u, drain, kErrTimeoutTma);
    }
  } else if (warp == kMma) {
    // ----------------------------------------------------------------- MMA
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    constexpr uint32_t idesc_s = idesc_f16(kBN, kBM, BF, false, false);  // M = keys, N = query rows
    constexpr uint32_t idesc_g = idesc_f16(kBN, D, BF, false, true);     // M = keys, N = D
    RingAt<QST> q;  // the entry of S^T and dK to come
    RingAt<OST> o;
    uint32_t units = 0, tiles = 0, nc = 0, care_ph = 0;  // parities
    bool any = false, ok = true;
    for (int i = 0; ok; ++i) {
      if (!__all_sync(0xffffffffu, ring_take(&ring, i, ctl))) break;
      int nq, ragged;
      {
        const KvUnit p(&ring, i);
        nq = p.nq;
        ragged = p.ragged;
      }
      if (nq > 0) {
        const uint32_t ph = care_ph >> (i & 1) & 1u;
        if (ragged) care_ph ^= 1u << (i & 1);
        const int care_u = ragged ? nq - 1 : -1;
        auto q_ready = [&](int u) {
          const bool c = u == care_u;
          return warp_wait(c ? &bar_care[(i & 1) * 2] : &bar_qf[q.st], c ? ph : q.ph, ctl, kErrTimeoutTma);
        };
        auto o_ready = [&](int u) {
          const bool c = u == care_u;
          return warp_wait(c ? &bar_care[(i & 1) * 2 + 1] : &bar_of[o.st], c ? ph : o.ph, ctl, kErrTimeoutTma);
        };
        if (!(ok = warp_wait(&bar_kv, units, ctl, kErrTimeoutTma))) break;
        units ^= 1u;
#pragma unroll 1
        for (int u = -1; u < nq; ++u) {
          const int sq = q.st, so = o.st;
          const bool next = u + 1 < nq;
          if (u >= 0) {
            q.step();
            o.step();
          }
          if (next) {
            if (any && !(ok = warp_wait(&bar_consumed, nc, ctl, kErrTimeoutSoftmax))) break;
            nc ^= any ? 1u : 0u;
            any = true;
            if (!(ok = q_ready(u + 1))) break;
            tc_fence_after();
            mma_abT<D>(tmem + C::COL_A, smem_u32(sK), smem_u32(sQ(q.st)), idesc_s);  // S^T = K Q^T
            commit_el(&bar_s);
          }
          if (u >= 0) {
            if (!(ok = warp_wait(&bar_ds[0], tiles, ctl, kErrTimeoutSoftmax))) break;
            tc_fence_after();
            mma_tY_il_g<0>(tmem + C::COL_DV, tmem + C::COL_B, smem_u32(sDO(so)), idesc_g, u > 0);
            mma_tY_il_g<0>(tmem + C::COL_DK, tmem + C::COL_B + 16, smem_u32(sQ(sq)), idesc_g, u > 0);
            if (!(ok = warp_wait(&bar_ds[1], tiles, ctl, kErrTimeoutSoftmax))) break;
            tiles ^= 1u;
            tc_fence_after();
            mma_tY_il_g<1>(tmem + C::COL_DV, tmem + C::COL_B, smem_u32(sDO(so)), idesc_g, true);
            commit_el(&bar_oe[so]);
            mma_tY_il_g<1>(tmem + C::COL_DK, tmem + C::COL_B + 16, smem_u32(sQ(sq)), idesc_g, true);
            commit_el(&bar_qe[sq]);
          }
          if (next) {
            if (!(ok = o_ready(u + 1))) break;
            tc_fence_after();
            mma_abT<D>(tmem + C::COL_B, smem_u32(sV), smem_u32(sDO(o.st)), idesc_s);  // dP^T = V dO^T
            commit_el(&bar_dp);
            if (u + 2 == nq) commit_el(&bar_kvfree);  // nothing reads K and V any more
          }
        }
        if (!ok) break;
        commit_el(&bar_done);
        q.step();  // the entries of dK and dV
        o.step();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.left[i & 1]);
    }
  } else if (warp >= kCare) {
    // ------------------------------ units ahead; rows behind the tokens
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == kCare) {
      RingAsker asker;
      int qs = 0, os = 0;  // slots of the unit's first entries
      uint32_t ph = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        if (!__all_sync(0xffffffffu, ring_take(&ring, i, ctl))) break;
        const KvUnit p(&ring, i);
        if (p.nq > 0) {
          if (p.ragged) {
            const int rows = (p.left - (p.nq - 1) * TB) * G;
            for (int x = 0; x < 2; ++x) {
              ok = warp_wait(&bar_last[(i & 1) * 2 + x], ph >> (i & 1) & 1u, ctl, kErrTimeoutTma);
              if (!ok) break;
              zero_tile_rows<D / 64>(x ? sDO((os + p.nq - 1) % OST) : sQ((qs + p.nq - 1) % QST), rows, lane);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bar_care[(i & 1) * 2 + x]);
            }
            if (!ok) break;
            ph ^= 1u << (i & 1);
          }
          qs = (qs + p.nq + 1) % QST;
          os = (os + p.nq + 1) % OST;
        }
        if (asks)
          ok = asker.pass(&ring, args, list, i, ctl,
                          [&](const PackedUnit& u, int4(&words)[4]) { make_kv_unit(u, TB, words); });
        ok = __all_sync(0xffffffffu, ok);
      }
      if (asks) asker.drain(&ring, drain);
    }
  } else {
    // ------------------------------------------- key-row softmax gradient
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int hc = warp >> 2;  // half of the query tile's rows: columns [64 hc, 64 hc + 64)
    const int cb = 64 * hc;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const bool serves = threadIdx.x == 0;  // stores dK and dV
    // L and delta of the half's 64 rows, one value a thread; rows of no token read
    // L = +inf (P = 0) and delta = 0
    const int ld_arr = (threadIdx.x & 127) >> 6;  // 0: L, 1: delta
    const int ld_col = threadIdx.x & 63;
    const int ld_tok = static_cast<int>(args.g_div.div(cb + ld_col)), ld_head = cb + ld_col - ld_tok * G;
    const int m = lane & 3;
    const int kl = 32 * (warp & 3) + (lane >> 2);  // the thread's first key of the tile (then + 8, + 16, + 24)
    const int r = threadIdx.x & 127;
    uint32_t tiles = 0, units = 0;  // so far (tiles with any tokens' units)
    RingAt<QST> q;
    RingAt<OST> o;
    int lent_q = -1, lent_o = -1;  // slots that stores still read
    auto give_back = [&] {
      if (lent_q >= 0) {
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        mbar_arrive(&bar_qe[lent_q]);
        mbar_arrive(&bar_oe[lent_o]);
        lent_q = -1;
      }
    };
    bool ok = true;
    for (int i = 0; ok; ++i) {
      if (!__all_sync(0xffffffffu, ring_take(&ring, i, ctl))) break;
      const KvUnit p(&ring, i);
      const int nq = p.nq;
      auto grad = [&](void* to, long long st, long long sh) {
        return static_cast<T*>(to) + p.head * sh + static_cast<long long>(p.krow) * st;
      };
      if (nq == 0) {  // keys that no query sees
        T *dk = grad(args.dk, args.dk_t, args.dk_h), *dv = grad(args.dv, args.dv_t, args.dv_h);
        zero_rows(min(p.n, kBN), args.dg, [&](int j) -> void* { return dk + j * args.dk_t; });
        zero_rows(min(p.n, kBN), args.dg, [&](int j) -> void* { return dv + j * args.dv_t; });
        if (serves) give_back();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ring.left[i & 1]);
        continue;
      }
      const float* ld_base = (ld_arr ? args.delta : args.lse) +
                             (static_cast<size_t>(p.row) + ld_tok) * args.shape.Hq + p.head * G + ld_head;
      auto ld_fetch = [&](int u) -> float {
        if (ld_tok >= TB || u * TB + ld_tok >= p.left) return ld_arr ? 0.f : INFINITY;
        return __ldg(ld_base + static_cast<size_t>(u) * TB * args.shape.Hq);
      };
      auto ld_slot = [&](uint32_t c) { return sLD + ((c & 1) * 2 + hc) * 128; };
      // (every warp is past the unit before: its last barrier)
      ld_slot(tiles)[ld_arr * 64 + ld_col] = ld_fetch(0);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_pub[(tiles & 1) * 2 + hc]);
      for (int u = 0; u < nq; ++u, ++tiles) {
        const float pre = (u + 1 < nq) ? ld_fetch(u + 1) : 0.f;
        if (!(ok = warp_wait(&bar_s, tiles & 1, ctl, kErrTimeoutMma))) break;
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
        if (!(ok = warp_wait(&bar_pub[(tiles & 1) * 2 + hc], (tiles >> 1) & 1, ctl, kErrTimeoutSoftmax))) break;
        const float* sL = ld_slot(tiles) + 2 * m;
        const float* sD = sL + 64;
        const float2 sc2 = make_float2(args.scale_log2, args.scale_log2);
        float pr[64];
#pragma unroll
        for (int jj = 0; jj < 8; ++jj) {
          const float2 l2 = *reinterpret_cast<const float2*>(sL + 8 * jj);
          const float2 nl = fmul2(l2, make_float2(-kLog2e, -kLog2e));
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int x = 32 * g + 4 * jj;
            const float2 y0 = ffma2(make_float2(__uint_as_float(sv[x]), __uint_as_float(sv[x + 1])), sc2, nl);
            const float2 y1 = ffma2(make_float2(__uint_as_float(sv[x + 2]), __uint_as_float(sv[x + 3])), sc2, nl);
            pr[x + 0] = ex2(y0.x);
            pr[x + 1] = ex2(y0.y);
            pr[x + 2] = ex2(y1.x);
            pr[x + 3] = ex2(y1.y);
          }
        }
        // key k of the tile is seen from token off + k on: column q (token u TB + q / G)
        // is masked iff q < (off + k - u TB) G
        if (p.causal && p.off + kBN - 1 > u * TB) {
          int lo[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            lo[x] = min(max(p.off + kl + 8 * x - u * TB, 0), kBM) * G - cb - 2 * m;  // (past the tile's end: everything)
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int jj = 0; jj < 8; ++jj)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (8 * jj + (e & 1) < lo[2 * g + (e >> 1)]) pr[32 * g + 4 * jj + e] = 0.f;
        }
        if (!(ok = warp_wait(&bar_dp, tiles & 1, ctl, kErrTimeoutMma))) break;
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
              const int x = 32 * g + 4 * (4 * c + jq);
              const int di = 16 * g + 4 * jq;
              pp[2 * jq] = pack2<BF>(pr[x], pr[x + 1]);
              pp[2 * jq + 1] = pack2<BF>(pr[x + 2], pr[x + 3]);
              const float2 s0 = fmul2(make_float2(pr[x], pr[x + 1]),
                                      fadd2(make_float2(__uint_as_float(dp[di]), __uint_as_float(dp[di + 1])), nd2[jq]));
              const float2 s1 =
                  fmul2(make_float2(pr[x + 2], pr[x + 3]),
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
        if (u == 0 && serves) give_back();
        if (u + 1 < nq) {  // every warp of the half is past tile u - 1, the buffer's previous tile
          ld_slot(tiles + 1)[ld_arr * 64 + ld_col] = pre;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_pub[((tiles + 1) & 1) * 2 + hc]);
        }
        q.step();
        o.step();
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      if (!(ok = warp_wait(&bar_done, units & 1, ctl, kErrTimeoutMma) &&
                 warp_wait(&bar_out[(units & 1) * 2], (units >> 1) & 1, ctl, kErrTimeoutMma) &&
                 warp_wait(&bar_out[(units & 1) * 2 + 1], (units >> 1) & 1, ctl, kErrTimeoutMma)))
        break;
      ++units;
      tc_fence_after();
      // dV staged in dO's ring, dK (x sm_scale) in Q's
#pragma unroll
      for (int a = 0; a < 2; ++a) {
#pragma unroll
        for (int cc = 0; cc < D / 64; ++cc) {
          const int c = hc * (D / 64) + cc;
          uint32_t v[32];
          tmem_ld_x32(lane_addr + (a == 0 ? C::COL_DV : C::COL_DK) + 32 * c, v);
          tmem_ld_wait(v);
          stage_row_chunk_sw128<BF>(smem_u32(a == 0 ? sDO(o.st) : sQ(q.st)), r, c, v, a ? args.sm_scale : 1.f);
        }
      }
      tc_fence_before();
      fence_proxy_async_smem();
      named_bar_sync(1, kRowWarps * 32);
      const bool whole = p.n >= kBN, refill = TB * G < kBM;
      if (whole) {
        if (serves) {
#pragma unroll
          for (int kb = 0; kb < D / 64; ++kb) {
            tma_store_3d(&tm_dv, sDO(o.st) + kb * (kBM * 128), kb * 64, p.krow, p.head);
            tma_store_3d(&tm_dk, sQ(q.st) + kb * (kBM * 128), kb * 64, p.krow, p.head);
          }
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          lent_q = q.st;
          lent_o = o.st;
        }
      } else {  // the rows behind the keys are another sequence's
        T *dk = grad(args.dk, args.dk_t, args.dk_h), *dv = grad(args.dv, args.dv_t, args.dv_h);
        copy_tile_rows(sDO(o.st), args.dg, threadIdx.x, kRowWarps * 32, p.n,
                       [&](int j) -> void* { return dv + j * args.dv_t; });
        copy_tile_rows(sQ(q.st), args.dg, threadIdx.x, kRowWarps * 32, p.n,
                       [&](int j) -> void* { return dk + j * args.dk_t; });
      }
      if (!whole || refill) {
        // the slots go back at once; rows that no box fills are zeros again
        if (whole && serves) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        named_bar_sync(1, kRowWarps * 32);
        if (refill) {
          if (warp < 2) zero_tile_rows<D / 64>(warp ? sDO(o.st) : sQ(q.st), TB * G, lane);
          fence_proxy_async_smem();
          named_bar_sync(1, kRowWarps * 32);
        }
        if (serves) {
          mbar_arrive(&bar_qe[q.st]);
          mbar_arrive(&bar_oe[o.st]);
          lent_q = -1;
        }
      }
      q.step();
      o.step();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.left[i & 1]);
    }
    if (serves) {
      give_back();
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
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
