// Attention of sequences packed one behind the other, with shared key heads:
// the plan (which tiles there are), the geometry of a tile, and the helpers of
// the kernels in packed_fwd.cu and packed_bwd.cu.
//
// A tile of 128 query rows holds TB = 128 / G consecutive tokens (rounded down) with
// the G query heads of one key head, token by token: row r is token r / G, head
// r % G.  All of its rows read the same keys, so a short sequence fills a tile
// G times better than with a tile per head, and the key side of the backward
// sums over the heads by walking rows.  TMA loads such a tile as a box of
// 64 columns x G heads x TB tokens.
#pragma once
#include <atomic>
#include <cuda.h>
#include <cuda_runtime.h>

#include "bwd_common.cuh"
#include "cache.cuh"
#include "common.cuh"

namespace ta {

// One CTA's work for one key head.  Query side (forward: two tiles, dQ: one):
// row, left: first token's row and the tokens from it to the sequence's end;
// krow, n: first key's row and the number of keys; off: last key the first
// token sees (causal).  Key side: krow, n: first key of the tile and the keys from it
// on; row, left: first token that sees any of it and the tokens from there
// on; off: such token (counted from it) from which the tile's first key is seen.
struct PackedUnit {
  int row, left, krow, n, off, pad[3];
};
static_assert(sizeof(PackedUnit) == 32, "two 16-byte loads");

enum PackedKind : int { kPackedFwd = 0, kPackedDq = 1, kPackedDkdv = 2, kPackedKinds = 3 };

constexpr int kPackedMagic = 0x70a7c4ed;

// Start of the plan's memory; the lists of units follow, kind by kind.
struct PackedHeader {
  int magic, B, total_q, total_k, Hq, Hkv, causal;
  int count[kPackedKinds];
  int pad[6];
};
static_assert(sizeof(PackedHeader) == 64, "units start on a 64-byte boundary");

struct PackedShape {
  int B, total_q, total_k, Hq, Hkv, G, TB, causal;
  // units of a kind at most: sum of ceil(len / size) <= total / size + B
  __host__ __device__ long long bound(int kind) const {
    if (kind == kPackedFwd) return total_q / (2 * TB) + B;
    return kind == kPackedDq ? total_q / TB + B : total_k / kBN + B;
  }
  __host__ __device__ size_t first(int kind) const {  // byte offset of a kind's list
    size_t at = sizeof(PackedHeader);
    for (int i = 0; i < kind; ++i) at += static_cast<size_t>(bound(i)) * sizeof(PackedUnit);
    return at;
  }
};

struct PackedArgs {
  const uint8_t* plan;
  PackedShape shape;
  FastDiv hkv_div, g_div;
  const void* v;        // [total_k, Hkv, D], element strides vt, vh
  long long vt, vh;
  void *o, *dq, *dk, *dv;  // element strides (token, head)
  long long o_t, o_h, dq_t, dq_h, dk_t, dk_h, dv_t, dv_h;
  float* lse;           // [total_q, Hq]
  float* delta;         // [total_q, Hq]
  float scale_log2, sm_scale;
  int dg;               // head dimension of the tensors in memory
  uint32_t* err;
  uint64_t timeout_ns;
};

// q, o, dO, dq: boxes of TB tokens x G heads; k, v, dk, dv: 128 rows of a head.
struct PackedMaps {
  CUtensorMap q, k, v, o, dO, dq, dk, dv;
};

cudaError_t launch_packed_plan(const PackedShape& p, const int* cu_q, const int* cu_k, void* plan, uint32_t* err,
                               cudaStream_t s);
cudaError_t launch_packed_fwd(bool bf16, int D, const PackedMaps& m, const PackedArgs& a, cudaStream_t s);
cudaError_t launch_packed_dq(bool bf16, int D, const PackedMaps& m, const PackedArgs& a, cudaStream_t s);
cudaError_t launch_packed_dkdv(bool bf16, int D, const PackedMaps& m, const PackedArgs& a, cudaStream_t s);

#ifdef __CUDACC__
// What a block reads of the plan's header.  A plan that was not made for these
// sizes is recorded in the error word and has no units.
struct PackedList {
  const int4* units;
  uint32_t items;  // units x key heads; item i is unit i / Hkv, head i % Hkv
  int causal;
};
__device__ __forceinline__ PackedList packed_list(const PackedArgs& a, int kind) {
  const int4* h = reinterpret_cast<const int4*>(a.plan);
  const int4 h0 = __ldg(h), h1 = __ldg(h + 1), h2 = __ldg(h + 2);
  PackedList l;
  l.units = reinterpret_cast<const int4*>(a.plan + a.shape.first(kind));
  l.causal = h1.z;
  l.items = static_cast<uint32_t>(kind == kPackedFwd ? h1.w : kind == kPackedDq ? h2.x : h2.y) * a.shape.Hkv;
  if (h0.x != kPackedMagic || h0.y != a.shape.B || h0.z != a.shape.total_q || h0.w != a.shape.total_k ||
      h1.x != a.shape.Hq || h1.y != a.shape.Hkv) {
    if (threadIdx.x == 0 && blockIdx.x == 0) cache_error(a.err);
    l.items = 0;
  }
  return l;
}
// An item's unit (PackedUnit::pad[0]: causal, pad[1]: the key head).
__device__ __forceinline__ PackedUnit packed_item(const PackedArgs& a, const PackedList& l, uint32_t item) {
  const uint32_t i = a.hkv_div.div(item);
  const int4 x = __ldg(l.units + 2 * static_cast<size_t>(i)), y = __ldg(l.units + 2 * static_cast<size_t>(i) + 1);
  return PackedUnit{x.x, x.y, x.z, x.w, y.x, {l.causal, static_cast<int>(item - i * a.hkv_div.d), 0}};
}

// Key tiles that a tile of `tokens` tokens visits, the first of which sees keys up to off.
__host__ __device__ inline int packed_key_tiles(int tokens, int off, int n, int causal) {
  if (tokens <= 0) return 0;
  const int all = (n + kBN - 1) / kBN;
  if (!causal) return all;
  const long long last = static_cast<long long>(off) + tokens - 1;
  if (last < 0) return 0;
  const long long t = last / kBN + 1;
  return t < all ? static_cast<int>(t) : all;
}

// ------------------------------------------------------- one block, many units
// Shared memory, tensor memory and the rings stay set up from unit to unit, and the
// next unit's tiles arrive while a block works on the last one's: a block that has
// done its unit takes over that of a block that has not been launched yet
// (cluster launch control: the launch is cancelled and its block index handed
// over), so units go out one by one, the longest first.
// One warp asks for the next unit once a producer has asked for the last tile of this
// one (earlier, and a block would sit on a unit that another could start on), and
// passes it to the others through two slots; unit i is in slot i % 2, and is
// passed on only once every other role has left unit i - 2, so that no role is
// ever two units ahead of another.
struct UnitRing {
  uint64_t full[2], left[2], near, answered;
  uint4 answer;       // of the cancellation asked for
  int4 unit[2][4];    // words of the kernel's own, made by pass()'s `fill`; [3].w: 1: there is one
};

__device__ __forceinline__ void ring_init(UnitRing* r, int roles) {
  for (int i = 0; i < 2; ++i) {
    mbar_init(&r->full[i], 1);
    mbar_init(&r->left[i], roles);
  }
  mbar_init(&r->near, 1);
  mbar_init(&r->answered, 1);
}

// Asks for the next block index (one thread; the one before must have been answered).
__device__ __forceinline__ void ring_ask(UnitRing* r) {
  // the last answer has been read before the next is written
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  mbar_expect_tx(&r->answered, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(&r->answer)),
               "r"(smem_u32(&r->answered))
               : "memory");
}
// The block index handed over; false: there is none left, and no more may be asked for.
__device__ __forceinline__ bool ring_answer(const UnitRing* r, uint32_t* block) {
  uint32_t got, x;
  asm volatile(
      "{\n .reg .b128 a;\n .reg .pred p;\n ld.shared.b128 a, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n}\n"
      : "=r"(got), "=r"(x)
      : "r"(smem_u32(&r->answer))
      : "memory");
  *block = x;
  return got != 0;
}

// The asking thread's side.
struct RingAsker {
  uint32_t asks = 0;  // requests made
  bool more = true, open = false;  // there may be another unit; a request is unanswered
  __device__ __forceinline__ bool wait(UnitRing* r, const WaitCtl& ctl) {
    if (!mbar_wait(&r->answered, (asks - 1) & 1, ctl, kErrTimeoutOther)) return false;
    open = false;
    return true;
  }
  // In unit i: passes unit i + 1 on; fill(u, words) makes the slot's words of it.
  // False: a wait ran out.
  template <typename F>
  __device__ __forceinline__ bool pass(UnitRing* r, const PackedArgs& a, const PackedList& l, int i, const WaitCtl& ctl,
                                       F fill) {
    const int next = i + 1, s = next & 1;
    int4 words[4] = {};
    if (!mbar_wait(&r->near, i & 1, ctl, kErrTimeoutOther)) return false;
    if (more) {
      ring_ask(r);
      ++asks;
      open = true;
      if (!wait(r, ctl)) return false;
      uint32_t block;
      more = ring_answer(r, &block) && block < l.items;
      if (more) {
        fill(packed_item(a, l, block), words);
        words[3].w = 1;
      }
    }
    if (next >= 2 && !mbar_wait(&r->left[s], ((next >> 1) - 1) & 1, ctl, kErrTimeoutOther)) return false;
#pragma unroll
    for (int k = 0; k < 4; ++k) r->unit[s][k] = words[k];
    mbar_arrive(&r->full[s]);
    return true;
  }
  // An answer under way must land before the block's shared memory goes.
  __device__ __forceinline__ void drain(UnitRing* r, const WaitCtl& ctl) {
    if (open) wait(r, ctl);
  }
};

// Whether the block has a unit i (false, too, where a wait ran out).  Whoever was
// told so arrives on left[i % 2] when done with it.
__device__ __forceinline__ bool ring_take(UnitRing* r, int i, const WaitCtl& ctl) {
  if (i == 0) return true;
  const int s = i & 1;
  if (!mbar_wait(&r->full[s], ((i - 1) >> 1) & 1, ctl, kErrTimeoutOther)) return false;
  return r->unit[s][3].w != 0;
}
// Words k of unit i, until the role has left it.
__device__ __forceinline__ int4 ring_words(const UnitRing* r, int i, int k) {
  int4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "r"(smem_u32(&r->unit[i & 1][k])));
  return x;
}

// Rows [first, 128) of a 128-row tile of NB 64-column blocks set to zero by one
// warp, then made visible to the MMAs (whoever waits for the barrier the warp
// arrives on next).
template <int NB>
__device__ __forceinline__ void zero_tile_rows(uint8_t* tile, int first, int lane) {
  for (int kb = 0; kb < NB; ++kb)
    for (int i = first * 8 + lane; i < kBM * 8; i += 32)
      *reinterpret_cast<uint4*>(tile + kb * (kBM * 128) + i * 16) = make_uint4(0u, 0u, 0u, 0u);
}

// The first `rows` rows of a staged output tile (stage_row_chunk_sw128's layout) to
// memory, 16 bytes a thread and a row's pieces side by side; row(r) is where row r
// goes.  `n` threads (a multiple of 128), tid among them: a thread keeps to its piece, and
// its rows are a multiple of 8 apart, so that it stays in one column of the swizzle.  (Four
// rows at a time take longer: 384 against 342 us for 1024 sequences of 32, 16 / 16 heads of 64.)
template <typename F>
__device__ __forceinline__ void copy_tile_rows(const uint8_t* tile, int dg, int tid, int n, int rows, F row) {
  const int c = dg >> 3;  // 16-byte pieces of a row: 2, 4, 8 or 16
  const int sh = __ffs(c) - 1, j = tid & (c - 1), r0 = tid >> sh, step = n >> sh;
  const uint8_t* src = tile + (j >> 3) * (kBM * 128) + r0 * 128 + (((j & 7) ^ (r0 & 7)) << 4);
#pragma unroll 1
  for (int r = r0; r < rows; r += step, src += step * 128)
    static_cast<uint4*>(row(r))[j] = *reinterpret_cast<const uint4*>(src);
}
#endif

}  // namespace ta
