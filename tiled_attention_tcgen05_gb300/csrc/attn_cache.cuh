// Work division of the attention over a cache, shared by its kernels.
//
// A unit is up to ROWS query rows of one sequence and key head: the G query
// heads that share the key head, times the new tokens (row r is token r / G of
// head r % G).  A unit needs the key tiles (TK keys) up to the last key its last
// token can see.  All units' tiles, in the order sequence, key head, row tile,
// make one line; block i of n takes the places cut(i) .. cut(i + 1), so that
// sequences of any mix of lengths keep every SM busy to the end.  A unit inside
// one block is finished there; a unit that block borders cut leaves one
// partial state per block (the block's first piece in slot 0 of its two, a
// later one in slot 1), and a second kernel joins them in a fixed order.  The
// cut depends on the lengths alone, never on timing.
#pragma once
#include "cache.cuh"
#include "launch.h"

namespace ta {

struct Seq {
  int kv, q, nrt;
  long long per_head, all;  // tiles of one key head, of the sequence
};

template <int ROWS, int TK>
struct Line {
  // key tiles of row tile rt
  static __device__ __forceinline__ int tiles(const CacheAttnArgs& a, const Seq& s, int rt) {
    int end = s.kv;
    if (!a.tree) {
      const int last = min(s.q - 1, static_cast<int>(a.g_div.div(min((rt + 1) * ROWS, s.q * a.G) - 1)));
      end = s.kv - s.q + last + 1;
    }
    return (end + TK - 1) / TK;
  }
  static __device__ __forceinline__ Seq seq(const CacheArgs& c, const CacheAttnArgs& a, int b) {
    const SeqLens n = cache_lens(c, b);
    Seq s;
    s.kv = n.kv;
    s.q = n.q;
    s.nrt = (n.q * a.G + ROWS - 1) / ROWS;
    s.per_head = 0;
    if (a.tree || s.nrt <= 1) {
      if (s.nrt > 0) s.per_head = static_cast<long long>(s.nrt) * tiles(a, s, s.nrt - 1);
    } else {
      for (int rt = 0; rt < s.nrt; ++rt) s.per_head += tiles(a, s, rt);
    }
    s.all = s.per_head * c.Hkv;
    return s;
  }

  struct Shared {
    long long warp_sum[32];
    int b;
    long long start;  // first place of sequence b
  };
  // Length of the line: every thread adds up a run of sequences (mine, with
  // `before` it on the line), a scan over the block joins the runs.
  template <int THREADS>
  static __device__ __forceinline__ long long length(const CacheArgs& c, const CacheAttnArgs& a, Shared& sh,
                                                     long long* mine, long long* before) {
    const int per = (c.B + THREADS - 1) / THREADS;
    const int b0 = min(static_cast<long long>(c.B), static_cast<long long>(threadIdx.x) * per), b1 = min(c.B - b0, per) + b0;
    long long sum = 0;
    for (int b = b0; b < b1; ++b) sum += seq(c, a, b).all;
    long long inc = sum;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, inc, s);
      if ((threadIdx.x & 31) >= s) inc += o;
    }
    if ((threadIdx.x & 31) == 31) sh.warp_sum[threadIdx.x >> 5] = inc;
    __syncthreads();
    long long total = 0, pre = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      const long long v = sh.warp_sum[w];
      if (w < static_cast<int>(threadIdx.x >> 5)) pre += v;
      total += v;
    }
    *mine = sum;
    *before = pre + inc - sum;
    return total;
  }

  // Place on the line: sequence b, head h, row tile rt, key tile t.
  struct Cursor {
    int b, h, rt, t;
    int ntiles;  // of this unit
    Seq s;
  };
  // Cursor at place x (below the line's length, the same in all threads).
  template <int THREADS>
  static __device__ __forceinline__ void find(const CacheArgs& c, const CacheAttnArgs& a, Shared& sh, long long x,
                                              long long mine, long long before, Cursor& u) {
    if (x >= before && x < before + mine) {
      const int per = (c.B + THREADS - 1) / THREADS;
      int b = threadIdx.x * per;
      long long at = before;
      while (true) {
        const long long n = seq(c, a, b).all;
        if (x < at + n) break;
        at += n;
        ++b;
      }
      sh.b = b;
      sh.start = at;
    }
    __syncthreads();
    u.b = sh.b;
    u.s = seq(c, a, u.b);
    const long long in = x - sh.start;
    u.h = u.s.all <= 0xffffffffll ? static_cast<int>(static_cast<uint32_t>(in) / static_cast<uint32_t>(u.s.per_head))
                                  : static_cast<int>(in / u.s.per_head);
    long long rest = in - u.h * u.s.per_head;
    u.rt = 0;
    u.ntiles = tiles(a, u.s, 0);
    while (rest >= u.ntiles) {
      rest -= u.ntiles;
      u.ntiles = tiles(a, u.s, ++u.rt);
    }
    u.t = static_cast<int>(rest);
  }
  // To the first tile of the next unit (b == B behind the last).
  static __device__ __forceinline__ void next_unit(const CacheArgs& c, const CacheAttnArgs& a, Cursor& u) {
    u.t = 0;
    if (++u.rt >= u.s.nrt) {
      u.rt = 0;
      if (++u.h >= c.Hkv) {
        u.h = 0;
        do {
          if (++u.b >= c.B) return;
          u.s = seq(c, a, u.b);
        } while (u.s.all == 0);
      }
    }
    u.ntiles = tiles(a, u.s, u.rt);
  }
  static __device__ __forceinline__ void next_tile(const CacheArgs& c, const CacheAttnArgs& a, Cursor& u) {
    if (++u.t >= u.ntiles) next_unit(c, a, u);
  }
};

// Block i's first place when the line of `len` is cut for N blocks (a constant:
// a 64-bit division by a variable takes about as long as a load), and the block
// that holds place y: cut(b) <= y < cut(b + 1).
template <int N>
__device__ __forceinline__ long long cut(long long len, int i) {
  return static_cast<long long>(static_cast<unsigned long long>(len * i) / N);
}
template <int N>
__device__ __forceinline__ int block_of(long long len, long long y) {
  return static_cast<int>(((y + 1) * N - 1) / len);
}

// A factor <= 1 for accumulators whose row got a larger maximum, kept above
// zero: an infinity that the row has seen stays one.  To finite accumulators
// 2^-126 is what a weight that small, flushed to zero, is.
__device__ __forceinline__ float keep_infinite(float f) { return fmaxf(f, 1.1754943508222875e-38f); }

// 8-bit caches.  A value's scale sv is part of the exponent of its weight,
// p = 2^(t - m) with t = s + log2 sv, and the softmax sum is that of the bare
// scores s, l = sum 2^(s - m + kSumUp).  p can be far too small for fp32 where
// 2^(s - m) decides the sum (a row of zeros, of scale 2^-60, beside values of
// 2^80), so that p / sv would not do: from h = 2^((t - m) / 2), p = h^2 and the
// sum's part is (h 2^((kSumUp - log2 sv) / 2))^2, which vanishes only where it does not
// count.  With kSumUp a part lies below 2^92 and those of keys with t near m
// above 2^-98 (scales 2^-60 to 2^122): 2^31 of them fit.  Two packed products a
// pair of keys more; a branch for such tiles alone cost more (48 rows of D = 64
// over int8, 16 x 4096: 76.5 us; this 75.5; the plain quotient 70.7).
constexpr float kSumUp = 24.f;
// A sum whose reference rises by -by.  The sum may be far above 1, so that 2^by
// alone would be zero where the product counts.
__device__ __forceinline__ float lower_sum(float l, float by) {
  const float h = ex2(0.5f * by);
  return l * h * h;
}
// 1 / sum and L of a row with reference m (0 and -inf for a row that saw
// nothing; a NaN sum stays one where no score was a number).
template <int CT>
__device__ __forceinline__ float sum_norm(float l) {
  return l == 0.f ? 0.f : (CT == kCache16 ? 1.f : 16777216.f) / l;  // 2^kSumUp
}
template <int CT>
__device__ __forceinline__ float row_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m == -INFINITY ? l : (m + (CT == kCache16 ? lg2(l) : lg2(l) - kSumUp)) * kLn2);
}

// ----------------------------------------------------------------- joining
// The join kernel is launched while the main kernel runs (programmatic
// dependent launch) and waits for its end before it reads anything.
__device__ __forceinline__ void let_dependents_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_main_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// What the join needs to know about the unit that block i's first border cuts,
// where this is the first border inside the unit; written by block i of the
// main kernel in every call (parts = 0 otherwise), so that the join does not
// look the unit up again.
struct __align__(16) CutUnit {
  int b, h, rt, parts;  // unit; blocks first .. first + parts - 1 hold its pieces
  int first;
  int first_slot;       // the first block's slot (the others': 0)
  int q;                // the sequence's new tokens
  int sparse;           // fewer tiles than blocks: some of the blocks are empty
  long long len, pad2;
};

// Block i's record; `u` is its first place, len the line's length (0: none).
template <int N, typename Cursor>
__device__ __forceinline__ void write_cut(CutUnit* out, long long len, int i, long long x0, long long x1,
                                          const Cursor* u) {
  CutUnit r = {};
  if (x0 < x1 && i > 0 && u->t > 0) {
    // the block that holds the place before starts at or before the unit?
    const long long u0 = x0 - u->t;
    const int first = block_of<N>(len, x0 - 1);
    const long long before = cut<N>(len, first);
    if (before <= u0) {
      r.b = u->b, r.h = u->h, r.rt = u->rt, r.q = u->s.q;
      r.first = first;
      r.parts = block_of<N>(len, u0 + u->ntiles - 1) - first + 1;
      r.first_slot = before < u0 ? 1 : 0;
      r.sparse = len < N;
      r.len = len;
    }
  }
  out[i] = r;
}
// Slot of part k, -1 for a block without a piece.
template <int N>
__device__ __forceinline__ int part_slot(const CutUnit& r, int k) {
  const int b = r.first + k;
  if (r.sparse && cut<N>(r.len, b) == cut<N>(r.len, b + 1)) return -1;
  return b * 2 + (k == 0 ? r.first_slot : 0);
}

// Launches the join kernel behind the main one.
template <typename K, typename... Args>
inline cudaError_t launch_join(K kern, dim3 grid, int threads, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace ta
