// The plan of packed attention: every tile of every sequence, the longest
// first, so that blocks in launch order finish at about the same time.
//
// One block per kind of tile (forward pairs, dQ tiles, dK/dV tiles): checks the
// offsets, counts the tiles by length in 1024 bins, and writes them in order of
// the bins.  Tiles of one bin may come in any order; no result depends on it.
//
// Latency is all it costs.  The tiles of 1024 sequences at a time make one line that the
// threads share, whatever the lengths: 4096 sequences of 16 tokens (8 / 8 heads) take 22 us (a
// warp a sequence took 177), 1024 of 300 (32 / 8) 27 (47), three of 12000 6.7 (8.5), one token 4.6 (4.0).
// Tiles of one bin within a warp are counted by one atomic: those of short sequences are all alike.
#include "launch.h"
#include "packed.cuh"

namespace ta {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBins = 1024;

struct Seq {
  int q0, nq, k0, nk;
};

__device__ __forceinline__ int seq_units(const PackedShape& p, int kind, const Seq& s) {
  if (kind == kPackedDkdv) return (s.nk + kBN - 1) / kBN;
  const int per = kind == kPackedFwd ? 2 * p.TB : p.TB;
  return (s.nq + per - 1) / per;
}

// Unit i of a sequence and its length in tiles of the other side.
__device__ __forceinline__ int make_unit(const PackedShape& p, int kind, const Seq& s, int i, PackedUnit* u) {
  const int P = s.nk - s.nq;
  *u = PackedUnit{};
  if (kind == kPackedDkdv) {
    const int k0 = i * kBN;
    int first = 0;
    if (p.causal) first = min(max(k0 - P, 0), s.nq);
    u->krow = s.k0 + k0;
    u->n = s.nk - k0;
    u->row = s.q0 + first;
    u->left = s.nq - first;
    u->off = k0 - P - first;
    return (u->left + p.TB - 1) / p.TB;
  }
  const int per = kind == kPackedFwd ? 2 * p.TB : p.TB;
  const int t0 = i * per;
  u->row = s.q0 + t0;
  u->left = s.nq - t0;
  u->krow = s.k0;
  u->n = s.nk;
  u->off = t0 + P;
  return packed_key_tiles(min(per, u->left), u->off, s.nk, p.causal);
}

__global__ void __launch_bounds__(kPlanThreads) packed_plan_kernel(const PackedShape p, const int* cu_q, const int* cu_k,
                                                                   uint8_t* plan, uint32_t* err) {
  __shared__ int hist[kBins], before[kPlanThreads], warps[32], longest, units;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kind = blockIdx.x;
  PackedHeader* h = reinterpret_cast<PackedHeader*>(plan);
  PackedUnit* list = reinterpret_cast<PackedUnit*>(plan + p.first(kind));
  auto seq = [&](int b) {
    Seq s;
    s.q0 = __ldg(cu_q + b);
    s.nq = __ldg(cu_q + b + 1) - s.q0;
    s.k0 = __ldg(cu_k + b);
    s.nk = __ldg(cu_k + b + 1) - s.k0;
    return s;
  };
  // sums of the threads' values before a thread's; warps[31]: of all
  auto exclusive = [&](int v) {
    int upto = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += x;
    }
    if (lane == 31) warps[warp] = upto;
    __syncthreads();
    if (warp == 0) {
      int w = warps[lane];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += x;
      }
      warps[lane] = w;
    }
    __syncthreads();
    return upto - v + (warp > 0 ? warps[warp - 1] : 0);
  };
  hist[tid] = 0;
  if (tid == 0) longest = 1;
  bool bad = false;
  for (int b = tid; b < p.B; b += kPlanThreads) {
    const int q0 = __ldg(cu_q + b), q1 = __ldg(cu_q + b + 1), k0 = __ldg(cu_k + b), k1 = __ldg(cu_k + b + 1);
    bad |= q0 < 0 || q1 < q0 || q1 > p.total_q || k0 < 0 || k1 < k0 || k1 > p.total_k;
  }
  bad = __syncthreads_or(bad);
  if (bad) {  // no unit at all
    if (tid == 0) {
      cache_error(err);
      h->count[kind] = 0;
    }
  } else {
    int top = 0;
    PackedUnit u;
    for (int b = tid; b < p.B; b += kPlanThreads) {
      const Seq s = seq(b);
      const int n = seq_units(p, kind, s);
      if (n > 0) top = max(top, make_unit(p, kind, s, kind == kPackedDkdv ? 0 : n - 1, &u));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) atomicMax(&longest, top);
    __syncthreads();
    const int most = longest;
    // the longest in bin 0
    auto bin = [&](int cost) { return kBins - 1 - static_cast<int>(static_cast<long long>(cost) * (kBins - 1) / most); };
    // f(unit, its bin, whether there is one) for every unit, by whole warps
    auto each_unit = [&](bool again, auto f) {
      for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int count = min(p.B - b0, kPlanThreads);
        if (!again || p.B > kPlanThreads) {
          const int n = tid < count ? seq_units(p, kind, seq(b0 + tid)) : 0;
          __syncthreads();  // the readers of the sequences before
          const int first = exclusive(n);
          before[tid] = first;
          if (tid == kPlanThreads - 1) units = first + n;
          __syncthreads();
        }
        const int all = units;
        for (int x0 = warp * 32; x0 < all; x0 += kPlanThreads) {
          const int x = x0 + lane;
          const bool there = x < all;
          int cost = 0;
          if (there) {
            int lo = 0, hi = count;  // before[lo] <= x < before[hi]
            while (hi - lo > 1) {
              const int mid = (lo + hi) >> 1;
              if (before[mid] <= x) lo = mid;
              else hi = mid;
            }
            cost = make_unit(p, kind, seq(b0 + lo), x - before[lo], &u);
          }
          f(u, there ? bin(cost) : -1, there);
        }
      }
    };
    each_unit(false, [&](const PackedUnit&, int at, bool there) {
      const uint32_t same = __match_any_sync(0xffffffffu, at);
      if (there && lane == __ffs(same) - 1) atomicAdd(&hist[at], __popc(same));
    });
    __syncthreads();
    const int start = exclusive(hist[tid]);
    hist[tid] = start;
    if (tid == 0) h->count[kind] = warps[31];
    __syncthreads();
    each_unit(true, [&](const PackedUnit& w, int b, bool there) {
      const uint32_t same = __match_any_sync(0xffffffffu, b);
      const int leader = __ffs(same) - 1;
      int at = 0;
      if (there && lane == leader) at = atomicAdd(&hist[b], __popc(same));
      at = __shfl_sync(0xffffffffu, at, leader) + __popc(same & ((1u << lane) - 1));
      if (!there) return;
      int4* dst = reinterpret_cast<int4*>(list + at);
      dst[0] = make_int4(w.row, w.left, w.krow, w.n);
      dst[1] = make_int4(w.off, 0, 0, 0);
    });
  }
  if (kind == 0 && tid == 0) {
    h->magic = kPackedMagic;
    h->B = p.B;
    h->total_q = p.total_q;
    h->total_k = p.total_k;
    h->Hq = p.Hq;
    h->Hkv = p.Hkv;
    h->causal = p.causal;
  }
}

}  // namespace

cudaError_t launch_packed_plan(const PackedShape& p, const int* cu_q, const int* cu_k, void* plan, uint32_t* err,
                               cudaStream_t s) {
  packed_plan_kernel<<<kPackedKinds, kPlanThreads, 0, s>>>(p, cu_q, cu_k, static_cast<uint8_t*>(plan), err);
  return cudaGetLastError();
}

}  // namespace ta

TA_GUARD_ACCESSOR(packed_plan)
