// The plan of packed attention: every tile of every sequence, the longest
// first, so that blocks in launch order finish at about the same time.
//
// One block per kind of tile (forward pairs, dQ tiles, dK/dV tiles): checks the
// offsets, counts the tiles by length in 1024 bins, and writes them in order of
// the bins.  Tiles of one bin may come in any order; no result depends on it.
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
  __shared__ int hist[kBins], warps[32], longest;
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
    for (int b = warp; b < p.B; b += kPlanThreads / 32) {
      const Seq s = seq(b);
      const int n = seq_units(p, kind, s);
      for (int i = lane; i < n; i += 32) atomicAdd(&hist[bin(make_unit(p, kind, s, i, &u))], 1);
    }
    __syncthreads();
    // exclusive sums of the bins
    const int mine = hist[tid];
    int upto = mine;
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
    hist[tid] = upto - mine + (warp > 0 ? warps[warp - 1] : 0);
    if (tid == 0) h->count[kind] = warps[31];
    __syncthreads();
    for (int b = warp; b < p.B; b += kPlanThreads / 32) {
      const Seq s = seq(b);
      const int n = seq_units(p, kind, s);
      for (int i = lane; i < n; i += 32) {
        const int at = atomicAdd(&hist[bin(make_unit(p, kind, s, i, &u))], 1);
        int4* dst = reinterpret_cast<int4*>(list + at);
        dst[0] = make_int4(u.row, u.left, u.krow, u.n);
        dst[1] = make_int4(u.off, 0, 0, 0);
      }
    }
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
