// cache_assign: pages, slots, positions and offsets of a step's tokens from the
// requests' lengths.
//
// Requests in order ask for pages and tokens; a prefix sum of each says who
// is served, and which entries of the stack of free pages are whose.  All
// of it is a few kilobytes, so latency is what it costs: one block of
// 1024 threads scans the requests, warps copy the page ids (one request
// each at a time), and the same block writes the tokens' slots where they are few.
// Otherwise a grid does, launched while the first kernel runs.
#include "assign.cuh"
#include "launch.h"
#include "pdl.cuh"

namespace ta {

namespace {

constexpr int kScan = 1024;

// Tokens up to which the scanning block writes the slots itself.
constexpr int kOneBlockTokens = 4096;

struct Asked {
  long long pages, tokens;
};

// Inclusive sums over the block's threads; *total those of all.
__device__ __forceinline__ Asked block_sums(Asked v, Asked* total) {
  __shared__ long long sp[32], st[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long p = __shfl_up_sync(0xffffffffu, v.pages, d), t = __shfl_up_sync(0xffffffffu, v.tokens, d);
    if (lane >= d) {
      v.pages += p;
      v.tokens += t;
    }
  }
  __syncthreads();  // the arrays' readers before
  if (lane == 31) {
    sp[warp] = v.pages;
    st[warp] = v.tokens;
  }
  __syncthreads();
  if (warp == 0) {
    long long p = sp[lane], t = st[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, p, d), b = __shfl_up_sync(0xffffffffu, t, d);
      if (lane >= d) {
        p += a;
        t += b;
      }
    }
    sp[lane] = p;
    st[lane] = t;
  }
  __syncthreads();
  if (warp > 0) {
    v.pages += sp[warp - 1];
    v.tokens += st[warp - 1];
  }
  *total = Asked{sp[31], st[31]};
  return v;
}

// A request as the call finds it.  Lengths that cannot be make it idle.
struct Request {
  int kv, add;  // add < 0: ended
  int held, need;
};
__device__ __forceinline__ Request request(const AssignArgs& a, int b) {
  Request r{0, 0, 0, 0};
  if (b >= a.B) return r;
  r.kv = __ldg(a.kv_lens + b);
  r.add = __ldg(a.new_lens + b);
  if (r.kv < 0 || r.kv > a.capacity || r.add < -1 || r.add > a.capacity - r.kv) {
    cache_error(a.err);
    r.add = 0;
    return r;
  }
  auto pages = [&](int n) { return n > 0 ? static_cast<int>(a.page.div(n - 1)) + 1 : 0; };
  r.held = pages(r.kv);
  r.need = r.add > 0 ? pages(r.kv + r.add) - r.held : 0;
  return r;
}

// Position and slot of token i; cu may lie in shared memory.
__device__ __forceinline__ void write_token(const AssignArgs& a, const int* cu, int i) {
  int pos = 0, slot = -1;
  if (i < cu[a.B]) {
    int lo = 0, hi = a.B;  // cu[lo] <= i < cu[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] <= i) lo = mid;
      else hi = mid;
    }
    pos = __ldg(a.kv_lens + lo) + (i - cu[lo]);
    const uint32_t col = a.page.div(pos);
    const int id = a.pages[static_cast<long long>(lo) * a.max_pages + col];
    if (static_cast<unsigned>(id) < static_cast<unsigned>(a.num_pages))
      slot = id * static_cast<int>(a.page.d) + (pos - static_cast<int>(col * a.page.d));
    else
      cache_error(a.err);
  }
  a.positions[i] = pos;
  a.slots[i] = slot;
}

__global__ void __launch_bounds__(kScan) assign_kernel(const AssignArgs a, bool tokens_too) {
  __shared__ long long first[kScan];  // a request's first entry of the stack
  __shared__ int at[kScan], num[kScan];  // its first column, and how many
  __shared__ int cu_s[kScan + 1];
  pdl_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int count = __ldg(a.free_count);
  if (count < 0 || count > a.num_pages) {
    if (tid == 0) cache_error(a.err);
    count = 0;
  }
  // ended requests' pages go on top of the stack, in order
  long long top = count;
  for (int b0 = 0; b0 < a.B; b0 += kScan) {
    const Request r = request(a, b0 + tid);
    const int back = r.add < 0 ? r.held : 0;
    if (!__syncthreads_or(back)) continue;
    Asked total;
    const Asked upto = block_sums(Asked{back, 0}, &total);
    first[tid] = top + upto.pages - back;
    num[tid] = back;
    __syncthreads();
    for (int k = warp; k < kScan && b0 + k < a.B; k += kScan / 32)
      for (int i = lane; i < num[k]; i += 32)
        if (first[k] + i < a.num_pages)
          a.free_ids[first[k] + i] = a.pages[static_cast<long long>(b0 + k) * a.max_pages + i];
    top += total.pages;
  }
  if (top > a.num_pages) {  // more pages came back than there are
    if (tid == 0) cache_error(a.err);
    top = a.num_pages;
  }
  Asked before{0, 0};
  long long taken = 0;
  int rows = 0;
  if (tid == 0) a.cu[0] = cu_s[0] = 0;
  for (int b0 = 0; b0 < a.B; b0 += kScan) {
    const int b = b0 + tid;
    const Request r = request(a, b);
    const int add = max(r.add, 0);
    Asked total;
    Asked upto = block_sums(Asked{r.need, add}, &total);
    upto.pages += before.pages;
    upto.tokens += before.tokens;
    before.pages += total.pages;
    before.tokens += total.tokens;
    const bool ok = (r.need == 0 || upto.pages <= top) && (add == 0 || upto.tokens <= a.total);
    const int q = ok ? add : 0;
    first[tid] = top - 1 - (upto.pages - r.need);
    at[tid] = r.held;
    num[tid] = ok ? r.need : 0;
    // who is served with pages is a prefix of those who ask for some
    const Asked served = block_sums(Asked{num[tid], q}, &total);
    taken += total.pages;
    if (b < a.B) {
      a.kv_out[b] = r.add < 0 ? 0 : r.kv + q;
      a.q_lens[b] = q;
      a.cu[b + 1] = rows + static_cast<int>(served.tokens);
      if (b0 == 0) cu_s[tid + 1] = static_cast<int>(served.tokens);
    }
    rows += static_cast<int>(total.tokens);
    for (int k = warp; k < kScan && b0 + k < a.B; k += kScan / 32)
      for (int i = lane; i < num[k]; i += 32)
        a.pages[static_cast<long long>(b0 + k) * a.max_pages + at[k] + i] = a.free_ids[first[k] - i];
  }
  if (tid == 0) *a.count_out = static_cast<int>(top - taken);
  if (tokens_too) {
    __syncthreads();
    const int* cu = a.B <= kScan ? cu_s : a.cu;
    for (int i = tid; i < a.total; i += kScan) write_token(a, cu, i);
  }
}

__global__ void __launch_bounds__(256) assign_tokens_kernel(const AssignArgs a) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  pdl_wait();
  if (i < a.total) write_token(a, a.cu, i);
}

}  // namespace

cudaError_t launch_cache_assign(const AssignArgs& a, cudaStream_t s) {
  const bool one = a.total <= kOneBlockTokens;
  assign_kernel<<<1, kScan, 0, s>>>(a, one);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || one) return e;
  return pdl_launch(assign_tokens_kernel, dim3((a.total + 255) / 256), 256, 0, s, a);
}

}  // namespace ta

TA_GUARD_ACCESSOR(assign)
