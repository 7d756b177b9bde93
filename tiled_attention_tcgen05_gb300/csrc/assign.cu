// cache_assign: pages, slots, positions and offsets of a step's tokens from the
// requests' lengths.
//
// Requests in order ask for pages and tokens; a prefix sum of each says who
// is served, and which entries of the stack of free pages are whose.  The inputs
// are a few kilobytes, so latency is what it costs, and it is one
// launch: every block makes the same sums of all requests in shared memory (three
// passes of 1024 threads, some 3 us), and then takes its share of the tokens and of the
// pages.  No block waits for another's results: a token finds its page by its
// request's first entry of the stack, or, where that entry is a page that an ended
// request gives back in this very call, in that request's row; the token
// that is a page's first writes it to the table.
//
// 512 requests with up to 4096 new tokens each (800 thousand, pages of 32): 12.4 us replayed
// (a block that copied the pages of all requests, and a second launch for the
// tokens, took 26.7).  64 requests of one token: 6.3 us, what a launch and its
// dependent loads take.
//
// More than kOneLaunch requests do not fit in shared memory: a block goes over them
// in pieces and copies the pages, and a grid writes the tokens, launched while it runs.
#include "assign.cuh"

#include <algorithm>
#include <atomic>

#include "launch.h"
#include "pdl.cuh"

namespace ta {

namespace {

constexpr int kScan = 1024;

// Requests up to which every block holds the sums (16 bytes a request).
constexpr int kOneLaunch = 8192;

struct Asked {
  long long pages, tokens;
};

// Inclusive sums of N values over the block's threads, total[] those of all.
template <int N>
__device__ __forceinline__ void block_sums(long long (&v)[N], long long (&total)[N]) {
  __shared__ long long part[N][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const long long x = __shfl_up_sync(0xffffffffu, v[k], d);
      if (lane >= d) v[k] += x;
    }
  __syncthreads();  // the array's readers before
  if (lane == 31)
#pragma unroll
    for (int k = 0; k < N; ++k) part[k][warp] = v[k];
  __syncthreads();
  if (warp < N) {
    long long x = part[warp][lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    part[warp][lane] = x;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (warp > 0) v[k] += part[k][warp - 1];
    total[k] = part[k][31];
  }
}
__device__ __forceinline__ Asked block_sums(Asked v, Asked* total) {
  long long x[2] = {v.pages, v.tokens}, t[2];
  block_sums(x, t);
  *total = Asked{t[0], t[1]};
  return Asked{x[0], x[1]};
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

// The last of first[lo .. hi) that is <= x, where first[lo] is.
__device__ __forceinline__ int last_at(const int* first, int lo, int hi, int x) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// A thread's tokens at a time, 32 apart: 1, 2, 4 and 8 took 14.4, 12.4, 14.4 and 18.5 us for 800
// thousand tokens.  Every launch fetches its code anew, so longer code costs a step of single tokens, too.
constexpr int kTokens = 2;

__global__ void __launch_bounds__(kScan) assign_kernel(const AssignArgs a) {
  // first token, first page taken and first page given back of a request; tokens it holds
  extern __shared__ int sums[];
  int *cu = sums, *took = cu + a.B + 1, *gave = took + a.B, *kv = gave + a.B;
  const int tid = threadIdx.x, lane = tid & 31, page = static_cast<int>(a.page.d);
  const bool writes = blockIdx.x == 0;
  int count = __ldg(a.free_count);
  if (count < 0 || count > a.num_pages) {
    if (tid == 0) cache_error(a.err);
    count = 0;
  }
  const int each = (a.B + kScan - 1) / kScan;
  const int b0 = min(tid * each, a.B), b1 = min(b0 + each, a.B);
  long long v[3] = {0, 0, 0}, all[3];  // pages given back, pages and tokens asked for
  for (int b = b0; b < b1; ++b) {
    const Request r = request(a, b);
    const int back = r.add < 0 ? r.held : 0;
    kv[b] = r.kv;
    cu[b] = r.add;
    took[b] = r.need;
    gave[b] = back;
    v[0] += back;
    v[1] += r.need;
    v[2] += max(r.add, 0);
  }
  const long long own[3] = {v[0], v[1], v[2]};
  block_sums(v, all);
  const long long given = all[0];
  long long top = count + given;
  if (top > a.num_pages) {  // more pages came back than there are
    if (tid == 0) cache_error(a.err);
    top = a.num_pages;
  }
  long long back = v[0] - own[0], pages = v[1] - own[1], tokens = v[2] - own[2];
  long long w[2] = {0, 0}, served[2];  // tokens and pages of those who are served
  for (int b = b0; b < b1; ++b) {
    const int asked = cu[b], add = max(asked, 0), need = took[b], held = gave[b];
    const bool ok = (need == 0 || pages + need <= top) && (add == 0 || tokens + add <= a.total);
    // who is served with pages is a prefix of those who ask for some
    gave[b] = static_cast<int>(min(back, 0x7fffffffll));
    took[b] = static_cast<int>(min(pages, 0x7fffffffll));
    cu[b] = ok ? add : 0;
    back += held;
    pages += need;
    tokens += add;
    w[0] += ok ? add : 0;
    w[1] += ok ? need : 0;
    if (writes) {
      a.kv_out[b] = asked < 0 ? 0 : kv[b] + (ok ? add : 0);
      a.q_lens[b] = ok ? add : 0;
    }
  }
  const long long mine = w[0];
  block_sums(w, served);
  int at = static_cast<int>(w[0] - mine);
  for (int b = b0; b < b1; ++b) {
    const int n = cu[b];
    cu[b] = at;
    if (writes) a.cu[b] = at;
    at += n;
  }
  const int used = static_cast<int>(served[0]);
  if (tid == 0) {
    cu[a.B] = used;
    if (writes) {
      a.cu[a.B] = used;
      *a.count_out = static_cast<int>(top - served[1]);
    }
  }
  __syncthreads();
  // where the page is that ended requests give back as their x-th
  auto returned = [&](int x) {
    const int b = last_at(gave, 0, a.B, x);
    return a.pages + static_cast<long long>(b) * a.max_pages + (x - gave[b]);
  };
  for (long long x = blockIdx.x * kScan + tid; x < top - count; x += gridDim.x * kScan)
    a.free_ids[count + x] = *returned(static_cast<int>(x));

  constexpr int kSpan = 32 * kTokens;
  for (long long base = static_cast<long long>(blockIdx.x * (kScan / 32) + (tid >> 5)) * kSpan; base < a.total;
       base += static_cast<long long>(gridDim.x) * (kScan / 32) * kSpan) {
    const int i0 = static_cast<int>(base) + lane;
    const int lo0 = base < used ? last_at(cu, 0, a.B, static_cast<int>(base)) : 0;
    const int* from[kTokens];
    int* to[kTokens];
    int pos[kTokens], row[kTokens], id[kTokens];
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
      const int i = i0 + 32 * k;
      from[k] = nullptr;
      to[k] = nullptr;
      pos[k] = row[k] = 0;
      if (i < used) {
        const int b = i < cu[lo0 + 1] ? lo0 : last_at(cu, lo0 + 1, a.B, i);
        const int n = kv[b];
        pos[k] = n + (i - cu[b]);
        const int col = static_cast<int>(a.page.div(pos[k]));
        row[k] = pos[k] - col * page;
        int* entry = a.pages + static_cast<long long>(b) * a.max_pages + col;
        from[k] = entry;
        if (col * page >= n) {  // a page taken in this call
          const int held = n > 0 ? static_cast<int>(a.page.div(n - 1)) + 1 : 0;
          const int e = static_cast<int>(top) - 1 - (took[b] + col - held);
          from[k] = e < count ? a.free_ids + e : returned(e - count);
          if (row[k] == 0) to[k] = entry;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kTokens; ++k) id[k] = from[k] ? *from[k] : 0;
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
      const int i = i0 + 32 * k;
      if (i >= a.total) break;
      int slot = -1;
      if (from[k]) {
        if (static_cast<unsigned>(id[k]) < static_cast<unsigned>(a.num_pages)) slot = id[k] * page + row[k];
        else cache_error(a.err);
        if (to[k]) *to[k] = id[k];
      }
      a.positions[i] = pos[k];
      a.slots[i] = slot;
    }
  }
}

// Position and slot of token i, from what the first kernel wrote.
__device__ __forceinline__ void write_token(const AssignArgs& a, int i) {
  const int* cu = a.cu;
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

__global__ void __launch_bounds__(kScan) assign_pieces_kernel(const AssignArgs a) {
  __shared__ long long first[kScan];  // a request's first entry of the stack
  __shared__ int at[kScan], num[kScan];  // its first column, and how many
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
  if (tid == 0) a.cu[0] = 0;
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
    }
    rows += static_cast<int>(total.tokens);
    for (int k = warp; k < kScan && b0 + k < a.B; k += kScan / 32)
      for (int i = lane; i < num[k]; i += 32)
        a.pages[static_cast<long long>(b0 + k) * a.max_pages + at[k] + i] = a.free_ids[first[k] - i];
  }
  if (tid == 0) *a.count_out = static_cast<int>(top - taken);
}

__global__ void __launch_bounds__(256) assign_tokens_kernel(const AssignArgs a) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  pdl_wait();
  if (i < a.total) write_token(a, i);
}

}  // namespace

cudaError_t launch_cache_assign(const AssignArgs& a, cudaStream_t s) {
  if (a.B > kOneLaunch) {
    assign_pieces_kernel<<<1, kScan, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.total == 0) return e;
    return pdl_launch(assign_tokens_kernel, dim3((a.total + 255) / 256), 256, 0, s, a);
  }
  static std::atomic<bool> done[kMaxDevices];
  if (cudaError_t e = smem_attr_once(assign_kernel, (4 * kOneLaunch + 1) * 4, done); e != cudaSuccess) return e;
  // a round of tokens a block (and, should all requests end, of some pages a thread), a block an SM at most
  const long long pages = std::min<long long>(a.num_pages, static_cast<long long>(a.B) * a.max_pages);
  const long long rounds = (std::max<long long>(a.total, pages / 4) + kScan * kTokens - 1) / (kScan * kTokens);
  const int blocks = static_cast<int>(std::min<long long>(std::max<long long>(rounds, 1), 152));
  assign_kernel<<<blocks, kScan, (4 * a.B + 1) * 4, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ta

TA_GUARD_ACCESSOR(assign)
