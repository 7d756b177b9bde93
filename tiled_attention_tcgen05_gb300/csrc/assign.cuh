// Arguments of the page assignment kernels (assign.cu).
#pragma once
#include <cuda_runtime.h>

#include "cache.cuh"

namespace ta {

struct AssignArgs {
  int* pages;           // [B, max_pages]
  const int* kv_lens;   // [B]
  const int* new_lens;  // [B]: tokens to add; -1: the request has ended
  int* free_ids;        // [num_pages]: a stack
  const int* free_count;
  int *kv_out, *q_lens, *cu, *positions, *slots, *count_out;
  int B, max_pages, num_pages, total;
  int capacity;         // min(max_pages * page, 2^31 - 1)
  FastDiv page;
  uint32_t* err;
};

cudaError_t launch_cache_assign(const AssignArgs& a, cudaStream_t s);

}  // namespace ta
