// Arguments of the rotary position kernels (rotary_kernels.cuh).
#pragma once
#include <cuda_runtime.h>

#include "cache.cuh"

namespace ta {

// Rows [B, heads, T, D] of 16-bit elements, element strides (b, h, t).
struct RotRows {
  void* p;
  long long sb, sh, st;
};

enum RotMode : int { kRotPlain = 0, kRotNorm = 1, kRotNormBwd = 2, kRotAppend = 3 };

struct RotArgs {
  RotRows q, k, v;     // inputs; in the backward of the norm the inputs of its forward
  RotRows dq, dk;      // backward of the norm: gradients of the outputs
  RotRows qo, ko;      // outputs
  const int* pos;      // position of token (b, t): pos[b * pos_b + t * pos_t]
  long long pos_b, pos_t;
  const int* slots;    // append: [B, T]
  const uint64_t* turns;  // [pairs]: a pair's angle per position, in units of 2^-64 of a turn
  int rot, pairs;      // rotated elements of a row, half of them
  int interleaved;
  float scale;         // of the rotated elements
  float sign;          // -1: by the negative angle
  const void *wq, *wk; // weights [D] of the norm (null: no norm)
  int w32;             // weights in fp32 (otherwise of the rows' type)
  float eps;
  float *dwq, *dwk;    // [D]
  float* part;         // [blocks][2][D] partial sums of dwq, dwk
  int blocks;          // blocks of the backward of the norm
  int T, Hq, Hkv;
  FastDiv t_div;       // by T
  FastDiv slice_div;   // by the slices of a token
  int slice_groups;    // groups of rows of a slice
  int units;           // tokens * slices
};

// Groups of rows of a slice at most: a warp copies all of a slice's to shared memory
// before it works on them (1 KB a group, 2 KB in the backward of the norm).
constexpr int kRotGroups = 12, kRotBwdGroups = 5;

// Blocks of the backward of the norm at most, two a SM: its partial sums take that many rows.
constexpr int kRotBwdBlocks = 152 * 2;

cudaError_t launch_rotary_bf16(int mode, int ct, int D, const RotArgs& a, const CacheArgs& c, cudaStream_t s);
cudaError_t launch_rotary_f16(int mode, int ct, int D, const RotArgs& a, const CacheArgs& c, cudaStream_t s);

}  // namespace ta
