// linear_ce_narrow.h -- the linear cross entropy of a handful of fp32 rows on
// the CUDA cores (linear_ce_narrow.cu). Internal; nothing here crosses the library
// boundary.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace gemm14 {

constexpr int kNarrowRows = 32;  // rows at most
constexpr int kNarrowCols = 4 * 256;  // columns of a dH or dW block
constexpr int64_t kNarrowMaxD = int64_t(65535) * kNarrowCols;

struct NarrowArgs {
  int T;
  int64_t V, D;
  const float* H;
  int64_t ldh;
  const float* W;
  int64_t ldw;
  const int64_t* targets;
  int64_t ignore;
  // forward: a part of each row's sum of exponentials for each block, [block][row]
  // with pitch part_ld, and the target's logit
  float2* part;
  int64_t part_ld;
  float* target_logit;
  // backward
  const float* lse;
  const float* dloss;
  float* dz;                   // T x V, pitch ldz
  int64_t ldz;
  float* sums;                 // narrow_splits(..) x T x D: dH's parts
  float* dH;
  int64_t lddh;
  float* dW;
  int64_t lddw;
};

bool narrow_in_one_slice(int64_t T, int64_t D);  // whether a block's shared memory holds H
int narrow_blocks(int64_t V, int sm_count);            // of the logits' launch
int narrow_splits(int T, int64_t V, int64_t D, int sm_count);  // of dH's sum over the vocabulary
cudaError_t launch_narrow_stats(const NarrowArgs& a, int sm_count, cudaStream_t stream);
// dZ, then dH and dW where they are asked for.
cudaError_t launch_narrow_backward(const NarrowArgs& a, int sm_count, cudaStream_t stream);

}  // namespace gemm14
