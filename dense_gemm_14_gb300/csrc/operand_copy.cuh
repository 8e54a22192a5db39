// operand_copy.cuh -- an operand of the training products as the tensor-core
// kernel reads it: rows of 16-bit elements that start on 16 bytes, from rows at
// any address and pitch; or an fp32 matrix as three bf16 parts whose sum is each
// value to 24 bits (the nearest bf16, the nearest to the rest, and to the rest of
// that). Memory-bound passes, by blocks of 256 threads of a kernel of their own
// or beside other work.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "train_tc.h"
#include "unaligned.cuh"

namespace gemm14 {

// Part p of the three bf16 parts of x, taken from it: the nearest bf16, but a
// finite one where a finite x would round to an infinity (only the first part
// can; the rest makes up for it). An infinity or a NaN goes to the later parts.
__device__ __forceinline__ __nv_bfloat16 take_part(float& x, int p) {
  constexpr float kMost = 3.3895313892515355e38f;  // the largest bf16
  const __nv_bfloat16 b = __float2bfloat16_rn(p == 0 ? fminf(fmaxf(x, -kMost), kMost) : x);
  x -= __bfloat162float(b);
  return b;
}

// A thread moves 16 bytes, 4 of them in flight; a warp 128 pieces of a row.
__device__ __forceinline__ void realign_rows(const OperandCopy& j, int block, int blocks) {
  constexpr int kUnroll = 4;
  const int lane = threadIdx.x & 31;
  const uint16_t* X = static_cast<const uint16_t*>(j.src);
  const uint16_t* end = X + (j.rows - 1) * j.ld_src + j.cols;
  const int64_t per_row = (j.cols + 256 * kUnroll - 1) / (256 * kUnroll);
  for (int64_t i = static_cast<int64_t>(block) * 8 + (threadIdx.x >> 5); i < j.rows * per_row;
       i += static_cast<int64_t>(blocks) * 8) {
    const int64_t r = i / per_row, c0 = (i - r * per_row) * 256 * kUnroll + 8 * lane;
    const uint16_t* x = X + r * j.ld_src;
    uint16_t* o = static_cast<uint16_t*>(j.dst) + r * j.ld_dst;
    uint4 v[kUnroll];
    bool wide[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t c = c0 + 256 * u;
      wide[u] = c + 8 <= j.cols && words_inside(x + c, 16, X, end);
      if (wide[u]) v[u] = load16_any(x + c);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t c = c0 + 256 * u;
      if (wide[u]) {
        *reinterpret_cast<uint4*>(o + c) = v[u];
      } else {
        for (int k = 0; k < 8 && c + k < j.cols; ++k) o[c + k] = x[c + k];
      }
    }
  }
}

// A warp takes 256 columns of a row, 8 loads in flight a lane.
__device__ __forceinline__ void split_rows(const OperandCopy& j, int block, int blocks) {
  constexpr int kUnroll = 8;
  const int lane = threadIdx.x & 31;
  const float* X = static_cast<const float*>(j.src);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(j.dst);
  const int64_t per_row = (j.cols + 32 * kUnroll - 1) / (32 * kUnroll);
  for (int64_t i = static_cast<int64_t>(block) * 8 + (threadIdx.x >> 5); i < j.rows * per_row;
       i += static_cast<int64_t>(blocks) * 8) {
    const int64_t r = i / per_row, c0 = (i - r * per_row) * 32 * kUnroll + lane;
    float x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      x[u] = c0 + 32 * u < j.cols ? X[r * j.ld_src + c0 + 32 * u] : 0.0f;
#pragma unroll
    for (int p = 0; p < 3; ++p)
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const __nv_bfloat16 b = take_part(x[u], p);
        if (c0 + 32 * u < j.cols) out[p * j.part_stride + r * j.ld_dst + c0 + 32 * u] = b;
      }
  }
}

// The share of the `block`-th of `blocks` blocks.
__device__ __forceinline__ void operand_copy(const OperandCopy& j, int block, int blocks) {
  if (j.parts == 3)
    split_rows(j, block, blocks);
  else
    realign_rows(j, block, blocks);
}

}  // namespace gemm14
