// elements.cuh -- fp32, bf16 and fp16 elements: to fp32 and back (rounded to
// nearest, ties to even), and a few of them moved as one word.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "unaligned.cuh"

namespace gemm14 {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

template <int kBytes>
struct Word;
template <>
struct Word<16> { using type = uint4; };
template <>
struct Word<8> { using type = uint2; };

// kN elements side by side, moved as one word of 8 or 16 bytes.
template <typename T, int kN>
union Pack {
  typename Word<kN * static_cast<int>(sizeof(T))>::type raw;
  T x[kN];
};

__device__ __forceinline__ uint4 load_word_any(const void* p, uint4) { return load16_any(p); }
__device__ __forceinline__ uint2 load_word_any(const void* p, uint2) { return load8_any(p); }

// Elements c .. c + kN - 1 of a row of `cols` (zeros outside it). kAny: the row
// starts at any address; [begin, end) is memory that may be read.
template <typename T, int kN, bool kAny>
__device__ __forceinline__ Pack<T, kN> load_pack(const T* row, int64_t c, int64_t cols,
                                                 const void* begin, const void* end) {
  using W = typename Word<kN * static_cast<int>(sizeof(T))>::type;
  Pack<T, kN> p;
  if (c >= 0 && c + kN <= cols && (!kAny || words_inside(row + c, sizeof(W), begin, end))) {
    if constexpr (kAny)
      p.raw = load_word_any(row + c, W());
    else
      p.raw = *reinterpret_cast<const W*>(row + c);
  } else {
#pragma unroll
    for (int j = 0; j < kN; ++j)
      p.x[j] = c + j >= 0 && c + j < cols ? row[c + j] : from_f32<T>(0.0f);
  }
  return p;
}

}  // namespace gemm14
