// unaligned.cuh -- 16- and 8-byte pieces read from any address as two aligned
// words and a shift, so that rows of odd pitch are read as wide as others (the
// words that neighbouring lanes share come from L1).
#pragma once

#include <cstdint>

namespace gemm14 {

// Whether the aligned words around `bytes` bytes at p (a power of two) lie in [begin, end).
__device__ __forceinline__ bool words_inside(const void* p, int bytes, const void* begin,
                                             const void* end) {
  const uintptr_t base = reinterpret_cast<uintptr_t>(p) & ~static_cast<uintptr_t>(bytes - 1);
  return base >= reinterpret_cast<uintptr_t>(begin) &&
         base + 2 * bytes <= reinterpret_cast<uintptr_t>(end);
}

// The 16 bytes from byte a (even, below 16) of lo on, those behind lo's from hi.
__device__ __forceinline__ uint4 shift16(const uint4& lo, const uint4& hi, uint32_t a) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = (a & 8u) ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = (a & 4u) ? w[i + 1] : w[i];
  const uint32_t s = (a & 3u) * 8u;
  return make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s),
                    __funnelshift_r(w[2], w[3], s), __funnelshift_r(w[3], w[4], s));
}

// 16 bytes at p (2-byte aligned; words_inside(p, 16, ..) holds).
__device__ __forceinline__ uint4 load16_any(const void* p) {
  const uint32_t a = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
  const uint4* base = reinterpret_cast<const uint4*>(static_cast<const char*>(p) - a);
  return shift16(base[0], base[1], a);
}

// 8 bytes at any p (words_inside(p, 8, ..) holds).
__device__ __forceinline__ uint2 load8_any(const void* p) {
  const uint32_t a = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 7u;
  const uint2* base = reinterpret_cast<const uint2*>(static_cast<const char*>(p) - a);
  const uint2 lo = base[0], hi = base[1];
  const bool up = (a & 4u) != 0;
  const uint32_t w0 = up ? lo.y : lo.x, w1 = up ? hi.x : lo.y, w2 = up ? hi.y : hi.x;
  const uint32_t s = (a & 3u) * 8u;
  return make_uint2(__funnelshift_r(w0, w1, s), __funnelshift_r(w1, w2, s));
}

// 4 bytes at any p (words_inside(p, 4, ..) holds).
__device__ __forceinline__ uint32_t load4_any(const void* p) {
  const uint32_t a = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 3u;
  const uint32_t* base = reinterpret_cast<const uint32_t*>(static_cast<const char*>(p) - a);
  return __funnelshift_r(base[0], base[1], a * 8u);
}

}  // namespace gemm14
