// linear_ce_narrow.cu -- the linear cross entropy of a handful of fp32 rows (up
// to 32) on the CUDA cores: few enough that a value of W read is worth only a few
// multiplies, so that the call is bound by reading W (and writing dW) however
// plainly it multiplies, and what matters is to touch W once in each product.
// The tensor-core path has to write W's three bf16 parts first and read them
// back, 22 bytes a value against 4: 100000 x 900 from one row takes 288 us
// forward and 633 backward, here 80 and 204 (from 16 rows 145 and 344).
//
//   logits: a warp takes 4 rows of W, a lane 16 bytes of each at a time against
//     every row of H, held in shared memory, a block's rows together through
//     slices of D when H does not fit; the lanes' sums are
//     exchanged once a row (31 shuffles for 32 sums) and each lane keeps the
//     statistics, or writes dZ, of its own pair of rows. From 16 rows on, reading H
//     from shared memory bounds it (4 cycles for 16 multiplies a lane);
//   dH: a thread holds 4 columns of every row's sum and goes down its block's
//     share of W; a last kernel adds the shares;
//   dW: a thread holds 4 columns of H and goes down dZ: W is not read.
// All sums are fp32 FMAs.
#include <algorithm>

#include "kernels.h"
#include "linear_ce_narrow.h"
#include "ptx.cuh"

namespace gemm14 {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
// Warps of a logits block (one an SM): 4 x 32 sums a thread leave room for 8.
constexpr int warps_of(int kT) { return kT > 16 ? 8 : 16; }
constexpr int kSliceBytes = 200 * 1024;     // of H in shared memory
constexpr int kCols = kNarrowCols;
constexpr int kDown = 32;                   // rows of W between two loads of dZ
constexpr int kStep = 128;                  // columns a warp reads of a row at a time

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 16 bytes of a row from column c on, zeros past D; `fast`: rows start on 16 bytes.
__device__ __forceinline__ float4 load4(const float* row, int64_t c, int64_t D, bool fast) {
  if (fast && c + 4 <= D) return __ldcs(reinterpret_cast<const float4*>(row + c));
  float x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = c + j < D ? row[c + j] : 0.0f;
  return make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ bool on16(const float* p, int64_t ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 4 == 0;
}

// Sums of N (a power of two, 32 at most) values over the 32 lanes; each lane
// returns that of value lane >> (5 - log2 N).
template <int N>
__device__ __forceinline__ float across_lanes(float (&x)[N], int lane) {
  int left = N;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    if (left > 1) {
      left /= 2;
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < N / 2; ++i)
        if (i < left) {
          const float send = up ? x[i] : x[i + left];
          const float keep = up ? x[i + left] : x[i];
          x[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    } else {
      x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
    }
  }
  return x[0];
}

// What the kernels need of the rows: targets (-1: none), and for the backward
// pass lse and the coefficient dloss (0: the row takes no part; NaN: its target is
// no row of W).
struct NarrowRows {
  float coef[kNarrowRows], lse[kNarrowRows];
  int64_t target[kNarrowRows];
};
__device__ __forceinline__ void narrow_rows(const NarrowArgs& a, NarrowRows& r) {
  const int t = threadIdx.x;
  if (t >= kNarrowRows) return;
  const int64_t y = t < a.T ? a.targets[t] : a.ignore;
  const bool off = t >= a.T || y == a.ignore, sound = y >= 0 && y < a.V;
  const float g = !off && a.dloss ? a.dloss[t] : 0.0f;
  r.coef[t] = g == 0.0f || sound ? g : __uint_as_float(0x7fc00000u);
  r.lse[t] = !off && a.lse ? a.lse[t] : 0.0f;
  r.target[t] = off || !sound ? -1 : y;
}

// kT: T rounded up to a power of two. Shared memory: H's slice, kT rows of
// `slice` columns.
template <int kT, bool kGrad>
__global__ void __launch_bounds__(warps_of(kT) * 32, 1)
    narrow_logits_kernel(const NarrowArgs a, int slice) {
  constexpr int kWarps = warps_of(kT);
  constexpr int kR = 4;
  constexpr int kN = kR * kT < 32 ? kR * kT : 32, kGroups = kR * kT / kN;
  extern __shared__ float4 h_slice[];
  __shared__ NarrowRows rows;
  __shared__ float2 parts[kWarps][kGroups * 32];
  float* hs = reinterpret_cast<float*>(h_slice);
  grid_dependency_wait();
  grid_launch_dependents();
  narrow_rows(a, rows);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool fast = on16(a.W, a.ldw);
  const int slices = static_cast<int>((a.D + slice - 1) / slice);
  const int64_t batch = static_cast<int64_t>(kWarps) * kR;  // rows of W a block takes at once
  const bool fast_h = on16(a.H, a.ldh);
  const auto load_h = [&](int s) {
    const int64_t c0 = static_cast<int64_t>(s) * slice;
    for (int t = 0; t < kT; ++t)
      for (int c = 4 * threadIdx.x; c < slice; c += 4 * kWarps * 32)
        *reinterpret_cast<float4*>(hs + t * slice + c) =
            t < a.T ? load4(a.H + t * a.ldh, c0 + c, a.D, fast_h)
                    : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  if (slices == 1) load_h(0);
  __syncthreads();
  float m[kGroups], l[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.0f;
  }
  for (int64_t b0 = blockIdx.x * batch; b0 < a.V; b0 += gridDim.x * batch) {
    const int64_t v0 = b0 + warp * kR;
    float acc[kR][kT];
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
      for (int t = 0; t < kT; ++t) acc[r][t] = 0.0f;
    for (int s = 0; s < slices; ++s) {
      if (slices > 1) {
        __syncthreads();
        load_h(s);
        __syncthreads();
      }
      const int64_t c0 = static_cast<int64_t>(s) * slice;
      const int64_t c_end = min(a.D, c0 + slice);
      float4 next[kR];
#pragma unroll
      for (int r = 0; r < kR; ++r)
        next[r] = v0 + r < a.V ? load4(a.W + (v0 + r) * a.ldw, c0 + lane * 4, c_end, fast)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
      for (int64_t c = c0; c < c_end; c += kStep) {
        float4 w[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) w[r] = next[r];
        if (c + kStep < c_end) {
#pragma unroll
          for (int r = 0; r < kR; ++r)
            if (v0 + r < a.V)
              next[r] = load4(a.W + (v0 + r) * a.ldw, c + kStep + lane * 4, c_end, fast);
        }
        const float4* hp =
            reinterpret_cast<const float4*>(hs + static_cast<int>(c - c0) + lane * 4);
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          const float4 h = hp[t * (slice / 4)];
#pragma unroll
          for (int r = 0; r < kR; ++r)
            acc[r][t] = fmaf(
                w[r].w, h.w, fmaf(w[r].z, h.z, fmaf(w[r].y, h.y, fmaf(w[r].x, h.x, acc[r][t]))));
        }
      }
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      float x[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) x[i] = acc[(g * kN + i) / kT][(g * kN + i) % kT];
      const float z = across_lanes<kN>(x, lane);
      const int i = g * kN + lane / (32 / kN), t = i % kT;
      const int64_t v = v0 + i / kT;
      if (lane % (32 / kN) != 0 || v >= a.V || t >= a.T) continue;
      if constexpr (kGrad) {
        const float k = rows.coef[t];
        const float d = exp2_approx((z - rows.lse[t]) * kLog2e) - (v == rows.target[t] ? 1.0f : 0.0f);
        a.dz[t * a.ldz + v] = k == 0.0f ? 0.0f : d * k;
      } else {
        if (v == rows.target[t]) a.target_logit[t] = z;
        const float top = fmaxf(m[g], z), base = top == -INFINITY ? 0.0f : top;
        l[g] = l[g] * exp2_approx((m[g] - base) * kLog2e) + exp2_approx((z - base) * kLog2e);
        m[g] = top;
      }
    }
  }
  if constexpr (!kGrad) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) parts[warp][g * 32 + lane] = make_float2(m[g], l[g]);
    __syncthreads();
    const int t = threadIdx.x;
    if (t < a.T) {
      float top = -INFINITY, sum = 0.0f;
      for (int pass = 0; pass < 2; ++pass) {
        const float base = top == -INFINITY ? 0.0f : top;
        for (int w = 0; w < kWarps; ++w)
          for (int r = 0; r < kR; ++r) {
            const int i = r * kT + t;
            const float2 p = parts[w][i / kN * 32 + i % kN * (32 / kN)];
            if (pass == 0) top = fmaxf(top, p.x);
            else sum += p.y * exp2_approx((p.x - base) * kLog2e);
          }
      }
      a.part[static_cast<int64_t>(blockIdx.x) * a.part_ld + t] = make_float2(top, sum);
    }
  }
}

// dZ of rows v0 .. of W in shared memory, kT to a row of W.
template <int kT>
__device__ __forceinline__ void stage_dz(const NarrowArgs& a, int64_t v0, int64_t v_end,
                                         float (&dz)[kDown][kT]) {
  for (int i = threadIdx.x; i < kDown * kT; i += 256) {
    const int v = i % kDown, t = i / kDown;
    dz[v][t] = t < a.T && v0 + v < v_end ? a.dz[t * a.ldz + v0 + v] : 0.0f;
  }
}

template <int kT>
__global__ void __launch_bounds__(256) narrow_dh_kernel(const NarrowArgs a, int64_t share) {
  __shared__ __align__(16) float dz[kDown][kT];
  grid_dependency_wait();
  grid_launch_dependents();
  const bool fast = on16(a.W, a.ldw);
  const int64_t c = static_cast<int64_t>(blockIdx.y) * kCols + threadIdx.x * 4;
  const int64_t v_end = min(a.V, (blockIdx.x + 1) * share);
  float4 acc[kT];
#pragma unroll
  for (int t = 0; t < kT; ++t) acc[t] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int64_t v0 = blockIdx.x * share; v0 < v_end; v0 += kDown) {
    __syncthreads();
    stage_dz<kT>(a, v0, v_end, dz);
    __syncthreads();
    if (c >= a.D) continue;
    const int down = static_cast<int>(min(static_cast<int64_t>(kDown), v_end - v0));
    constexpr int kAhead = 8;
    for (int u0 = 0; u0 < down; u0 += kAhead) {
      float4 w[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        w[u] = u0 + u < down ? load4(a.W + (v0 + u0 + u) * a.ldw, c, a.D, fast)
                             : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          const float d = dz[u0 + u][t];
          acc[t].x = fmaf(d, w[u].x, acc[t].x);
          acc[t].y = fmaf(d, w[u].y, acc[t].y);
          acc[t].z = fmaf(d, w[u].z, acc[t].z);
          acc[t].w = fmaf(d, w[u].w, acc[t].w);
        }
    }
  }
  if (c >= a.D) return;
  float* out = a.sums + static_cast<int64_t>(blockIdx.x) * a.T * a.D;
#pragma unroll
  for (int t = 0; t < kT; ++t)
    if (t < a.T) {
      const float x[4] = {acc[t].x, acc[t].y, acc[t].z, acc[t].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < a.D) out[t * a.D + c + j] = x[j];
    }
}

// 32 columns of a row's sum a block; its 8 warps share the parts.
__global__ void __launch_bounds__(256) narrow_sum_kernel(const NarrowArgs a, int splits) {
  __shared__ NarrowRows rows;
  __shared__ float part[8][32];
  grid_dependency_wait();
  grid_launch_dependents();
  narrow_rows(a, rows);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.y;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float sum = 0.0f;
  if (c < a.D) {
    const float* from = a.sums + t * a.D + c;
#pragma unroll 8
    for (int s = warp; s < splits; s += 8) sum += __ldcg(from + static_cast<int64_t>(s) * a.T * a.D);
  }
  part[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || c >= a.D) return;
  for (int w = 1; w < 8; ++w) sum += part[w][lane];
  a.dH[t * a.lddh + c] = rows.coef[t] == 0.0f ? 0.0f : sum;
}

template <int kT>
__global__ void __launch_bounds__(256) narrow_dw_kernel(const NarrowArgs a, int64_t share) {
  __shared__ NarrowRows rows;
  __shared__ __align__(16) float dz[kDown][kT];
  grid_dependency_wait();
  grid_launch_dependents();
  narrow_rows(a, rows);
  __syncthreads();
  const bool fast = on16(a.dW, a.lddw);
  const int64_t c = static_cast<int64_t>(blockIdx.y) * kCols + threadIdx.x * 4;
  const int64_t v_end = min(a.V, (blockIdx.x + 1) * share);
  float4 h[kT];
#pragma unroll
  for (int t = 0; t < kT; ++t)
    h[t] = t < a.T && rows.coef[t] != 0.0f && c < a.D ? load4(a.H + t * a.ldh, c, a.D, false)
                                                      : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int64_t v0 = blockIdx.x * share; v0 < v_end; v0 += kDown) {
    __syncthreads();
    stage_dz<kT>(a, v0, v_end, dz);
    __syncthreads();
    if (c >= a.D) continue;
    const int down = static_cast<int>(min(static_cast<int64_t>(kDown), v_end - v0));
#pragma unroll 4
    for (int u = 0; u < down; ++u) {
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        const float d = dz[u][t];
        s.x = fmaf(d, h[t].x, s.x);
        s.y = fmaf(d, h[t].y, s.y);
        s.z = fmaf(d, h[t].z, s.z);
        s.w = fmaf(d, h[t].w, s.w);
      }
      float* to = a.dW + (v0 + u) * a.lddw + c;
      if (fast && c + 4 <= a.D) {
        *reinterpret_cast<float4*>(to) = s;
      } else {
        const float x[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c + j < a.D) to[j] = x[j];
      }
    }
  }
}

// Columns of H's slice in shared memory, a multiple of a turn's.
int slice_of(int kT, int64_t D) {
  const int most = kSliceBytes / (4 * kT) / kStep * kStep;
  const int64_t need = (D + kStep - 1) / kStep * kStep;
  return static_cast<int>(need < most ? need : most);
}

template <int kT, bool kGrad>
cudaError_t logits_as(const NarrowArgs& a, int sm_count, cudaStream_t stream) {
  static DeviceOnce once;
  const auto kernel = narrow_logits_kernel<kT, kGrad>;
  const cudaError_t e = set_smem_once(once, kernel, kSliceBytes);
  if (e != cudaSuccess) return e;
  const int slice = slice_of(kT, a.D);
  return launch_kernel(kernel, dim3(narrow_blocks(a.V, sm_count)), dim3(warps_of(kT) * 32),
                       static_cast<size_t>(kT) * slice * 4, stream, a, slice);
}

int64_t share_of(int64_t V, int splits) {
  return ((V + splits - 1) / splits + kDown - 1) / kDown * kDown;
}

template <int kT>
cudaError_t backward_as(const NarrowArgs& a, int sm_count, cudaStream_t stream) {
  cudaError_t e = logits_as<kT, true>(a, sm_count, stream);
  if (e != cudaSuccess) return e;
  const int splits = narrow_splits(a.T, a.V, a.D, sm_count);
  const int64_t share = share_of(a.V, splits);
  const dim3 grid(static_cast<unsigned>((a.V + share - 1) / share),
                  static_cast<unsigned>((a.D + kCols - 1) / kCols));
  if (a.dH) {
    e = launch_kernel(narrow_dh_kernel<kT>, grid, dim3(256), 0, stream, a, share);
    if (e != cudaSuccess) return e;
    e = launch_kernel(narrow_sum_kernel, dim3(static_cast<unsigned>((a.D + 31) / 32), a.T),
                      dim3(256), 0, stream, a, static_cast<int>(grid.x));
    if (e != cudaSuccess) return e;
  }
  if (!a.dW) return cudaSuccess;
  return launch_kernel(narrow_dw_kernel<kT>, grid, dim3(256), 0, stream, a, share);
}

template <int kT>
cudaError_t run_as(const NarrowArgs& a, bool backward, int sm_count, cudaStream_t stream) {
  return backward ? backward_as<kT>(a, sm_count, stream)
                  : logits_as<kT, false>(a, sm_count, stream);
}
cudaError_t run(const NarrowArgs& a, bool backward, int sm_count, cudaStream_t stream) {
  if (a.T <= 1) return run_as<1>(a, backward, sm_count, stream);
  if (a.T <= 2) return run_as<2>(a, backward, sm_count, stream);
  if (a.T <= 4) return run_as<4>(a, backward, sm_count, stream);
  if (a.T <= 8) return run_as<8>(a, backward, sm_count, stream);
  if (a.T <= 16) return run_as<16>(a, backward, sm_count, stream);
  return run_as<32>(a, backward, sm_count, stream);
}

}  // namespace

bool narrow_in_one_slice(int64_t T, int64_t D) {
  int kT = 1;
  while (kT < T) kT *= 2;
  return slice_of(kT, D) >= D;
}

int narrow_blocks(int64_t V, int sm_count) {
  const int64_t most = (V + 31) / 32;  // (4 rows of W for each of 8 warps)
  return static_cast<int>(std::min<int64_t>(most, sm_count));
}

int narrow_splits(int T, int64_t V, int64_t D, int sm_count) {
  // as many blocks as an SM holds: their registers hold 4 columns of every row
  const int64_t blocks = static_cast<int64_t>(sm_count) * (T > 16 ? 1 : T > 8 ? 2 : 4);
  const int64_t across = (D + kCols - 1) / kCols;
  const int64_t most = (V + kDown - 1) / kDown;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, blocks / across)));
}

cudaError_t launch_narrow_stats(const NarrowArgs& a, int sm_count, cudaStream_t stream) {
  return run(a, false, sm_count, stream);
}
cudaError_t launch_narrow_backward(const NarrowArgs& a, int sm_count, cudaStream_t stream) {
  return run(a, true, sm_count, stream);
}

}  // namespace gemm14
