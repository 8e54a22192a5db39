// embedding.cu -- rows of a table looked up by token, and the gradient that the
// lookup gives back:
//     out[t] = scale W[tokens[t]],
//     dW[v] = scale sum over {t: tokens[t] = v} of dY[t]  +  beta dW[v].
// Both are memory-bound: they move rows and do one operation a value.
//
// The gradient's sums are formed in an order fixed by the sizes and the tokens
// alone: the places t are sorted by token (stable, so a token's places stay in
// order), ranges of equal length of the sorted places are summed by one group
// of threads each, and the parts of a token's sum that lie in several ranges are
// joined in order. No atomics on values, so a call repeats bit for bit, and a
// token that fills a tenth of the batch costs no more than others.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/gemm14.h"
#include "api_internal.h"
#include "checks.h"
#include "elements.cuh"
#include "kernels.h"
#include "plan.h"
#include "ptx.cuh"
#include "train_tc.h"

namespace gemm14 {
namespace {

constexpr int kThreads = 256;

struct Tokens {
  const void* p;
  int wide;  // 8 bytes each, else 4
  int64_t T, V, ignore;
};
__device__ __forceinline__ int64_t token_at(const Tokens& k, int64_t t) {
  return k.wide ? static_cast<const int64_t*>(k.p)[t] : static_cast<const int32_t*>(k.p)[t];
}
__device__ __forceinline__ bool takes_part(const Tokens& k, int64_t token) {
  return token != k.ignore && token >= 0 && token < k.V;
}

// ---- the lookup

// A thread moves kPer elements at a time, one 16-byte word of the wider type,
// kAhead of them in flight; `along` threads (a power of two) share a row, the
// block's others take other rows, and the next row's token is read while a row
// is moved. A value is multiplied in fp32 and rounded to the output's type
// (a second rounding, of a product that is right to 2^-24).
// kAny: rows at any address; the pieces are then the aligned words of the
// output's row, the table's are read as two words and a shift.
// An output that L2 cannot hold is stored past it, so that the table's rows that
// recur stay there.
constexpr int kAhead = 4;
constexpr double kStreamBytes = 64e6;

template <typename S, typename O>
__host__ __device__ constexpr int lookup_values() {
  return 16 / static_cast<int>(sizeof(S) > sizeof(O) ? sizeof(S) : sizeof(O));
}

template <typename S, typename O, bool kAny>
__global__ void __launch_bounds__(kThreads)
    embedding_kernel(const S* W, int64_t ldw, const Tokens k, O* out, int64_t ldo, int64_t D,
                     float scale, int along, int stream_out) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int kPer = lookup_values<S, O>();
  const int tx = threadIdx.x & (along - 1), ty = threadIdx.x / along;
  const int64_t row_step = static_cast<int64_t>(gridDim.x) * (kThreads / along);
  int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / along) + ty;
  const S* end = W + (k.V - 1) * ldw + D;
  int64_t next = t < k.T ? token_at(k, t) : 0;
  for (; t < k.T; t += row_step) {
    const int64_t token = next;
    if (t + row_step < k.T) next = token_at(k, t + row_step);
    const bool real = takes_part(k, token);
    const float other = token == k.ignore ? 0.0f : __uint_as_float(0x7fc00000u);
    const S* from = W + (real ? token : 0) * ldw;
    O* to = out + t * ldo;
    const int before =
        kAny ? static_cast<int>(reinterpret_cast<uintptr_t>(to) & (kPer * sizeof(O) - 1)) /
                   static_cast<int>(sizeof(O))
             : 0;
    for (int64_t c0 = static_cast<int64_t>(tx) * kPer - before; c0 < D;
         c0 += static_cast<int64_t>(along) * kAhead * kPer) {
      Pack<S, kPer> x[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int64_t c = c0 + static_cast<int64_t>(u) * along * kPer;
        if (real) x[u] = load_pack<S, kPer, kAny>(from, c, D, W, end);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int64_t c = c0 + static_cast<int64_t>(u) * along * kPer;
        Pack<O, kPer> y;
#pragma unroll
        for (int j = 0; j < kPer; ++j) y.x[j] = from_f32<O>(real ? scale * to_f32(x[u].x[j]) : other);
        if (c >= 0 && c + kPer <= D) {
          if (stream_out)
            __stcs(reinterpret_cast<decltype(y.raw)*>(to + c), y.raw);
          else
            *reinterpret_cast<decltype(y.raw)*>(to + c) = y.raw;
        } else {
#pragma unroll
          for (int j = 0; j < kPer; ++j)
            if (c + j >= 0 && c + j < D) to[c + j] = y.x[j];
        }
      }
    }
  }
}

// Rows at any address between types of different widths: a lane an element.
template <typename S, typename O>
__global__ void __launch_bounds__(kThreads)
    embedding_elements_kernel(const S* W, int64_t ldw, const Tokens k, O* out, int64_t ldo,
                              int64_t D, float scale, int along) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int kEach = 8;
  const int tx = threadIdx.x & (along - 1), ty = threadIdx.x / along;
  const int64_t row_step = static_cast<int64_t>(gridDim.x) * (kThreads / along);
  int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / along) + ty;
  int64_t next = t < k.T ? token_at(k, t) : 0;
  for (; t < k.T; t += row_step) {
    const int64_t token = next;
    if (t + row_step < k.T) next = token_at(k, t + row_step);
    const bool real = takes_part(k, token);
    const float other = token == k.ignore ? 0.0f : __uint_as_float(0x7fc00000u);
    const S* from = W + (real ? token : 0) * ldw;
    O* to = out + t * ldo;
    for (int64_t c0 = tx; c0 < D; c0 += static_cast<int64_t>(along) * kEach) {
      float x[kEach];
#pragma unroll
      for (int u = 0; u < kEach; ++u) {
        const int64_t c = c0 + static_cast<int64_t>(u) * along;
        x[u] = real && c < D ? to_f32(from[c]) : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < kEach; ++u) {
        const int64_t c = c0 + static_cast<int64_t>(u) * along;
        if (c < D) to[c] = from_f32<O>(real ? scale * x[u] : other);
      }
    }
  }
}

// Threads along a row of so many items, a power of two of 8 at least: as many as
// leave each `ahead` items, more where the rows are too few for the SMs.
int threads_along(int64_t rows, int64_t items, int ahead, int sms) {
  int x = 8;
  while (x < kThreads && static_cast<int64_t>(x) * ahead < items) x *= 2;
  while (x < kThreads && x < items && rows * x < static_cast<int64_t>(sms) * 1024) x *= 2;
  return x;
}

int grid_for(int64_t threads_needed, int sms) {
  const int64_t blocks = (threads_needed + kThreads - 1) / kThreads;
  const int64_t most = static_cast<int64_t>(sms) * 8;
  return static_cast<int>(blocks < most ? blocks : most);
}

bool rows_on(const void* p, int64_t ld, int size, int bytes) {
  return aligned(p, bytes) && ld * size % bytes == 0;
}

template <typename S, typename O>
cudaError_t lookup_as(const void* W, int64_t ldw, const Tokens& k, void* out, int64_t ldo,
                      int64_t D, float scale, int sms, cudaStream_t stream) {
  constexpr int kPer = lookup_values<S, O>();
  const S* w = static_cast<const S*>(W);
  O* o = static_cast<O*>(out);
  const bool words = rows_on(W, ldw, sizeof(S), kPer * sizeof(S)) &&
                     rows_on(out, ldo, sizeof(O), kPer * sizeof(O));
  if (!words && sizeof(S) != sizeof(O)) {
    const int along = threads_along(k.T, D, 8, sms);
    return launch_kernel(embedding_elements_kernel<S, O>, dim3(grid_for(k.T * along, sms)),
                         dim3(kThreads), 0, stream, w, ldw, k, o, ldo, D, scale, along);
  }
  const int along = threads_along(k.T, (D + kPer - 1) / kPer + (words ? 0 : 1), kAhead, sms);
  const int stream_out = static_cast<double>(k.T) * D * sizeof(O) > kStreamBytes;
  if constexpr (sizeof(S) == sizeof(O)) {
    if (!words)
      return launch_kernel(embedding_kernel<S, O, true>, dim3(grid_for(k.T * along, sms)),
                           dim3(kThreads), 0, stream, w, ldw, k, o, ldo, D, scale, along, stream_out);
  }
  return launch_kernel(embedding_kernel<S, O, false>, dim3(grid_for(k.T * along, sms)),
                       dim3(kThreads), 0, stream, w, ldw, k, o, ldo, D, scale, along, stream_out);
}

// ---- rows of the gradient that no token stands for

// What the summing kernels do not write: rows of dW without tokens become beta
// times what they are (beta = 0: zeros, nothing is read; beta = 1: nothing is done).
template <typename O>
struct Rest {
  O* dW;
  int64_t lddw, D;
  float beta;
};
constexpr int kRestRows = 65536;  // rows that a block marks at a time, a bit each

// Rows [v0, v1): marks those that tokens stand for, then writes the others, a warp a row.
template <typename O>
__device__ __forceinline__ void write_rest(const Rest<O>& r, const Tokens& k, int64_t v0,
                                           int64_t v1, uint32_t* marks, int most) {
  constexpr int kWord = 16 / static_cast<int>(sizeof(O));
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  for (int64_t begin = v0; begin < v1; begin += most) {
    const int rows = static_cast<int>(min(static_cast<int64_t>(most), v1 - begin));
    __syncthreads();
    for (int i = threadIdx.x; i < (rows + 31) / 32; i += blockDim.x) marks[i] = 0u;
    __syncthreads();
    for (int64_t t0 = threadIdx.x; t0 < k.T; t0 += static_cast<int64_t>(blockDim.x) * 8) {
      int64_t token[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int64_t t = t0 + static_cast<int64_t>(u) * blockDim.x;
        token[u] = t < k.T ? token_at(k, t) : -1;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (takes_part(k, token[u]) && token[u] >= begin && token[u] < begin + rows)
          atomicOr(&marks[(token[u] - begin) >> 5], 1u << ((token[u] - begin) & 31));
    }
    __syncthreads();
    for (int i = warp; i < rows; i += warps) {
      if (marks[i >> 5] >> (i & 31) & 1u) continue;
      O* row = r.dW + (begin + i) * r.lddw;
      const int64_t lead = min(r.D, static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) /
                                        static_cast<int64_t>(sizeof(O)));
      const int64_t words = (r.D - lead) / kWord;
      if (lane < lead) row[lane] = from_f32<O>(r.beta == 0.0f ? 0.0f : r.beta * to_f32(row[lane]));
      const int64_t tail = lead + words * kWord;
      if (tail + lane < r.D)
        row[tail + lane] = from_f32<O>(r.beta == 0.0f ? 0.0f : r.beta * to_f32(row[tail + lane]));
      uint4* at = reinterpret_cast<uint4*>(row + lead);
      if (r.beta == 0.0f) {
        for (int64_t w = lane; w < words; w += 32) at[w] = make_uint4(0u, 0u, 0u, 0u);
      } else {
        for (int64_t w = lane; w < words; w += 32) {
          Pack<O, kWord> p;
          p.raw = at[w];
#pragma unroll
          for (int j = 0; j < kWord; ++j) p.x[j] = from_f32<O>(r.beta * to_f32(p.x[j]));
          at[w] = p.raw;
        }
      }
    }
  }
}

// Runs beside the sort: the sort lets it start once everything before the sort
// has completed, so it needs no wait before its first access; the wait at its
// end makes whatever waits for it wait for the sort too.
constexpr int kRestThreads = 512;
template <typename O>
__global__ void __launch_bounds__(kRestThreads)
    embedding_rest_kernel(const Rest<O> r, const Tokens k, int64_t share) {
  __shared__ uint32_t marks[kRestRows / 32];
  const int64_t v0 = blockIdx.x * share;
  write_rest(r, k, v0, min(k.V, v0 + share), marks, kRestRows);
  grid_dependency_wait();
  grid_launch_dependents();
}

// ---- sums of rows

// kPer values of a row of dW from their sums.
template <typename O, int kPer>
__device__ __forceinline__ void put_sums(O* row, int64_t c, int64_t D, const float (&sum)[kPer],
                                         float scale, float beta, bool words) {
  constexpr int kWord = 16 / static_cast<int>(sizeof(O));
  if (words && c + kPer <= D) {
#pragma unroll
    for (int w = 0; w < kPer / kWord; ++w) {
      Pack<O, kWord> p;
      uint4* at = reinterpret_cast<uint4*>(row + c + w * kWord);
      if (beta != 0.0f) p.raw = *at;
#pragma unroll
      for (int j = 0; j < kWord; ++j) {
        const float s = scale * sum[w * kWord + j];
        p.x[j] = from_f32<O>(beta != 0.0f ? fmaf(beta, to_f32(p.x[j]), s) : s);
      }
      *at = p.raw;
    }
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (c + j >= D) break;
      const float s = scale * sum[j];
      row[c + j] = from_f32<O>(beta != 0.0f ? fmaf(beta, to_f32(row[c + j]), s) : s);
    }
  }
}

template <typename S, int kPer>
__device__ __forceinline__ void add_to(float (&sum)[kPer], const Pack<S, kPer>& x) {
#pragma unroll
  for (int j = 0; j < kPer; ++j) sum[j] += to_f32(x.x[j]);
}

constexpr int kRowsAhead = 8;  // rows of dY in flight

// Columns a thread has: one 16-byte word of the wider type.
template <typename S, typename O>
__host__ __device__ constexpr int sum_values() { return lookup_values<S, O>(); }

template <typename S, typename O>
struct GradArgs {
  const S* dY;
  int64_t lddy;
  O* dW;
  int64_t lddw, D;
  float scale, beta;
  int words;  // dW's rows start on 16 bytes
  unsigned* err;
};

// A few tokens: a block a token and a slice of the columns. The block of a
// token's first place sums all its places, in order; the blocks past them write
// the rows without tokens. One launch, no workspace.
constexpr int kFewTokens = kThreads;

template <typename S, typename O, bool kAny>
__global__ void __launch_bounds__(kThreads)
    embedding_grad_few_kernel(const GradArgs<S, O> a, const Tokens k, int slices, int64_t share) {
  constexpr int kPer = sum_values<S, O>();
  constexpr int kWarps = kThreads / 32, kMarked = 8192;
  __shared__ uint32_t marks[kMarked / 32];
  __shared__ int places[kFewTokens];
  __shared__ int counts[kWarps];
  grid_dependency_wait();
  grid_launch_dependents();
  const int T = static_cast<int>(k.T), tid = threadIdx.x;
  if (static_cast<int64_t>(blockIdx.x) >= static_cast<int64_t>(T) * slices) {
    const int64_t v0 = (blockIdx.x - static_cast<int64_t>(T) * slices) * share;
    write_rest(Rest<O>{a.dW, a.lddw, a.D, a.beta}, k, v0, min(k.V, v0 + share), marks, kMarked);
    return;
  }
  const int t = blockIdx.x / slices, slice = blockIdx.x - t * slices;
  const int64_t token = token_at(k, t);
  const bool same = tid < T && token_at(k, tid) == token;
  if (__syncthreads_or(same && tid < t) || !takes_part(k, token)) return;
  const uint32_t mine = __ballot_sync(0xffffffffu, same);
  if ((tid & 31) == 0) counts[tid >> 5] = __popc(mine);
  __syncthreads();
  int at = __popc(mine & ((1u << (tid & 31)) - 1u)), n = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < tid >> 5) at += counts[w];
    n += counts[w];
  }
  if (same) places[at] = tid;
  __syncthreads();
  const int64_t c = (static_cast<int64_t>(slice) * kThreads + tid) * kPer;
  if (c >= a.D) return;
  const S* end = a.dY + (k.T - 1) * a.lddy + a.D;
  float sum[kPer] = {};
  for (int i = 0; i < n; i += kRowsAhead) {
    Pack<S, kPer> x[kRowsAhead];
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u)
      if (i + u < n) x[u] = load_pack<S, kPer, kAny>(a.dY + places[i + u] * a.lddy, c, a.D, a.dY, end);
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u)
      if (i + u < n) add_to<S, kPer>(sum, x[u]);
  }
  put_sums<O, kPer>(a.dW + token * a.lddw, c, a.D, sum, a.scale, a.beta, a.words != 0);
}

// ---- the places sorted by token

// Radix sort, least significant digit first, of the places that take part, by
// one cluster of kCtas CTAs whose barriers are the hardware's. In a pass every
// warp has a range of the list: it counts its digits (shared-memory atomics on
// its own counts), the counts are summed over warps and CTAs (through
// distributed shared memory) to each warp's first position for each digit, and
// the warp goes through its range again and moves the places there, in order:
// a ballot for each bit of the digit finds the lanes that have the same one.
// Two passes for a vocabulary of up to 2^18; the first leaves out what takes no
// part. Between passes the list lies in L2; in shared memory where one CTA does.
// @SORT@
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int kSortAhead = 8;  // words in flight a lane

struct SortArgs {
  Tokens k;
  uint2* list[2];   // the sorted places: the token, and which place it is
  uint32_t* count;  // how many take part, and (count[1], set to 0) long sums
  int bits, passes;  // digits of this many bits
  unsigned* err;
};

constexpr int kOneCta = kSortThreads * kSortAhead;  // places that one CTA sorts
constexpr int kEightCtas = 2 * kOneCta;
template <int kCtas>
constexpr size_t sort_smem_bytes() {
  return (static_cast<size_t>(kSortWarps) * kDigits + 2 * kDigits + 32) * 4 +
         (kCtas == 1 ? static_cast<size_t>(kOneCta) * sizeof(uint2) : 0);
}

__device__ __forceinline__ uint32_t load_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

template <int kCtas>
__global__ void __launch_bounds__(kSortThreads)
    embedding_sort_kernel(const SortArgs a) {
  extern __shared__ __align__(16) uint32_t sort_smem[];
  uint32_t* hist = sort_smem;                     // [warp][digit]
  uint32_t* total = hist + kSortWarps * kDigits;  // of this CTA, read by the others
  uint32_t* base = total + kDigits;
  uint32_t* sums = base + kDigits;                // of a warp's digits in the scan
  uint2* own = reinterpret_cast<uint2*>(sums + 32);  // kCtas == 1: the list between passes
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = kCtas > 1 ? cluster_ctarank() : 0u;
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t T = static_cast<uint32_t>(a.k.T);
  uint32_t n = T;
  uint32_t* my_hist = hist + warp * kDigits;
  for (int pass = 0; pass < a.passes; ++pass) {
    const uint2* in = kCtas == 1 ? own : a.list[(pass + 1) & 1];
    uint2* out = kCtas == 1 && pass + 1 < a.passes ? own : a.list[pass & 1];
    const int shift = pass * a.bits;
    const uint32_t mask = (1u << a.bits) - 1u;
    const uint32_t per_cta = (n + kCtas - 1) / kCtas;
    const uint32_t per_warp = ((per_cta + kSortWarps - 1) / kSortWarps + 31u) & ~31u;
    const uint32_t cta_begin = min(n, rank * per_cta), cta_end = min(n, cta_begin + per_cta);
    const uint32_t begin = min(cta_end, cta_begin + warp * per_warp);
    const uint32_t end = min(cta_end, begin + per_warp);
    for (int i = tid; i < kSortWarps * kDigits / 4; i += kSortThreads)
      reinterpret_cast<uint4*>(hist)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    // ~0u: takes no part (tokens are below 2^31)
    uint32_t key[kSortAhead], at[kSortAhead];
    const auto load = [&](uint32_t i0) {
#pragma unroll
      for (int u = 0; u < kSortAhead; ++u) {
        const uint32_t i = i0 + u * 32u + lane;
        key[u] = ~0u;
        at[u] = i;
        if (i >= end) continue;
        if (pass == 0) {
          const int64_t token = token_at(a.k, i);
          if (takes_part(a.k, token)) key[u] = static_cast<uint32_t>(token);
        } else {
          const uint2 v = kCtas == 1 ? in[i] : __ldcg(in + i);
          key[u] = v.x;
          at[u] = v.y;
        }
      }
    };
    for (uint32_t i0 = begin; i0 < end; i0 += kSortAhead * 32u) {
      load(i0);
#pragma unroll
      for (int u = 0; u < kSortAhead; ++u)
        if (key[u] != ~0u) atomicAdd(&my_hist[(key[u] >> shift) & mask], 1u);
    }
    __syncthreads();
    if (tid < kDigits) {
      uint32_t c[kSortWarps], s = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) c[w] = hist[w * kDigits + tid];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        hist[w * kDigits + tid] = s;
        s += c[w];
      }
      total[tid] = s;
    }
    if (kCtas > 1)
      cluster_sync();
    else
      __syncthreads();
    uint32_t all = 0, before = 0;
    if (tid < kDigits) {
#pragma unroll
      for (int c = 0; c < kCtas; ++c) {
        const uint32_t v =
            kCtas > 1 ? load_cluster_u32(mapa_shared(smem_u32(total + tid), c)) : total[tid];
        all += v;
        if (c < static_cast<int>(rank)) before += v;
      }
    }
    uint32_t upto = all;  // of the warp's digits up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    uint32_t lower = 0, found = 0;
#pragma unroll
    for (int w = 0; w < kDigits / 32; ++w) {
      if (w < warp) lower += sums[w];
      found += sums[w];
    }
    if (tid < kDigits) base[tid] = lower + upto - all + before;
    __syncthreads();
    const bool kept = end - begin <= kSortAhead * 32u;  // the keys are still in registers
    for (uint32_t i0 = begin; i0 < end; i0 += kSortAhead * 32u) {
      if (!kept) load(i0);
#pragma unroll
      for (int u = 0; u < kSortAhead; ++u) {
        if (i0 + u * 32u >= end) break;
        const uint32_t digit = (key[u] >> shift) & mask;
        const bool on = key[u] != ~0u;
        uint32_t peers = __ballot_sync(0xffffffffu, on);  // lanes of this lane's digit
#pragma unroll
        for (int b = 0; b < kDigitBits; ++b) {
          const uint32_t set = __ballot_sync(0xffffffffu, digit >> b & 1u);
          peers &= digit >> b & 1u ? set : ~set;
        }
        uint32_t first = 0;
        if (on) first = base[digit] + my_hist[digit];
        __syncwarp();
        if (on && lane == __ffs(peers) - 1) my_hist[digit] += __popc(peers);
        __syncwarp();
        if (on) {
          const uint32_t to = first + __popc(peers & ((1u << lane) - 1u));
          if (dev_check(index_ok(to, T), a.err)) out[to] = make_uint2(key[u], at[u]);
        }
      }
    }
    n = found;
    // the next pass reads what the others wrote, and writes what they read
    if (kCtas > 1)
      cluster_sync();
    else
      __syncthreads();
  }
  if (rank == 0 && tid < 2) a.count[tid] = tid == 0 ? n : 0u;
}

// ---- sums over ranges of the sorted places

// A group of `along` threads takes one range of the sorted places and a slice of
// the columns, kPer of them a thread (16 bytes of dY's type), kRowsAhead rows in
// flight. A token of up to kWhole places is one range's, the one where it begins;
// the sum of a longer one may lie in several: what a range holds of a sum that
// began before it, or goes on behind it, goes to the range's first or second slot,
// and the range where it began goes on a list for the join.
struct Ranges {
  const uint2* place;  // sorted: token, place
  uint32_t* count;     // places, and long sums
  uint32_t* list;      // of the ranges where a sum begins that goes on behind them
  float* slots;        // two rows of slot_ld floats a range
  int64_t slot_ld;
  int64_t ranges;
  int along, slices;
};
constexpr uint32_t kLeastRange = 8, kWhole = 16;

// Places of a range: all ranges but the last hold as many, before their ends move.
__device__ __forceinline__ uint32_t range_length(uint32_t n, int64_t ranges) {
  const uint32_t even = static_cast<uint32_t>((n + ranges - 1) / ranges);
  return max(kLeastRange, even);
}
// Where a range that should begin at p does, from which of the places p - 16 ..
// p + 15 have p's token: at p, or behind the token that has places on both sides
// of p, if it has no more than kWhole.
__device__ __forceinline__ uint32_t moved(uint32_t p, uint32_t same) {
  const uint32_t before = static_cast<uint32_t>(__clz(static_cast<int>(~(same << 16))));  // <= 16
  const uint32_t after = static_cast<uint32_t>(__ffs(static_cast<int>(~(same >> 16))) - 1);
  return before == 0 || before + after > kWhole ? p : p + after;
}
// The range's places [p0, p1).
__device__ __forceinline__ void range_ends(const Ranges& r, int64_t range, uint32_t n,
                                           uint32_t& p0, uint32_t& p1) {
  const uint32_t length = range_length(n, r.ranges);
  const uint32_t q[2] = {
      static_cast<uint32_t>(min(static_cast<int64_t>(n), range * length)),
      static_cast<uint32_t>(min(static_cast<int64_t>(n), (range + 1) * length))};
  uint32_t same[2] = {0u, 0u};
  if (r.along >= 32) {  // a warp's range: its lanes look at a place each
    uint32_t token[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int64_t i = static_cast<int64_t>(q[e]) - 16 + (threadIdx.x & 31);
      token[e] = i >= 0 && i < n ? r.place[i].x : ~0u;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
      same[e] = __ballot_sync(0xffffffffu, token[e] == __shfl_sync(0xffffffffu, token[e], 16) &&
                                               token[e] != ~0u);
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t token = q[e] < n ? r.place[q[e]].x : ~0u;
#pragma unroll 8
      for (int u = 0; u < 32; ++u) {
        const int64_t i = static_cast<int64_t>(q[e]) - 16 + u;
        if (i >= 0 && i < n && r.place[i].x == token) same[e] |= 1u << u;
      }
    }
  }
  p0 = q[0] < n ? moved(q[0], same[0]) : n;
  p1 = q[1] < n ? moved(q[1], same[1]) : n;
}

// A thread's columns of a row of dW.
template <typename O, int kPer>
struct alignas(kPer * sizeof(O)) Columns {
  O x[kPer];
};

// kMode kWordsAdd: sums are added to rows that are there (beta != 0). The old words
// of the sums that end among the rows in flight are loaded with them, so that no
// sum waits for its own (65536 places of 2048 columns, bf16 added to fp32: 225 us
// with a load at each sum's end, @SUMADD@ so). kAnywhere: rows of dY or dW at any
// address (dW's values are then moved one by one).
enum SumMode { kWordsSet, kWordsAdd, kAnywhere };
constexpr int kSumBlocks = 4;  // resident of an SM
template <typename S, typename O, int kMode>
__global__ void __launch_bounds__(kThreads, kSumBlocks)
    embedding_sum_kernel(const GradArgs<S, O> a, const Ranges r, int64_t T, int64_t V) {
  constexpr int kPer = sum_values<S, O>();
  constexpr bool kAny = kMode == kAnywhere, kAdd = kMode == kWordsAdd;
  constexpr int kRows = kAdd ? 4 : kRowsAhead;
  constexpr uint32_t kFlag = 0x80000000u;  // beside a token or a place, below 2^31
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t n = *r.count;
  const int tx = threadIdx.x & (r.along - 1), group = threadIdx.x / r.along;
  const int64_t part = blockIdx.x / r.slices;
  const int slice = static_cast<int>(blockIdx.x - part * r.slices);
  const int64_t range = part * (kThreads / r.along) + group;
  const int64_t c = (static_cast<int64_t>(slice) * r.along + tx) * kPer;
  uint32_t p0 = n, p1 = n;
  if (range < r.ranges) range_ends(r, range, n, p0, p1);
  const uint32_t most = __reduce_max_sync(0xffffffffu, p1 - p0);  // of the warp's ranges
  const bool live = c < a.D, whole = c + kPer <= a.D;
  const uint32_t length = live ? p1 - p0 : 0u;
  const S* from = a.dY + (kAny ? 0 : c);
  O* to = a.dW + c;
  float* slot = r.slots + 2 * range * r.slot_ld + c;
  // a stage of the range's places, one a lane: the token (kFlag: its sum goes on
  // behind the range) and the place (kFlag: the last of its sum here)
  const int stage = min(r.along, 32), in_stage = threadIdx.x & (stage - 1);
  const auto places = [&](uint32_t q) {
    const uint32_t p = p0 + q + in_stage;
    if (p >= p1) return make_uint2(0u, 0u);
    uint2 v = r.place[p];
    const bool same = p + 1 < n && r.place[p + 1].x == v.x;
    if (p + 1 == p1 && same) v.x |= kFlag;
    if (p + 1 == p1 || !same) v.y |= kFlag;
    return v;
  };
  float sum[kPer] = {};
  bool began_before = p0 > 0 && p0 < p1 && r.place[p0 - 1].x == r.place[p0].x;
  uint2 next = places(0);
  for (uint32_t q = 0; q < most; q += stage) {
    const uint2 now = next;
    next = places(q + stage);
    for (int u0 = 0; u0 < stage && q + u0 < most; u0 += kRows) {
      Pack<S, kPer> x[kRows];
      Columns<O, kPer> old[kAdd ? kRows : 1];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const uint32_t at = __shfl_sync(0xffffffffu, now.y, u0 + u, stage);
        const bool on = q + u0 + u < length;
        const S* row = from + static_cast<int64_t>(at & ~kFlag) * a.lddy;
        if constexpr (kAny) {
          if (on)
            x[u] = load_pack<S, kPer, true>(row, c, a.D, a.dY, a.dY + (T - 1) * a.lddy + a.D);
        } else if (on && whole) {
          x[u].raw = *reinterpret_cast<const decltype(x[u].raw)*>(row);
        } else if (on) {
#pragma unroll
          for (int j = 0; j < kPer; ++j) x[u].x[j] = c + j < a.D ? row[j] : from_f32<S>(0.0f);
        }
        if constexpr (kAdd) {
          const uint32_t token = __shfl_sync(0xffffffffu, now.x, u0 + u, stage);
          if (on && whole && (at & kFlag) && !(token & kFlag) && dev_check(index_ok(token, V), a.err))
            old[u] = *reinterpret_cast<const Columns<O, kPer>*>(to + token * a.lddw);
        }
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const uint32_t at = __shfl_sync(0xffffffffu, now.y, u0 + u, stage);
        const uint32_t token = __shfl_sync(0xffffffffu, now.x, u0 + u, stage);
        if (q + u0 + u >= length) continue;
        add_to<S, kPer>(sum, x[u]);
        if (!(at & kFlag)) continue;
        if (began_before || (token & kFlag)) {
          float* s = began_before ? slot : slot + r.slot_ld;
#pragma unroll
          for (int j = 0; j < kPer; j += 4)
            *reinterpret_cast<float4*>(s + j) = make_float4(sum[j], sum[j + 1], sum[j + 2], sum[j + 3]);
          if (c == 0 && !began_before)
            r.list[atomicAdd(r.count + 1, 1u)] = static_cast<uint32_t>(range);
        } else if (dev_check(index_ok(token, V), a.err)) {
          O* row = to + token * a.lddw;
          if (!kAny && whole) {
            Columns<O, kPer> y;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
              const float s = a.scale * sum[j];
              y.x[j] = from_f32<O>(kAdd ? fmaf(a.beta, to_f32(old[kAdd ? u : 0].x[j]), s) : s);
            }
            *reinterpret_cast<Columns<O, kPer>*>(row) = y;
          } else {
            float y[kPer];
#pragma unroll
            for (int j = 0; j < kPer; ++j)
              y[j] = a.beta != 0.0f && c + j < a.D ? to_f32(row[j]) : 0.0f;
#pragma unroll
            for (int j = 0; j < kPer; ++j)
              if (c + j < a.D)
                row[j] = from_f32<O>(a.beta != 0.0f ? fmaf(a.beta, y[j], a.scale * sum[j])
                                                    : a.scale * sum[j]);
          }
        }
        began_before = false;
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum[j] = 0.0f;
      }
    }
  }
}

// The sums that lie in several ranges, 128 columns of one by a block at a time:
// its warps add the ranges' slots in turn, every eighth each, and the warps' sums
// are added in order. (The list's order, which varies, decides nothing but which
// block that is.)
template <typename O>
__global__ void __launch_bounds__(kThreads)
    embedding_join_kernel(O* dW, int64_t lddw, int64_t D, float scale, float beta, const Ranges r,
                          int64_t V, unsigned* err) {
  constexpr int kWarps = kThreads / 32, kEach = 4;
  __shared__ float4 sums[kWarps][32];
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t n = r.count[0], listed = r.count[1];
  const uint32_t length = range_length(n, r.ranges);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t slices = (D + 127) / 128;
  for (int64_t item = blockIdx.x; item < listed * slices; item += gridDim.x) {
    const int64_t range = r.list[item / slices];
    const int64_t c = (item % slices) * 128 + lane * 4;
    const uint32_t token = r.place[(range + 1) * length].x;
    // the ranges behind it that begin within the sum
    int64_t last = range;
    for (bool more = true; more; last += more ? 32 : 0) {
      const int64_t i = last + 1 + lane;
      const uint32_t in = __ballot_sync(0xffffffffu, i * length < n && r.place[i * length].x == token);
      more = in == 0xffffffffu;
      if (!more) last += __popc(in);
    }
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    // slot 0 of this loop is the range's own second one, slot k the first of the k-th behind it
    for (int64_t k0 = warp; k0 <= last - range; k0 += kWarps * kEach) {
      float4 v[kEach];
#pragma unroll
      for (int u = 0; u < kEach; ++u) {
        const int64_t k = k0 + u * kWarps;
        v[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (k <= last - range && c < r.slot_ld)
          v[u] = *reinterpret_cast<const float4*>(r.slots + (2 * (range + k) + (k == 0)) * r.slot_ld + c);
      }
#pragma unroll
      for (int u = 0; u < kEach; ++u) {
        s.x += v[u].x;
        s.y += v[u].y;
        s.z += v[u].z;
        s.w += v[u].w;
      }
    }
    __syncthreads();
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < D) {
      float all[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        const float4 v = sums[w][lane];
        all[0] += v.x;
        all[1] += v.y;
        all[2] += v.z;
        all[3] += v.w;
      }
      if (dev_check(index_ok(token, V), err))
        put_sums<O, 4>(dW + token * lddw, c, D, all, scale, beta, false);
    }
  }
}

// ---- the call's plan

struct GradPlan {
  bool few = false;        // one launch, no workspace
  int along = 8, slices = 1, ctas = 1;
  int bits = 1, passes = 1;
  int64_t ranges = 1, slot_ld = 0, blocks = 1;
  size_t place_off[2] = {}, count_off = 0, list_off = 0, slots_off = 0, total = 0;
};

void grad_plan(int dtype, int dtype_out, int64_t T, int64_t V, int64_t D, int sms, GradPlan* g) {
  const int wider = std::max(elem_bytes_of(dtype), elem_bytes_of(dtype_out)), per = 16 / wider;
  const int64_t pieces = (D + per - 1) / per;
  if (T <= kFewTokens) {
    g->few = true;
    g->slices = static_cast<int>((pieces + kThreads - 1) / kThreads);
    return;
  }
  while (g->along < kThreads && g->along < pieces) g->along *= 2;
  g->slices = static_cast<int>((pieces + g->along - 1) / g->along);
  const int groups = kThreads / g->along;
  // as many ranges as are resident at once, of 8 places at least
  const int64_t most = (T + kLeastRange - 1) / kLeastRange;
  g->ranges = static_cast<int64_t>(sms) * kSumBlocks * groups / g->slices;
  if (g->ranges < 1) g->ranges = 1;
  if (g->ranges > most) g->ranges = most;
  g->blocks = (g->ranges + groups - 1) / groups * g->slices;
  g->slot_ld = pieces * per;
  int width = 1;
  while (width < 31 && (V - 1) >> width) ++width;
  g->passes = (width + kDigitBits - 1) / kDigitBits;
  g->bits = (width + g->passes - 1) / g->passes;
  g->ctas = T <= kOneCta ? 1 : T <= kEightCtas ? 8 : 16;
  size_t at = streamk_flag_bytes(sms);
  const auto take = [&](size_t bytes) {
    const size_t o = at;
    at += round256(bytes);
    return o;
  };
  g->count_off = take(8);
  g->list_off = take(static_cast<size_t>(g->ranges) * 4);
  for (int i = 0; i < 2; ++i) g->place_off[i] = take(static_cast<size_t>(T) * sizeof(uint2));
  g->slots_off = take(static_cast<size_t>(g->ranges) * 2 * g->slot_ld * 4);
  g->total = at;
}

// Clusters of 16 are not portable: whether this device runs one, else 8 do.
template <int kCtas>
cudaError_t sort_config(cudaStream_t stream, cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr) {
  static DeviceOnce configured;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg->gridDim = dim3(kCtas);
  cfg->blockDim = dim3(kSortThreads);
  cfg->dynamicSmemBytes = sort_smem_bytes<kCtas>();
  cfg->stream = stream;
  cfg->attrs = attr;
  cfg->numAttrs = 2;
  return static_cast<cudaError_t>(configured.get(
      dev,
      [&] {
        cudaError_t r = cudaFuncSetAttribute(embedding_sort_kernel<kCtas>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(cfg->dynamicSmemBytes));
        if (r == cudaSuccess && kCtas > 8)
          r = cudaFuncSetAttribute(embedding_sort_kernel<kCtas>,
                                   cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        int clusters = 1;
        if (r == cudaSuccess && kCtas > 8)
          r = cudaOccupancyMaxActiveClusters(&clusters, embedding_sort_kernel<kCtas>, cfg);
        if (r == cudaSuccess && clusters < 1) r = cudaErrorInvalidConfiguration;
        return static_cast<int>(r);
      },
      [](int r) { return r == static_cast<int>(cudaSuccess) ||
                       r == static_cast<int>(cudaErrorInvalidConfiguration); }));
}
template <int kCtas>
cudaError_t launch_sort(const SortArgs& s, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  const cudaError_t e = sort_config<kCtas>(stream, &cfg, attr);
  if (e == cudaSuccess) return cudaLaunchKernelEx(&cfg, embedding_sort_kernel<kCtas>, s);
  if (kCtas <= 8) return e;
  cudaGetLastError();
  return launch_sort<(kCtas > 8 ? 8 : kCtas)>(s, stream);
}

template <typename S, typename O>
int grad_as(const Tokens& k, int64_t D, const void* dY, int64_t lddy, void* dW, int64_t lddw,
            float scale, float beta, const GradPlan& g, char* ws, const CallContext& ctx,
            cudaStream_t stream) {
  const int sms = ctx.sm_count;
  const GradArgs<S, O> a{static_cast<const S*>(dY), lddy,  static_cast<O*>(dW), lddw, D, scale, beta,
                         rows_on(dW, lddw, sizeof(O), 16), ctx.err};
  const bool any = !rows_on(dY, lddy, sizeof(S), sum_values<S, O>() * sizeof(S));
  // the rows without tokens: about 32 KB a block at least, two blocks an SM at most
  // (each looks at all tokens)
  const int64_t row_bytes = D * static_cast<int64_t>(sizeof(O));
  int64_t share = (32768 + row_bytes - 1) / row_bytes;
  const int64_t even = (k.V + static_cast<int64_t>(sms) * 2 - 1) / (static_cast<int64_t>(sms) * 2);
  if (share < even) share = even;
  const int64_t rest = beta == 1.0f ? 0 : (k.V + share - 1) / share;
  if (g.few) {
    const int64_t blocks = k.T * g.slices + rest;
    if (blocks == 0) return GEMM14_OK;
    if (blocks > INT32_MAX) return GEMM14_ERR_INVALID_ARG;
    const auto kernel =
        any ? embedding_grad_few_kernel<S, O, true> : embedding_grad_few_kernel<S, O, false>;
    return finish_launch(launch_kernel(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads),
                                       0, stream, a, k, g.slices, share),
                         "embedding gradient launch", stream);
  }
  SortArgs s{};
  s.k = k;
  for (int i = 0; i < 2; ++i) s.list[i] = reinterpret_cast<uint2*>(ws + g.place_off[i]);
  s.count = reinterpret_cast<uint32_t*>(ws + g.count_off);
  s.bits = g.bits;
  s.passes = g.passes;
  s.err = ctx.err;
  int st = finish_launch(g.ctas == 1   ? launch_sort<1>(s, stream)
                         : g.ctas == 8 ? launch_sort<8>(s, stream)
                                       : launch_sort<16>(s, stream),
                         "embedding sort launch", stream);
  if (st != GEMM14_OK) return st;
  if (rest) {
    st = finish_launch(
        launch_kernel(embedding_rest_kernel<O>, dim3(static_cast<unsigned>(rest)),
                      dim3(kRestThreads), 0, stream, Rest<O>{a.dW, lddw, D, beta}, k, share),
        "embedding gradient launch", stream);
    if (st != GEMM14_OK) return st;
  }
  const int last = (g.passes - 1) & 1;
  const Ranges r{s.list[last], s.count, reinterpret_cast<uint32_t*>(ws + g.list_off),
                 reinterpret_cast<float*>(ws + g.slots_off), g.slot_ld, g.ranges, g.along, g.slices};
  const auto sum = any || !a.words ? embedding_sum_kernel<S, O, kAnywhere>
                   : beta == 0.0f  ? embedding_sum_kernel<S, O, kWordsSet>
                                   : embedding_sum_kernel<S, O, kWordsAdd>;
  st = finish_launch(launch_kernel(sum, dim3(static_cast<unsigned>(g.blocks)), dim3(kThreads), 0,
                                   stream, a, r, k.T, k.V),
                     "embedding gradient launch", stream);
  if (st != GEMM14_OK) return st;
  if (g.ranges == 1) return GEMM14_OK;
  const int64_t items = g.ranges * ((D + 127) / 128), most = static_cast<int64_t>(sms) * 4;
  return finish_launch(
      launch_kernel(embedding_join_kernel<O>, dim3(static_cast<unsigned>(items < most ? items : most)),
                    dim3(kThreads), 0, stream, a.dW, lddw, D, scale, beta, r, k.V, ctx.err),
      "embedding gradient launch", stream);
}

bool element_type(int dtype) {
  return dtype == GEMM14_DTYPE_F32 || dtype == GEMM14_DTYPE_BF16 || dtype == GEMM14_DTYPE_F16;
}

// Sizes, tokens and the two matrices of either call; `in` has rows_in rows, `out` rows_out.
int validate(int dtype_in, int dtype_out, int64_t T, int64_t V, int64_t D, const void* tokens,
             int token_bytes, int64_t rows_in, const void* in, int64_t ld_in, int64_t rows_out,
             const void* out, int64_t ld_out) {
  if (!element_type(dtype_in) || !element_type(dtype_out)) return GEMM14_ERR_INVALID_ARG;
  if (token_bytes != 4 && token_bytes != 8) return GEMM14_ERR_INVALID_ARG;
  if (T < 0 || T > kTrainMaxSize || V < 1 || V > kTrainMaxSize || D < 1 || D > kTrainMaxSize)
    return GEMM14_ERR_INVALID_ARG;
  if (ld_in < D || ld_out < D) return GEMM14_ERR_INVALID_ARG;
  if (T > 0 && (!tokens || !aligned(tokens, token_bytes))) return GEMM14_ERR_INVALID_ARG;
  if ((rows_in > 0 && !in) || (rows_out > 0 && !out)) return GEMM14_ERR_INVALID_ARG;
  if (!aligned(in, elem_bytes_of(dtype_in)) || !aligned(out, elem_bytes_of(dtype_out)))
    return GEMM14_ERR_INVALID_ARG;
  return GEMM14_OK;
}

bool finite(float x) { return x - x == 0.0f; }

template <typename S>
cudaError_t lookup_from(int dtype_out, const void* W, int64_t ldw, const Tokens& k, void* out,
                        int64_t ldo, int64_t D, float scale, int sms, cudaStream_t stream) {
  switch (dtype_out) {
    case GEMM14_DTYPE_BF16:
      return lookup_as<S, __nv_bfloat16>(W, ldw, k, out, ldo, D, scale, sms, stream);
    case GEMM14_DTYPE_F16: return lookup_as<S, __half>(W, ldw, k, out, ldo, D, scale, sms, stream);
    default: return lookup_as<S, float>(W, ldw, k, out, ldo, D, scale, sms, stream);
  }
}

}  // namespace
}  // namespace gemm14

using namespace gemm14;

extern "C" {

int gemm14_embedding_forward(int dtype, int dtype_out, int64_t T, int64_t V, int64_t D,
                             const void* W, int64_t ldw, const void* tokens, int token_bytes,
                             int64_t ignore_index, float scale, void* out, int64_t ldo,
                             void* stream_ptr) {
  int st = validate(dtype, dtype_out, T, V, D, tokens, token_bytes, V, W, ldw, T, out, ldo);
  if (st != GEMM14_OK) return st;
  if (!finite(scale)) return GEMM14_ERR_INVALID_ARG;
  if (T == 0) return GEMM14_OK;
  int sms = 0;
  if ((st = current_sm_count(&sms)) != GEMM14_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  const Tokens k{tokens, token_bytes == 8, T, V, ignore_index};
  const cudaError_t e =
      dtype == GEMM14_DTYPE_BF16
          ? lookup_from<__nv_bfloat16>(dtype_out, W, ldw, k, out, ldo, D, scale, sms, stream)
      : dtype == GEMM14_DTYPE_F16
          ? lookup_from<__half>(dtype_out, W, ldw, k, out, ldo, D, scale, sms, stream)
          : lookup_from<float>(dtype_out, W, ldw, k, out, ldo, D, scale, sms, stream);
  return finish_launch(e, "embedding launch", stream);
}

size_t gemm14_embedding_backward_workspace_bytes(int dtype, int dtype_out, int64_t T, int64_t V,
                                                 int64_t D, int sm_count) {
  if (sm_count <= 0 && current_sm_count(&sm_count) != GEMM14_OK) return 0;
  if (!element_type(dtype) || !element_type(dtype_out) || T < 0 || T > kTrainMaxSize || V < 1 || V > kTrainMaxSize || D < 1 ||
      D > kTrainMaxSize)
    return 0;
  GradPlan g;
  grad_plan(dtype, dtype_out, T, V, D, sm_count, &g);
  return g.total;
}

int gemm14_embedding_backward(int dtype, int dtype_out, int64_t T, int64_t V, int64_t D,
                              const void* dY, int64_t lddy, const void* tokens, int token_bytes,
                              int64_t ignore_index, float scale, float beta, void* dW, int64_t lddw,
                              void* workspace, size_t workspace_bytes, void* stream_ptr) {
  int st = validate(dtype, dtype_out, T, V, D, tokens, token_bytes, T, dY, lddy, V, dW, lddw);
  if (st != GEMM14_OK) return st;
  if (dtype_out != dtype && dtype_out != GEMM14_DTYPE_F32) return GEMM14_ERR_INVALID_ARG;
  if (!finite(scale) || !finite(beta)) return GEMM14_ERR_INVALID_ARG;
  if (workspace && !aligned(workspace, 16)) return GEMM14_ERR_INVALID_ARG;
  CallContext ctx;
  if ((st = call_device(&ctx)) != GEMM14_OK) return st;
  GradPlan g;
  grad_plan(dtype, dtype_out, T, V, D, ctx.sm_count, &g);
  if (g.total && (!workspace || workspace_bytes < g.total)) {
    note_error("gemm14_embedding_backward: %zu bytes of workspace given, %zu needed",
               workspace_bytes, g.total);
    return GEMM14_ERR_INVALID_ARG;
  }
  const Tokens k{tokens, token_bytes == 8, T, V, ignore_index};
  char* ws = static_cast<char*>(workspace);
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  const bool same = dtype_out == dtype;
  switch (dtype) {
    case GEMM14_DTYPE_BF16:
      return same ? grad_as<__nv_bfloat16, __nv_bfloat16>(k, D, dY, lddy, dW, lddw, scale, beta, g,
                                                          ws, ctx, stream)
                  : grad_as<__nv_bfloat16, float>(k, D, dY, lddy, dW, lddw, scale, beta, g, ws, ctx,
                                                  stream);
    case GEMM14_DTYPE_F16:
      return same ? grad_as<__half, __half>(k, D, dY, lddy, dW, lddw, scale, beta, g, ws, ctx, stream)
                  : grad_as<__half, float>(k, D, dY, lddy, dW, lddw, scale, beta, g, ws, ctx, stream);
    default:
      return grad_as<float, float>(k, D, dY, lddy, dW, lddw, scale, beta, g, ws, ctx, stream);
  }
}

}  // extern "C"
