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
constexpr int kAhead = 4;

template <typename S, typename O>
__host__ __device__ constexpr int lookup_values() {
  return 16 / static_cast<int>(sizeof(S) > sizeof(O) ? sizeof(S) : sizeof(O));
}

template <typename S, typename O, bool kAny>
__global__ void __launch_bounds__(kThreads)
    embedding_kernel(const S* W, int64_t ldw, const Tokens k, O* out, int64_t ldo, int64_t D,
                     float scale, int along) {
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
  if constexpr (sizeof(S) == sizeof(O)) {
    if (!words)
      return launch_kernel(embedding_kernel<S, O, true>, dim3(grid_for(k.T * along, sms)),
                           dim3(kThreads), 0, stream, w, ldw, k, o, ldo, D, scale, along);
  }
  return launch_kernel(embedding_kernel<S, O, false>, dim3(grid_for(k.T * along, sms)),
                       dim3(kThreads), 0, stream, w, ldw, k, o, ldo, D, scale, along);
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
  constexpr int kPer = 16 / static_cast<int>(sizeof(S));
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
// warp has a range of the list: it counts its digits (places of one digit found
// with match.any), the counts are summed over warps and CTAs (through
// distributed shared memory) to each warp's first position for each digit, and
// the warp goes through its range again and moves the places there, in order.
// Two passes for up to 2^18 tokens; the list lies in L2. The first pass leaves
// out what takes no part.
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int kSortAhead = 8;  // words in flight a lane

struct SortArgs {
  Tokens k;
  uint32_t* key[2];  // of the sorted places: their tokens ...
  uint32_t* at[2];   // ... and which they are
  uint32_t* count;   // how many take part
  int bits, passes;  // digits of this many bits
  unsigned* err;
};

constexpr size_t kSortSmem = (static_cast<size_t>(kSortWarps) * kDigits + 2 * kDigits + 32) * 4;

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
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = kCtas > 1 ? cluster_ctarank() : 0u;
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t T = static_cast<uint32_t>(a.k.T);
  uint32_t n = T;
  uint32_t* my_hist = hist + warp * kDigits;
  for (int pass = 0; pass < a.passes; ++pass) {
    const uint32_t* key_in = a.key[(pass + 1) & 1];
    const uint32_t* at_in = a.at[(pass + 1) & 1];
    uint32_t* key_out = a.key[pass & 1];
    uint32_t* at_out = a.at[pass & 1];
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
    uint32_t key[kSortAhead];
    const auto load = [&](uint32_t i0) {
#pragma unroll
      for (int u = 0; u < kSortAhead; ++u) {
        const uint32_t i = i0 + u * 32u + lane;
        key[u] = ~0u;
        if (i >= end) continue;
        if (pass == 0) {
          const int64_t token = token_at(a.k, i);
          if (takes_part(a.k, token)) key[u] = static_cast<uint32_t>(token);
        } else {
          key[u] = __ldcg(key_in + i);
        }
      }
    };
    // lanes of this lane's digit, and those before it among them
    const auto peers_of = [&](uint32_t k) {
      return __match_any_sync(0xffffffffu, k == ~0u ? ~0u : (k >> shift) & mask);
    };
    for (uint32_t i0 = begin; i0 < end; i0 += kSortAhead * 32u) {
      load(i0);
#pragma unroll
      for (int u = 0; u < kSortAhead; ++u) {
        if (i0 + u * 32u >= end) break;
        const uint32_t peers = peers_of(key[u]);
        if (key[u] != ~0u && lane == __ffs(peers) - 1)
          my_hist[(key[u] >> shift) & mask] += __popc(peers);
        __syncwarp();
      }
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
      for (uint32_t c = 0; c < kCtas; ++c) {
        const uint32_t v =
            kCtas > 1 ? load_cluster_u32(mapa_shared(smem_u32(total + tid), c)) : total[tid];
        all += v;
        if (c < rank) before += v;
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
      uint32_t at[kSortAhead];
#pragma unroll
      for (int u = 0; u < kSortAhead; ++u) {
        const uint32_t i = i0 + u * 32u + lane;
        at[u] = pass == 0 ? i : i < end ? __ldcg(at_in + i) : 0u;
      }
#pragma unroll
      for (int u = 0; u < kSortAhead; ++u) {
        if (i0 + u * 32u >= end) break;
        const uint32_t peers = peers_of(key[u]);
        const uint32_t digit = (key[u] >> shift) & mask;
        const bool on = key[u] != ~0u;
        uint32_t first = 0;
        if (on) first = base[digit] + my_hist[digit];
        __syncwarp();
        if (on && lane == __ffs(peers) - 1) my_hist[digit] += __popc(peers);
        __syncwarp();
        if (on) {
          const uint32_t to = first + __popc(peers & ((1u << lane) - 1u));
          if (dev_check(index_ok(to, T), a.err)) {
            key_out[to] = key[u];
            at_out[to] = at[u];
          }
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
  if (rank == 0 && tid == 0) *a.count = n;
}

// ---- sums over ranges of the sorted places

// A group of `along` threads takes one range of the sorted places and a slice of
// the columns, kPer of them a thread (16 bytes of dY's type), kRowsAhead rows in
// flight. Each token's sum that begins and ends in the range goes to dW; what a
// range holds of a sum that began before it, or goes on behind it, goes to the
// range's first or second slot, for the join.
struct Ranges {
  const uint32_t* key;
  const uint32_t* at;
  const uint32_t* count;
  float* slots;       // two rows of slot_ld floats a range
  int64_t slot_ld;
  int64_t ranges;
  int along, slices;
};
constexpr uint32_t kLeastRange = 8;

// Places of a range: all ranges but the last hold as many.
__device__ __forceinline__ uint32_t range_length(uint32_t n, int64_t ranges) {
  const uint32_t even = static_cast<uint32_t>((n + ranges - 1) / ranges);
  return max(kLeastRange, even);
}

template <typename S, typename O, bool kAny>
__global__ void __launch_bounds__(kThreads)
    embedding_sum_kernel(const GradArgs<S, O> a, const Ranges r, int64_t T, int64_t V) {
  constexpr int kPer = 16 / static_cast<int>(sizeof(S));
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t n = *r.count;
  const int tx = threadIdx.x & (r.along - 1), group = threadIdx.x / r.along;
  const int64_t part = blockIdx.x / r.slices;
  const int slice = static_cast<int>(blockIdx.x - part * r.slices);
  const int64_t range = part * (kThreads / r.along) + group;
  const uint32_t length = range_length(n, r.ranges);
  const int64_t c = (static_cast<int64_t>(slice) * r.along + tx) * kPer;
  if (range >= r.ranges || range * length >= n || c >= a.D) return;
  const uint32_t p0 = static_cast<uint32_t>(range) * length, p1 = min(n, p0 + length);
  const S* end = a.dY + (T - 1) * a.lddy + a.D;
  float sum[kPer] = {};
  uint32_t token = r.key[p0];
  bool began_before = p0 > 0 && r.key[p0 - 1] == token;
  const auto to_slot = [&](int which) {
    float* slot = r.slots + (2 * range + which) * r.slot_ld + c;
#pragma unroll
    for (int j = 0; j < kPer; j += 4)
      *reinterpret_cast<float4*>(slot + j) = make_float4(sum[j], sum[j + 1], sum[j + 2], sum[j + 3]);
  };
  const auto to_row = [&]() {
    if (dev_check(index_ok(token, V), a.err))
      put_sums<O, kPer>(a.dW + token * a.lddw, c, a.D, sum, a.scale, a.beta, a.words != 0);
  };
  for (uint32_t p = p0; p < p1; p += kRowsAhead) {
    uint32_t key[kRowsAhead];
    Pack<S, kPer> x[kRowsAhead];
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      if (p + u >= p1) continue;
      key[u] = r.key[p + u];
      x[u] = load_pack<S, kPer, kAny>(a.dY + static_cast<int64_t>(r.at[p + u]) * a.lddy, c, a.D,
                                      a.dY, end);
    }
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      if (p + u >= p1) continue;
      if (key[u] != token) {
        if (began_before)
          to_slot(0);
        else
          to_row();
        began_before = false;
        token = key[u];
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum[j] = 0.0f;
      }
      add_to<S, kPer>(sum, x[u]);
    }
  }
  if (began_before)
    to_slot(0);
  else if (p1 < n && r.key[p1] == token)
    to_slot(1);
  else
    to_row();
}

// The sums that lie in several ranges: the group of the range where one begins
// adds what the later ranges hold of it, in order.
template <typename S, typename O>
__global__ void __launch_bounds__(kThreads)
    embedding_join_kernel(const GradArgs<S, O> a, const Ranges r, int64_t V) {
  constexpr int kPer = 16 / static_cast<int>(sizeof(S));
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t n = *r.count;
  const int tx = threadIdx.x & (r.along - 1), group = threadIdx.x / r.along;
  const int64_t part = blockIdx.x / r.slices;
  const int slice = static_cast<int>(blockIdx.x - part * r.slices);
  const int64_t range = part * (kThreads / r.along) + group;
  const uint32_t length = range_length(n, r.ranges);
  const int64_t c = (static_cast<int64_t>(slice) * r.along + tx) * kPer;
  if (range >= r.ranges || (range + 1) * length >= n || c >= a.D) return;
  const uint32_t p0 = static_cast<uint32_t>(range) * length, p1 = p0 + length;
  const uint32_t token = r.key[p1];
  if (r.key[p1 - 1] != token || (r.key[p0] == token && p0 > 0 && r.key[p0 - 1] == token)) return;
  float sum[kPer];
  const auto add_slot = [&](int64_t i, bool first) {
    const float* slot = r.slots + i * r.slot_ld + c;
#pragma unroll
    for (int j = 0; j < kPer; j += 4) {
      const float4 v = *reinterpret_cast<const float4*>(slot + j);
      sum[j] = first ? v.x : sum[j] + v.x;
      sum[j + 1] = first ? v.y : sum[j + 1] + v.y;
      sum[j + 2] = first ? v.z : sum[j + 2] + v.z;
      sum[j + 3] = first ? v.w : sum[j + 3] + v.w;
    }
  };
  add_slot(2 * range + 1, true);
  for (int64_t i = range + 1; i * length < n && r.key[i * length] == token; ++i) add_slot(2 * i, false);
  if (dev_check(index_ok(token, V), a.err))
    put_sums<O, kPer>(a.dW + token * a.lddw, c, a.D, sum, a.scale, a.beta, a.words != 0);
}

// ---- the call's plan

struct GradPlan {
  bool few = false;        // one launch, no workspace
  int along = 8, slices = 1, ctas = 1;
  int bits = 1, passes = 1;
  int64_t ranges = 1, slot_ld = 0, blocks = 1;
  size_t key_off[2] = {}, at_off[2] = {}, count_off = 0, slots_off = 0, total = 0;
};

void grad_plan(int dtype, int64_t T, int64_t V, int64_t D, int sms, GradPlan* g) {
  const int per = 16 / elem_bytes_of(dtype);
  const int64_t pieces = (D + per - 1) / per;
  if (T <= kFewTokens) {
    g->few = true;
    g->slices = static_cast<int>((pieces + kThreads - 1) / kThreads);
    return;
  }
  while (g->along < kThreads && g->along < pieces) g->along *= 2;
  g->slices = static_cast<int>((pieces + g->along - 1) / g->along);
  const int groups = kThreads / g->along;
  // as many ranges as are resident at once (4 blocks an SM), of 8 places at least
  const int64_t most = (T + kLeastRange - 1) / kLeastRange;
  g->ranges = static_cast<int64_t>(sms) * 4 * groups / g->slices;
  if (g->ranges < 1) g->ranges = 1;
  if (g->ranges > most) g->ranges = most;
  g->blocks = (g->ranges + groups - 1) / groups * g->slices;
  g->slot_ld = pieces * per;
  int width = 1;
  while (width < 31 && (V - 1) >> width) ++width;
  g->passes = (width + kDigitBits - 1) / kDigitBits;
  g->bits = (width + g->passes - 1) / g->passes;
  g->ctas = T <= 2048 ? 1 : 8;
  size_t at = streamk_flag_bytes(sms);
  const auto take = [&](size_t bytes) {
    const size_t o = at;
    at += round256(bytes);
    return o;
  };
  g->count_off = take(4);
  for (int i = 0; i < 2; ++i) {
    g->key_off[i] = take(static_cast<size_t>(T) * 4);
    g->at_off[i] = take(static_cast<size_t>(T) * 4);
  }
  g->slots_off = take(static_cast<size_t>(g->ranges) * 2 * g->slot_ld * 4);
  g->total = at;
}

template <int kCtas>
cudaError_t launch_sort(const SortArgs& s, cudaStream_t stream) {
  static DeviceOnce configured;
  const cudaError_t e = set_smem_once(configured, embedding_sort_kernel<kCtas>, kSortSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kCtas);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = kSortSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, embedding_sort_kernel<kCtas>, s);
}

template <typename S, typename O>
int grad_as(const Tokens& k, int64_t D, const void* dY, int64_t lddy, void* dW, int64_t lddw,
            float scale, float beta, const GradPlan& g, char* ws, const CallContext& ctx,
            cudaStream_t stream) {
  const int sms = ctx.sm_count;
  const GradArgs<S, O> a{static_cast<const S*>(dY), lddy,  static_cast<O*>(dW), lddw, D, scale, beta,
                         rows_on(dW, lddw, sizeof(O), 16), ctx.err};
  const bool any = !rows_on(dY, lddy, sizeof(S), 16);
  // the rows without tokens: about 32 KB a block at least, four blocks an SM at most
  const int64_t row_bytes = D * static_cast<int64_t>(sizeof(O));
  int64_t share = (32768 + row_bytes - 1) / row_bytes;
  const int64_t even = (k.V + static_cast<int64_t>(sms) * 4 - 1) / (static_cast<int64_t>(sms) * 4);
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
  for (int i = 0; i < 2; ++i) {
    s.key[i] = reinterpret_cast<uint32_t*>(ws + g.key_off[i]);
    s.at[i] = reinterpret_cast<uint32_t*>(ws + g.at_off[i]);
  }
  s.count = reinterpret_cast<uint32_t*>(ws + g.count_off);
  s.bits = g.bits;
  s.passes = g.passes;
  s.err = ctx.err;
  int st = finish_launch(g.ctas == 1 ? launch_sort<1>(s, stream) : launch_sort<8>(s, stream),
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
  const Ranges r{s.key[last],   s.at[last], s.count, reinterpret_cast<float*>(ws + g.slots_off),
                 g.slot_ld,     g.ranges,   g.along, g.slices};
  const auto sum = any ? embedding_sum_kernel<S, O, true> : embedding_sum_kernel<S, O, false>;
  st = finish_launch(launch_kernel(sum, dim3(static_cast<unsigned>(g.blocks)), dim3(kThreads), 0,
                                   stream, a, r, k.T, k.V),
                     "embedding gradient launch", stream);
  if (st != GEMM14_OK) return st;
  return finish_launch(launch_kernel(embedding_join_kernel<S, O>,
                                     dim3(static_cast<unsigned>(g.blocks)), dim3(kThreads), 0,
                                     stream, a, r, k.V),
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

size_t gemm14_embedding_backward_workspace_bytes(int dtype, int64_t T, int64_t V, int64_t D,
                                                 int sm_count) {
  if (sm_count <= 0 && current_sm_count(&sm_count) != GEMM14_OK) return 0;
  if (!element_type(dtype) || T < 0 || T > kTrainMaxSize || V < 1 || V > kTrainMaxSize || D < 1 ||
      D > kTrainMaxSize)
    return 0;
  GradPlan g;
  grad_plan(dtype, T, V, D, sm_count, &g);
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
  grad_plan(dtype, T, V, D, ctx.sm_count, &g);
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
