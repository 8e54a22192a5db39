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
#include <type_traits>

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
// (a second rounding, of a product that is right to 2^-24); where nothing
// changes, words are moved as they are.
// kAny: rows at any address; the pieces are then the aligned words of the
// output's row, the table's are read as two words and a shift, and the elements
// before and behind them go one by one.
// An output that L2 cannot hold is stored past it, so that the table's rows that
// recur stay there (rows of 4096 bf16: 8192 of them, 67 MB, 12.9 us so and 15.4 without,
// 65536 120.6 and 127.1; below it the output may be there for its reader: 4096 of them,
// 33 MB, and a sum of it 21.1 and 20.2).
constexpr int kAhead = 4;
constexpr double kStreamBytes = 64e6;
enum : int { kStreamOut = 1, kCopy = 2 };  // flags of a lookup

template <typename S, typename O>
__host__ __device__ constexpr int lookup_values() {
  return 16 / static_cast<int>(sizeof(S) > sizeof(O) ? sizeof(S) : sizeof(O));
}

template <typename S, typename O, bool kAny>
__global__ void __launch_bounds__(kThreads)
    embedding_kernel(const S* W, int64_t ldw, const Tokens k, O* out, int64_t ldo, int64_t D,
                     float scale, int along, int flags) {
  constexpr int kPer = lookup_values<S, O>();
  using WordS = decltype(Pack<S, kPer>().raw);
  using WordO = decltype(Pack<O, kPer>().raw);
  grid_dependency_wait();
  grid_launch_dependents();
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
    const auto one = [&](int64_t c) { to[c] = from_f32<O>(real ? scale * to_f32(from[c]) : other); };
    int lead = 0;  // elements before the row's first aligned word
    if (kAny) {
      const int off = static_cast<int>(reinterpret_cast<uintptr_t>(to) & (kPer * sizeof(O) - 1)) /
                      static_cast<int>(sizeof(O));
      lead = static_cast<int>(min(D, static_cast<int64_t>((kPer - off) & (kPer - 1))));
    }
    const int64_t words = (D - lead) / kPer;
    const int tail = static_cast<int>(D - lead - words * kPer);
    if (kAny && real && words > 0 &&
        !(words_inside(from + lead, sizeof(WordS), W, end) &&
          words_inside(from + lead + (words - 1) * kPer, sizeof(WordS), W, end))) {
      // a row whose words reach past the table's ends
      for (int64_t c = tx; c < D; c += along) one(c);
      continue;
    }
    for (int64_t i0 = tx; i0 < words; i0 += static_cast<int64_t>(along) * kAhead) {
      const S* x = from + lead + i0 * kPer;
      O* y = to + lead + i0 * kPer;
      const int step = along * kPer;
      const int64_t here = words - i0;
      Pack<S, kPer> p[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (u * along >= here || !real) break;
        if constexpr (kAny)
          p[u].raw = load_word_any(x + u * step, WordS());
        else
          p[u].raw = *reinterpret_cast<const WordS*>(x + u * step);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (u * along >= here) break;
        Pack<O, kPer> q;
        bool copied = false;
        if constexpr (sizeof(S) == sizeof(O)) {
          if ((flags & kCopy) && real) {
            q.raw = p[u].raw;
            copied = true;
          }
        }
        if (!copied) {
#pragma unroll
          for (int j = 0; j < kPer; ++j)
            q.x[j] = from_f32<O>(real ? scale * to_f32(p[u].x[j]) : other);
        }
        if (flags & kStreamOut)
          __stcs(reinterpret_cast<WordO*>(y + u * step), q.raw);
        else
          *reinterpret_cast<WordO*>(y + u * step) = q.raw;
      }
    }
    if (tx < lead) one(tx);
    if (tx < tail) one(D - tail + tx);
  }
}

// Threads along a row of so many items, a power of two of 8 at least: as many as
// leave each `ahead` items, more where the rows are too few for the SMs.
int threads_along(int64_t rows, int64_t items, int ahead, int sms) {
  int x = 8;
  while (x < kThreads && static_cast<int64_t>(x) * ahead < items) x *= 2;
  while (x < kThreads && x < items && rows * x < static_cast<int64_t>(sms) * 512) x *= 2;
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
  const bool words = rows_on(W, ldw, sizeof(S), kPer * sizeof(S)) &&
                     rows_on(out, ldo, sizeof(O), kPer * sizeof(O));
  const int along = threads_along(k.T, (D + kPer - 1) / kPer, kAhead, sms);
  int flags = static_cast<double>(k.T) * D * sizeof(O) > kStreamBytes ? kStreamOut : 0;
  if (std::is_same<S, O>::value && scale == 1.0f) flags |= kCopy;
  return launch_kernel(words ? embedding_kernel<S, O, false> : embedding_kernel<S, O, true>,
                       dim3(grid_for(k.T * along, sms)), dim3(kThreads), 0, stream,
                       static_cast<const S*>(W), ldw, k, static_cast<O*>(out), ldo, D, scale, along,
                       flags);
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
        if (static_cast<uint64_t>(token[u] - begin) < static_cast<uint64_t>(rows) &&
            token[u] != k.ignore)
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
    float old[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) old[j] = beta != 0.0f && c + j < D ? to_f32(row[c + j]) : 0.0f;
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (c + j < D)
        row[c + j] = from_f32<O>(beta != 0.0f ? fmaf(beta, old[j], scale * sum[j]) : scale * sum[j]);
  }
}

template <typename S, int kPer>
__device__ __forceinline__ void add_to(float (&sum)[kPer], const Pack<S, kPer>& x) {
#pragma unroll
  for (int j = 0; j < kPer; ++j) sum[j] += to_f32(x.x[j]);
}

constexpr int kRowsAhead = 8;  // rows of dY in flight

// Columns a thread has: 16 bytes of dY's.
template <typename S>
__host__ __device__ constexpr int sum_values() { return 16 / static_cast<int>(sizeof(S)); }

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

// A few tokens: a block a place and a slice of the columns. The block of a token's
// first place lists all its places, in order, and sums their rows, groups of
// `along` threads a part of the list each (parts of 8 rows at least), the groups'
// sums added in order; the other places' blocks end at once. The blocks behind
// them write the rows without tokens. One launch, no workspace.
constexpr int kFewTokens = 1024;

template <typename S, typename O, bool kAny>
__global__ void __launch_bounds__(kThreads)
    embedding_grad_few_kernel(const GradArgs<S, O> a, const Tokens k, int along, int slices,
                              int64_t share) {
  constexpr int kPer = sum_values<S>(), kEach = kFewTokens / kThreads;
  constexpr int kWarps = kThreads / 32, kMarked = 8192;
  __shared__ uint32_t marks[kMarked / 32];
  __shared__ int places[kFewTokens];
  __shared__ int counts[kEach * kWarps];
  __shared__ float parts[kThreads * kPer];
  grid_dependency_wait();
  grid_launch_dependents();
  const int T = static_cast<int>(k.T), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (static_cast<int64_t>(blockIdx.x) >= static_cast<int64_t>(T) * slices) {
    const int64_t v0 = (blockIdx.x - static_cast<int64_t>(T) * slices) * share;
    write_rest(Rest<O>{a.dW, a.lddw, a.D, a.beta}, k, v0, min(k.V, v0 + share), marks, kMarked);
    return;
  }
  const int t = blockIdx.x / slices, slice = blockIdx.x - t * slices;
  const int64_t token = token_at(k, t);
  bool same[kEach], earlier = false;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = e * kThreads + tid;
    same[e] = i < T && token_at(k, i) == token;
    earlier = earlier || (same[e] && i < t);
  }
  if (__syncthreads_or(earlier) || !takes_part(k, token)) return;
  uint32_t mine[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    mine[e] = __ballot_sync(0xffffffffu, same[e]);
    if (lane == 0) counts[e * kWarps + warp] = __popc(mine[e]);
  }
  __syncthreads();
  // the counts before this warp's, and of all: a lane a count
  int before = lane < kEach * kWarps ? counts[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  const int n = __shfl_sync(0xffffffffu, before, 31);
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int at = e * kWarps + warp, base = __shfl_sync(0xffffffffu, before, at) - __popc(mine[e]);
    if (same[e]) places[base + __popc(mine[e] & ((1u << lane) - 1u))] = e * kThreads + tid;
  }
  __syncthreads();
  const int tx = tid & (along - 1), group = tid / along;
  const int64_t c = (static_cast<int64_t>(slice) * along + tx) * kPer;
  const int groups = min(kThreads / along, (n + kRowsAhead - 1) / kRowsAhead);
  const int share_of = (n + groups - 1) / groups;
  const int end = group < groups ? min(n, (group + 1) * share_of) : 0;
  const S* last = a.dY + (k.T - 1) * a.lddy + a.D;
  float sum[kPer] = {};
  if (c < a.D) {
    for (int i = group * share_of; i < end; i += kRowsAhead) {
      Pack<S, kPer> x[kRowsAhead];
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u)
        if (i + u < end)
          x[u] = load_pack<S, kPer, kAny>(a.dY + places[i + u] * a.lddy, c, a.D, a.dY, last);
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u)
        if (i + u < end) add_to<S, kPer>(sum, x[u]);
    }
  }
  if (groups > 1) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) parts[j * kThreads + tid] = sum[j];
    __syncthreads();
    for (int g = 1; g < groups && group == 0; ++g)
#pragma unroll
      for (int j = 0; j < kPer; ++j) sum[j] += parts[j * kThreads + g * along + tx];
  }
  if (group == 0 && c < a.D)
    put_sums<O, kPer>(a.dW + token * a.lddw, c, a.D, sum, a.scale, a.beta, a.words != 0);
}

// ---- the places sorted by token

// Up to kRanked places: each place's position is counted, the places of a lower
// token and the earlier ones of its own, T^2 comparisons over all SMs with no
// exchange between them. A block has 32 places, a lane each, and a warp every
// 32nd chunk of 32 tokens to compare them with. 5.5 us for 4096 places, where the
// radix sort below takes 12; 13.8 for 8192, where it takes 12 too. A whole call on rows
// of 64 columns takes 13.1 us so and 16.8 with the sort for 4096 places, 18.4 and 18.5
// for 5000, 19.9 and 18.5 for 6000.
constexpr int kRankThreads = 1024, kRanked = 4096;

__global__ void __launch_bounds__(kRankThreads)
    embedding_rank_kernel(const Tokens k, uint2* list, uint32_t* count) {
  __shared__ __align__(16) uint32_t tokens[kRanked];
  __shared__ uint32_t counts[kRankThreads];
  __shared__ uint32_t total;
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int T = static_cast<int>(k.T), chunks = (T + 31) / 32;
  if (tid == 0) total = 0u;
  __syncthreads();
  uint32_t valid = 0;
  for (int i = tid; i < chunks * 32; i += kRankThreads) {
    uint32_t v = ~0u;  // takes no part: above every token
    if (i < T) {
      const int64_t token = token_at(k, i);
      if (takes_part(k, token)) v = static_cast<uint32_t>(token);
    }
    tokens[i] = v;
    valid += v != ~0u;
  }
  valid = __reduce_add_sync(0xffffffffu, valid);
  if (lane == 0 && blockIdx.x == 0) atomicAdd(&total, valid);
  __syncthreads();
  const int own = blockIdx.x;
  const uint32_t mine = tokens[own * 32 + lane];
  uint32_t lower = 0;
  for (int chunk = warp; chunk < chunks; chunk += kRankThreads / 32) {
    const uint4* at = reinterpret_cast<const uint4*>(tokens + chunk * 32);
    if (chunk == own) {
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const uint32_t v = tokens[chunk * 32 + j];
        lower += v < mine || (v == mine && j < lane);
      }
    } else {
      const uint32_t below = mine + (chunk < own ? 1u : 0u);  // (for ~0u no position is used)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint4 v = at[j];
        lower += (v.x < below) + (v.y < below) + (v.z < below) + (v.w < below);
      }
    }
  }
  counts[tid] = lower;
  __syncthreads();
  if (warp == 0) {
    uint32_t to = 0;
#pragma unroll
    for (int w = 0; w < kRankThreads / 32; ++w) to += counts[w * 32 + lane];
    if (mine != ~0u) list[to] = make_uint2(mine, static_cast<uint32_t>(own * 32 + lane));
  }
  if (blockIdx.x == 0 && tid < 2) count[tid] = tid == 0 ? total : 0u;
}

// Radix sort, least significant digit first, of the places that take part, by
// one cluster of kCtas CTAs whose barriers are the hardware's. In a pass every
// warp has a range of the list: it counts its digits (shared-memory atomics on
// its own counts), the counts are summed over warps and CTAs (through
// distributed shared memory) to each warp's first position for each digit, and
// the warp goes through its range again and moves the places there, in order:
// a ballot for each bit of the digit finds the lanes that have the same one.
// Two passes for a vocabulary of up to 2^18; the first leaves out what takes no
// part. Between passes the list lies in L2. A pass takes some 5 us for its barriers
// and the sums alone: 13 us for 16384 places, 21 for 65536 (with the lanes of a
// digit from match.any, and a store for each of token and place, 44).
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int kSortAhead = 8;  // words in flight a lane

struct SortArgs {
  Tokens k;
  uint2* list[2];   // the sorted places: the token, and which place it is
  uint32_t* count;  // how many take part, and (count[1], set to 0) long sums
  int bits, passes;  // digits of this many bits
  unsigned* err;
};

// A cluster of 8 CTAs of 16 warps sorts up to kEightCtas places, 16 of them up to
// kHalfCtas, 16 of 32 warps more (5467 places: 12 us with 32 warps, 11 so; 65536: 21
// with 32, 22 with 16). A call on rows of 64 columns: 8192 places 18.9 us with 8 CTAs
// and 19.3 with 16, 12000 21.1 and 21.3, 16384 23.1 and 22.4, 24000 27.4 and 23.7.
constexpr int kEightCtas = 16384, kHalfCtas = 32768;
constexpr size_t sort_smem_bytes(int warps) {
  return (static_cast<size_t>(warps) * kDigits + 2 * kDigits + 32) * 4;
}

__device__ __forceinline__ uint32_t load_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

template <int kCtas, int kSortWarps>
__global__ void __launch_bounds__(kSortWarps * 32)
    embedding_sort_kernel(const SortArgs a) {
  extern __shared__ __align__(16) uint32_t sort_smem[];
  uint32_t* hist = sort_smem;                     // [warp][digit]
  uint32_t* total = hist + kSortWarps * kDigits;  // of this CTA, read by the others
  uint32_t* base = total + kDigits;
  uint32_t* sums = base + kDigits;                // of a warp's digits in the scan
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_ctarank();
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t T = static_cast<uint32_t>(a.k.T);
  uint32_t n = T;
  uint32_t* my_hist = hist + warp * kDigits;
  for (int pass = 0; pass < a.passes; ++pass) {
    const uint2* in = a.list[(pass + 1) & 1];
    uint2* out = a.list[pass & 1];
    const int shift = pass * a.bits;
    const uint32_t mask = (1u << a.bits) - 1u;
    const uint32_t per_cta = (n + kCtas - 1) / kCtas;
    const uint32_t per_warp = ((per_cta + kSortWarps - 1) / kSortWarps + 31u) & ~31u;
    const uint32_t cta_begin = min(n, rank * per_cta), cta_end = min(n, cta_begin + per_cta);
    const uint32_t begin = min(cta_end, cta_begin + warp * per_warp);
    const uint32_t end = min(cta_end, begin + per_warp);
    for (int i = tid; i < kSortWarps * kDigits / 4; i += kSortWarps * 32)
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
          const uint2 v = __ldcg(in + i);
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
    cluster_sync();
    uint32_t all = 0, before = 0;
    if (tid < kDigits) {
#pragma unroll
      for (int c = 0; c < kCtas; ++c) {
        const uint32_t v = load_cluster_u32(mapa_shared(smem_u32(total + tid), c));
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
    cluster_sync();
  }
  if (rank == 0 && tid < 2) a.count[tid] = tid == 0 ? n : 0u;
}

// ---- sums over ranges of the sorted places

// A group of `along` threads takes one range of the sorted places and a slice of
// the columns. A token of up to kWhole places is one range's, the one where it
// begins; the sum of a longer one may lie in several: what a range holds of a sum
// that began before it, or goes on behind it, goes to the range's first or second
// slot, and the range where it began goes on a list for the join.
struct Ranges {
  const uint2* place;  // sorted: token, place
  uint32_t* count;     // places, and long sums
  uint32_t* list;      // of the ranges where a sum begins that goes on behind them
  float* slots;        // two rows of slot_ld floats a range
  int64_t slot_ld;
  uint32_t ranges;
  int along, slices;
};
constexpr uint32_t kLeastRange = 8, kWhole = 16;

// Places of a range: all ranges but the last hold as many, before their ends move.
__device__ __forceinline__ uint32_t range_length(uint32_t n, uint32_t ranges) {
  return max(kLeastRange, (n + ranges - 1u) / ranges);
}
// Where a range that should begin at p does, from which of the places p - 16 ..
// p + 15 have p's token: at p, or behind the token that has places on both sides
// of p, if it has no more than kWhole.
__device__ __forceinline__ uint32_t moved(uint32_t p, uint32_t same) {
  const uint32_t before = static_cast<uint32_t>(__clz(static_cast<int>(~(same << 16))));  // <= 16
  const uint32_t after = static_cast<uint32_t>(__ffs(static_cast<int>(~(same >> 16))) - 1);
  return before == 0 || before + after > kWhole ? p : p + after;
}

// A thread's group of `along` threads, the places [p0, p1) of its range, its slice
// of the columns and its place there. All of a warp's lanes look for the ends of
// its groups' ranges, a place each.
struct Group {
  uint32_t range, p0, p1, most;  // most: places of the longest range of the warp's
  int slice, tx;
  bool began_before;  // the first sum, before the range
};
__device__ __forceinline__ Group group_of(const Ranges& r, uint32_t n) {
  Group g;
  const int lane = threadIdx.x & 31;
  const uint32_t part = blockIdx.x / static_cast<uint32_t>(r.slices);
  g.slice = static_cast<int>(blockIdx.x - part * r.slices);
  g.tx = threadIdx.x & (r.along - 1);
  g.range = part * (kThreads / r.along) + threadIdx.x / r.along;
  const uint32_t length = range_length(n, r.ranges);
  const uint32_t q0 = g.range < r.ranges ? min(n, g.range * length) : n;
  const uint32_t q1 = g.range < r.ranges ? min(n, g.range * length + length) : n;
  g.p0 = g.p1 = n;
  g.began_before = false;
  for (int from = 0; from < 32; from += r.along) {
    const uint32_t a0 = __shfl_sync(0xffffffffu, q0, from), a1 = __shfl_sync(0xffffffffu, q1, from);
    const int64_t i0 = static_cast<int64_t>(a0) - 16 + lane, i1 = static_cast<int64_t>(a1) - 16 + lane;
    const uint32_t t0 = i0 >= 0 && i0 < n ? r.place[i0].x : ~0u;
    const uint32_t t1 = i1 >= 0 && i1 < n ? r.place[i1].x : ~0u;
    const uint32_t s0 = __ballot_sync(0xffffffffu, t0 == __shfl_sync(0xffffffffu, t0, 16));
    const uint32_t s1 = __ballot_sync(0xffffffffu, t1 == __shfl_sync(0xffffffffu, t1, 16));
    if (r.along < 32 && (lane & ~(r.along - 1)) != from) continue;
    g.p0 = a0 < n ? moved(a0, a0 ? s0 : s0 & ~0xffffu) : n;
    g.p1 = a1 < n ? moved(a1, s1) : n;
    // a sum that goes on here is a long one, whose ranges' ends do not move
    g.began_before = g.p0 < g.p1 && g.p0 == a0 && (s0 >> 15 & 1u) && a0 > 0;
  }
  g.most = __reduce_max_sync(0xffffffffu, g.p1 - g.p0);
  return g;
}

// A stage of a range's places, one a lane (of each 32, or of the group's lanes):
// the token (kFlag: its sum goes on behind the range) and the place (kFlag: the
// last of its sum here).
constexpr uint32_t kFlag = 0x80000000u;
__device__ __forceinline__ uint2 places_of(const Ranges& r, const Group& g, uint32_t n, uint32_t q,
                                           int stage) {
  const uint32_t p = g.p0 + q + (threadIdx.x & (stage - 1));
  if (p >= g.p1) return make_uint2(0u, 0u);
  uint2 v = r.place[p];
  const bool same = p + 1 < n && r.place[p + 1].x == v.x;
  if (p + 1 == g.p1 && same) v.x |= kFlag;
  if (p + 1 == g.p1 || !same) v.y |= kFlag;
  return v;
}
__device__ __forceinline__ uint2 from_lane(const uint2& v, int lane, int stage) {
  return make_uint2(__shfl_sync(0xffffffffu, v.x, lane, stage),
                    __shfl_sync(0xffffffffu, v.y, lane, stage));
}

// bytes (at most 8 or 16) of kBytes from global to shared memory, zeros behind them.
template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, int bytes) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(from), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

constexpr int kSumBlocks = 4;  // resident of an SM

// Rows that start on 16 bytes. What bounds it is how much is in flight: a row's
// words go to shared memory by asynchronous copies, kDepth rows ahead, each
// thread's to a place of its own, so that it waits for nothing but its own copies;
// and where sums are added to rows that are there (kAdd), the old words of a sum
// that ends come with the row that ends it. (With the words in registers, 4 or 8
// rows loaded and then added, 65536 places of 2048 columns, bf16 added to fp32,
// took 165 us for 597 MB; 95 so,
// 6.3 TB/s.)
// kPieces: 16 bytes of dY's columns that a thread has; two where a row has enough
// for a warp, as a row costs a thread some forty instructions whatever it moves.
template <typename S, typename O, bool kAdd, int kPieces>
struct SumShape {
  static constexpr int kWords = kPieces * static_cast<int>(sizeof(O) / sizeof(S));
  static constexpr int kCols = 16 / static_cast<int>(sizeof(O));  // of a word: 16 bytes of dW's
  static constexpr int kRowBytes = kCols * static_cast<int>(sizeof(S));
  static constexpr int kBytes = kThreads * kWords * (kRowBytes + (kAdd ? 16 : 0));  // of a row
  static constexpr int kDepth = 49152 / kBytes < 8 ? 49152 / kBytes : 8;
  static constexpr int kSmem = kDepth * kBytes;
};
// Sums of the words that a thread adds, two values an instruction.
__device__ __forceinline__ void add_pair(uint64_t& sum, float a, float b) {
  asm("{\n\t.reg .b64 x;\n\tmov.b64 x, {%1, %2};\n\tadd.rn.f32x2 %0, %0, x;\n\t}"
      : "+l"(sum)
      : "f"(a), "f"(b));
}
__device__ __forceinline__ float2 pair(uint64_t sum) {
  return make_float2(__uint_as_float(static_cast<uint32_t>(sum)),
                     __uint_as_float(static_cast<uint32_t>(sum >> 32)));
}

template <typename S, typename O, bool kAdd, int kPieces>
__global__ void __launch_bounds__(kThreads, kSumBlocks)
    embedding_sum_kernel(const GradArgs<S, O> a, const Ranges r, int64_t V) {
  using Q = SumShape<S, O, kAdd, kPieces>;
  constexpr int kWords = Q::kWords, kCols = Q::kCols, kDepth = Q::kDepth;
  extern __shared__ __align__(16) unsigned char sum_smem[];
  __shared__ uint2 staged[kThreads * 2];  // two stages of places a lane
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t n = *r.count;
  const Group g = group_of(r, n);
  // the thread's words, `along` words apart
  const int64_t c = (static_cast<int64_t>(g.slice) * r.along * kWords + g.tx) * kCols;
  const int apart = r.along * kCols;
  const uint32_t length = c < a.D ? g.p1 - g.p0 : 0u;
  const S* from = a.dY + c;
  O* to = a.dW + c;
  float* slot = r.slots + 2 * static_cast<int64_t>(g.range) * r.slot_ld + c;
  unsigned char* rows = sum_smem + threadIdx.x * Q::kRowBytes;
  unsigned char* olds = sum_smem + kDepth * kWords * kThreads * Q::kRowBytes + threadIdx.x * 16;
  int left[kWords];  // columns of a word that there are
  bool all_there = true;
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    left[w] = static_cast<int>(max(int64_t(0), min(int64_t(kCols), a.D - c - w * apart)));
    all_there = all_there && left[w] == kCols;
  }
  // places of the range, two stages of them in shared memory, the next in a register
  const int stage = min(r.along, 32), in_stage = threadIdx.x & (stage - 1);
  uint2* places = staged + (threadIdx.x & ~(stage - 1)) * 2;
  const uint32_t ring = 2u * stage - 1u;
  places[in_stage] = places_of(r, g, n, 0, stage);
  places[stage + in_stage] = places_of(r, g, n, stage, stage);
  uint2 next = places_of(r, g, n, 2 * stage, stage);
  __syncwarp();

  const auto run = [&](auto whole) {
    constexpr bool kWhole_ = decltype(whole)::value;  // no word reaches past the columns
    const auto fetch = [&](uint32_t i, int at) {
      if (i < length) {
        const uint2 v = places[i & ring];
        const S* row = from + static_cast<int64_t>(v.y & ~kFlag) * a.lddy;
        const bool ends = kAdd && (v.y & kFlag) && !(v.x & kFlag) && dev_check(index_ok(v.x, V), a.err);
        const O* old = to + (ends ? v.x * a.lddw : 0);
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          if (!kWhole_ && left[w] == 0) break;
          copy_async<Q::kRowBytes>(smem_u32(rows + (at * kWords + w) * kThreads * Q::kRowBytes),
                                   row + w * apart,
                                   kWhole_ ? Q::kRowBytes : left[w] * static_cast<int>(sizeof(S)));
          if (ends)
            copy_async<16>(smem_u32(olds + (at * kWords + w) * kThreads * 16), old + w * apart,
                           kWhole_ ? 16 : left[w] * static_cast<int>(sizeof(O)));
        }
      }
      copy_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kDepth; ++i) fetch(i, i);
    uint64_t sum[kWords][kCols / 2] = {};  // two columns each
    bool began_before = g.began_before;
    int at = 0;  // the ring's place
#pragma unroll 1
    for (uint32_t i = 0; i < g.most; ++i) {
      copy_wait<kDepth - 1>();
      if (i < length) {
        const uint2 v = places[i & ring];
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          Pack<S, kCols> x;
          x.raw = *reinterpret_cast<const decltype(x.raw)*>(rows + (at * kWords + w) * kThreads *
                                                                       Q::kRowBytes);
#pragma unroll
          for (int k = 0; k < kCols; k += 2) add_pair(sum[w][k / 2], to_f32(x.x[k]), to_f32(x.x[k + 1]));
        }
        if (v.y & kFlag) {
          const bool part = began_before || (v.x & kFlag);
          float* s = began_before ? slot : slot + r.slot_ld;
          if (c == 0 && part && !began_before) r.list[atomicAdd(r.count + 1, 1u)] = g.range;
          const bool mine = !part && dev_check(index_ok(v.x, V), a.err);
          O* row = to + (mine ? v.x * a.lddw : 0);
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
            if (!kWhole_ && left[w] == 0) break;
            float p[kCols];
#pragma unroll
            for (int k = 0; k < kCols; k += 2) {
              const float2 two = pair(sum[w][k / 2]);
              p[k] = two.x;
              p[k + 1] = two.y;
              sum[w][k / 2] = 0;
            }
            if (part) {
#pragma unroll
              for (int k = 0; k < kCols; k += 4)
                *reinterpret_cast<float4*>(s + w * apart + k) =
                    make_float4(p[k], p[k + 1], p[k + 2], p[k + 3]);
            } else if (mine) {
              Pack<O, kCols> y;
              if (kAdd) {
                y.raw = *reinterpret_cast<const decltype(y.raw)*>(olds + (at * kWords + w) * kThreads * 16);
#pragma unroll
                for (int k = 0; k < kCols; ++k)
                  y.x[k] = from_f32<O>(a.beta == 1.0f ? fmaf(a.scale, p[k], to_f32(y.x[k]))
                                                      : fmaf(a.beta, to_f32(y.x[k]), a.scale * p[k]));
              } else {
#pragma unroll
                for (int k = 0; k < kCols; ++k) y.x[k] = from_f32<O>(a.scale * p[k]);
              }
              if (kWhole_ || left[w] == kCols) {
                *reinterpret_cast<decltype(y.raw)*>(row + w * apart) = y.raw;
              } else {
#pragma unroll
                for (int k = 0; k < kCols; ++k)
                  if (k < left[w]) row[w * apart + k] = y.x[k];
              }
            }
          }
          began_before = false;
        }
      }
      fetch(i + kDepth, at);
      at = at + 1 == kDepth ? 0 : at + 1;
      if (((i + 1) & (stage - 1)) == 0) {  // a stage is done: the one after the next takes its place
        __syncwarp();
        places[(i & ring & ~(stage - 1)) + in_stage] = next;
        next = places_of(r, g, n, i + 1 + 2 * stage, stage);
        __syncwarp();
      }
    }
  };
  if (__all_sync(0xffffffffu, all_there))
    run(std::true_type());
  else
    run(std::false_type());
}

// Rows of dY or dW at any address, the same way: a thread copies the aligned word
// that its columns begin in, and takes them from that and its neighbour's (a group's
// last lane copies a second one). A row of dW is moved a value a lane, side by side,
// from sums that the warp's lanes hand each other through shared memory. (With two
// words a lane loaded and shifted and 8 or 4 values of dW a lane moved one by one,
// 18826 places of 1258 columns, bf16, took 40 us, 27 so.) What bounds it is the issue of
// instructions: 42 million of a warp in 47 us for 24505 places of 1627 columns, fp16 into
// fp32, 72 % of what the SMs issue, DRAM at 23 %. A call on them takes 94 us, on 1632
// aligned columns 72.
struct AnyShape {
  static constexpr int kDepth = 8;
  static constexpr int kWords = kThreads + kThreads / 8;  // of a row; groups have 8 lanes at least
  static constexpr int kStaged = kThreads * 8 * 4;        // bytes of the sums that are handed on
  static constexpr int kSmem = kDepth * kWords * 16 + kStaged;
};
template <typename S>
__device__ __forceinline__ void copy_inside(uint4* to, const char* from, const char* begin,
                                            const char* end) {
  if (from >= begin) {
    const int64_t n = min(int64_t(16), max(int64_t(0), static_cast<int64_t>(end - from)));
    copy_async<16>(smem_u32(to), n > 0 ? from : begin - (reinterpret_cast<uintptr_t>(begin) & 15),
                   static_cast<int>(n));
  } else {  // the word that the buffer begins in
#pragma unroll 1
    for (int i = 0; i < 16 / static_cast<int>(sizeof(S)); ++i) {
      const char* p = from + i * sizeof(S);
      reinterpret_cast<S*>(to)[i] =
          p >= begin && p < end ? *reinterpret_cast<const S*>(p) : from_f32<S>(0.0f);
    }
  }
}

template <typename S, typename O>
__global__ void __launch_bounds__(kThreads, kSumBlocks)
    embedding_sum_any_kernel(const GradArgs<S, O> a, const Ranges r, int64_t T, int64_t V) {
  constexpr int kPer = sum_values<S>(), kDepth = AnyShape::kDepth;
  extern __shared__ __align__(16) unsigned char sum_smem[];
  uint4* words = reinterpret_cast<uint4*>(sum_smem);
  float* staged = reinterpret_cast<float*>(sum_smem + kDepth * AnyShape::kWords * 16) +
                  (threadIdx.x >> 5) * 32 * kPer;  // the warp's
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t n = *r.count;
  const Group g = group_of(r, n);
  const int lane = threadIdx.x & 31, stage = min(r.along, 32);
  const int64_t c = (static_cast<int64_t>(g.slice) * r.along + g.tx) * kPer;
  const uint32_t length = g.p1 - g.p0;
  const bool live = c < a.D, by_warp = r.along >= 32;
  const bool last_lane = (lane & (stage - 1)) == stage - 1;
  const char* begin = reinterpret_cast<const char*>(a.dY);
  const char* end = reinterpret_cast<const char*>(a.dY + (T - 1) * a.lddy + a.D);
  float* slot = r.slots + 2 * static_cast<int64_t>(g.range) * r.slot_ld + c;
  // a row's byte in its word where the thread's columns begin, in 32 bits
  const uint32_t low = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(a.dY + c));
  const uint32_t pitch = static_cast<uint32_t>(a.lddy * static_cast<int64_t>(sizeof(S)));
  const auto byte_of = [&](uint32_t at) { return (low + (at & ~kFlag) * pitch) & 15u; };
  // words of rows that others lie before and behind are all inside
  const uint32_t inner = a.lddy * static_cast<int64_t>(sizeof(S)) >= 32 && T > 2 ? static_cast<uint32_t>(T - 2) : 0u;
  const auto fetch = [&](uint32_t i, const uint2& v, int at) {
    if (i < length && c < a.D + kPer) {  // (a lane behind the last column: its neighbour's word)
      const uint32_t place = v.y & ~kFlag;
      const char* from = reinterpret_cast<const char*>(a.dY + static_cast<int64_t>(place) * a.lddy + c) - byte_of(v.y);
      uint4* to = words + at * AnyShape::kWords;
      if (place - 1u < inner) {
        copy_async<16>(smem_u32(to + threadIdx.x), from, 16);
        if (last_lane) copy_async<16>(smem_u32(to + kThreads + threadIdx.x / 8), from + 16, 16);
      } else {
        copy_inside<S>(to + threadIdx.x, from, begin, end);
        if (last_lane) copy_inside<S>(to + kThreads + threadIdx.x / 8, from + 16, begin, end);
      }
      if (a.beta != 0.0f && live && (v.y & kFlag) && !(v.x & kFlag) &&
          dev_check(index_ok(v.x, V), a.err))
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.dW + v.x * a.lddw + c));
    }
    copy_commit();
  };
  uint2 now = places_of(r, g, n, 0, stage), next = places_of(r, g, n, stage, stage);
#pragma unroll 1
  for (int i = 0; i < kDepth; ++i) fetch(i, from_lane(now, i, stage), i);
  float sum[kPer] = {};
  bool began_before = g.began_before;
  int at = 0, j = 0;  // the ring's place, the stage's
#pragma unroll 1
  for (uint32_t i = 0; i < g.most; ++i) {
    copy_wait<kDepth - 1>();
    __syncwarp();
    const uint2 v = from_lane(now, j, stage);
    if (i < length) {
      if (live) {
        const uint4* w = words + at * AnyShape::kWords;
        Pack<S, kPer> x;
        x.raw = shift16(w[threadIdx.x], w[last_lane ? kThreads + threadIdx.x / 8 : threadIdx.x + 1],
                        byte_of(v.y));
        add_to<S, kPer>(sum, x);
      }
      if (v.y & kFlag) {
        if (began_before || (v.x & kFlag)) {
          float* s = began_before ? slot : slot + r.slot_ld;
          if (c == 0 && !began_before) r.list[atomicAdd(r.count + 1, 1u)] = g.range;
          if (live) {
#pragma unroll
            for (int k = 0; k < kPer; k += 4)
              *reinterpret_cast<float4*>(s + k) =
                  make_float4(sum[k], sum[k + 1], sum[k + 2], sum[k + 3]);
          }
        } else if (!dev_check(index_ok(v.x, V), a.err)) {
        } else if (by_warp) {  // (all of the warp's lanes are here)
#pragma unroll
          for (int k = 0; k < kPer; k += 4)
            *reinterpret_cast<float4*>(staged + lane * kPer + k) =
                make_float4(sum[k], sum[k + 1], sum[k + 2], sum[k + 3]);
          __syncwarp();
          O* row = a.dW + v.x * a.lddw;
          const int64_t c0 = c - lane * kPer + lane;
          float old[kPer];
#pragma unroll
          for (int k = 0; k < kPer; ++k)
            old[k] = a.beta != 0.0f && c0 + 32 * k < a.D ? to_f32(row[c0 + 32 * k]) : 0.0f;
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            const float s = a.scale * staged[32 * k + lane];
            if (c0 + 32 * k < a.D)
              row[c0 + 32 * k] = from_f32<O>(a.beta != 0.0f ? fmaf(a.beta, old[k], s) : s);
          }
        } else if (live) {
          put_sums<O, kPer>(a.dW + v.x * a.lddw, c, a.D, sum, a.scale, a.beta, false);
        }
        began_before = false;
#pragma unroll
        for (int k = 0; k < kPer; ++k) sum[k] = 0.0f;
      }
    }
    __syncwarp();  // the row's words have been read, and the sums handed on
    const int ahead = j + kDepth;
    fetch(i + kDepth, ahead < stage ? from_lane(now, ahead, stage) : from_lane(next, ahead - stage, stage), at);
    at = at + 1 == kDepth ? 0 : at + 1;
    if (++j == stage) {
      j = 0;
      now = next;
      next = places_of(r, g, n, i + 1 + stage, stage);
    }
  }
}

// The sums that lie in several ranges, 128 columns of one an item. Where the items
// are few a block has one, whose warps add every eighth of its slots each, and then
// the warps' sums in order; else a warp has one, a block's being of different sums,
// and those of many slots are the block's all the same. (The list's order, which
// varies, decides nothing but who adds what.) A call on 65536 places of 256 tokens, 1024
// columns, takes 49.9 us so, 66.3 with no sum by a block, 51.2 with those of 12 slots.
constexpr uint32_t kManySlots = 48;

// Every `each`-th of slots 0 .. behind from the `from`-th; slot 0 is the first
// range's second one, slot k the first of the k-th range behind it. (The loads are
// unconditional, so that they are all in flight before the first is added.)
__device__ __forceinline__ float4 add_slots(const float* slots, int64_t ld, uint32_t behind,
                                            uint32_t from, uint32_t each) {
  constexpr int kEach = 8;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (uint32_t k0 = from; k0 <= behind; k0 += each * kEach) {
    float4 v[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const uint32_t k = min(k0 + u * each, behind);
      v[u] = *reinterpret_cast<const float4*>(slots + (2 * static_cast<int64_t>(k) + (k == 0)) * ld);
    }
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const bool on = k0 + u * each <= behind;
      s.x += on ? v[u].x : 0.0f;
      s.y += on ? v[u].y : 0.0f;
      s.z += on ? v[u].z : 0.0f;
      s.w += on ? v[u].w : 0.0f;
    }
  }
  return s;
}

template <typename O>
__global__ void __launch_bounds__(kThreads)
    embedding_join_kernel(O* dW, int64_t lddw, int64_t D, float scale, float beta, const Ranges r,
                          int64_t V, unsigned* err) {
  constexpr int kWarps = kThreads / 32, kTests = 4;
  __shared__ float4 sums[kWarps][32];
  __shared__ uint32_t many[kWarps][4];  // the warp's item, [0] 0: it is done
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t n = r.count[0], listed = r.count[1];
  const uint32_t length = range_length(n, r.ranges);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t slices = (D + 127) / 128, items = listed * slices;
  const auto put = [&](uint32_t token, int64_t c, const float4& s) {
    const float all[4] = {s.x, s.y, s.z, s.w};
    if (c < D && dev_check(index_ok(token, V), err))
      put_sums<O, 4>(dW + token * lddw, c, D, all, scale, beta, false);
  };
  const auto slots_of = [&](uint32_t range, int64_t c) {
    return r.slots + 2 * static_cast<int64_t>(range) * r.slot_ld + (c < r.slot_ld ? c : 0);
  };
  // places of the sum that begins in a range: the token, and the ranges behind it
  // that begin within the sum
  const auto behind_of = [&](uint32_t range, uint32_t token) {
    uint32_t behind = 0;
    for (bool more = true; more;) {
      uint32_t in[kTests];
#pragma unroll
      for (int u = 0; u < kTests; ++u) {
        const int64_t i = static_cast<int64_t>(range + 1 + behind + 32 * u + lane) * length;
        in[u] = __ballot_sync(0xffffffffu, i < n && r.place[i].x == token);
      }
#pragma unroll
      for (int u = 0; u < kTests; ++u) {
        if (more) behind += __popc(in[u]);
        more = more && in[u] == ~0u;
      }
    }
    return behind;
  };
  const auto by_block = [&](uint32_t range, uint32_t token, uint32_t behind, int64_t c) {
    sums[warp][lane] = add_slots(slots_of(range, c), r.slot_ld, behind, warp, kWarps);
    __syncthreads();
    if (warp == 0) {
      float4 s = sums[0][lane];
#pragma unroll
      for (int k = 1; k < kWarps; ++k) {
        const float4 v = sums[k][lane];
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
      put(token, c, s);
    }
    __syncthreads();
  };
  const bool few = items <= 2 * static_cast<int64_t>(gridDim.x);
  const int each = few ? 1 : kWarps;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * each; base < items;
       base += static_cast<int64_t>(gridDim.x) * each) {
    const int64_t item = few ? base : base + warp;
    uint32_t behind = 0, range = 0, token = 0;
    int64_t c = 0;
    if (item < items) {
      const int64_t slice = item / listed;
      c = slice * 128 + lane * 4;
      range = r.list[item - slice * listed];
      token = r.place[(range + 1) * length].x;
      behind = behind_of(range, token);
    }
    if (few) {
      by_block(range, token, behind, c);
      continue;
    }
    if (item < items && behind < kManySlots)
      put(token, c, add_slots(slots_of(range, c), r.slot_ld, behind, 0u, 1u));
    if (lane == 0) {
      many[warp][0] = behind < kManySlots ? 0u : behind;
      many[warp][1] = range;
      many[warp][2] = token;
      many[warp][3] = static_cast<uint32_t>(c / 128);  // (lane 0's is the slice's first)
    }
    __syncthreads();
    for (int w = 0; w < kWarps; ++w)
      if (many[w][0] != 0u)
        by_block(many[w][1], many[w][2], many[w][0], static_cast<int64_t>(many[w][3]) * 128 + lane * 4);
    __syncthreads();
  }
}

// ---- the call's plan

struct GradPlan {
  bool few = false;        // one launch, no workspace
  int pieces = 1;          // 16 bytes of a row of dY that a thread has
  int along = 8, slices = 1, ctas = 0;  // ctas of the sort (0: the places are ranked)
  int bits = 1, passes = 1;
  int64_t ranges = 1, slot_ld = 0, blocks = 1;
  size_t place_off[2] = {}, count_off = 0, list_off = 0, slots_off = 0, total = 0;
};

// pieces: as many as the rows allow (see SumShape).
void grad_plan(int dtype, int pieces, int64_t T, int64_t V, int64_t D, int sms, GradPlan* g) {
  const int per = 16 / elem_bytes_of(dtype) * pieces;
  const int64_t items = (D + per - 1) / per;  // threads of a row
  g->pieces = pieces;
  g->few = T <= kFewTokens;
  // groups of a quarter of a block, where a token may have many places
  const int widest = g->few && T > kThreads ? kThreads / 4 : kThreads;
  while (g->along < widest && g->along < items) g->along *= 2;
  // a warp's time for a row is the same whatever its lanes have: as few idle as may be
  const auto threads = [&](int along) { return (items + along - 1) / along * along; };
  for (int x = g->along; !g->few && x > 32; x /= 2)
    if (threads(x / 2) < threads(g->along)) g->along = x / 2;
  g->slices = static_cast<int>((items + g->along - 1) / g->along);
  if (g->few) return;
  const int groups = kThreads / g->along;
  // as many ranges as are resident at once, of 8 places at least; twice as many, of
  // 16, where the vocabulary has more tokens than that: a range of frequent tokens
  // writes few rows and is done early (65536 places of 2048 columns, bf16 added to
  // fp32: 139 us a call with one wave of ranges, 130 with two; a vocabulary of 256,
  // whose sums lie in many ranges each: 47 with one, 73 with two)
  const int64_t most = (T + kLeastRange - 1) / kLeastRange;
  g->ranges = std::max<int64_t>(1, static_cast<int64_t>(sms) * kSumBlocks / g->slices) * groups;
  if (2 * g->ranges <= V && 2 * g->ranges <= T / 16) g->ranges *= 2;
  if (g->ranges > most) g->ranges = most;
  g->blocks = (g->ranges + groups - 1) / groups * g->slices;
  g->slot_ld = (D + 7) / 8 * 8;
  int width = 1;
  while (width < 31 && (V - 1) >> width) ++width;
  g->ctas = T <= kRanked ? 0 : T <= kEightCtas ? 8 : 16;
  g->passes = g->ctas ? (width + kDigitBits - 1) / kDigitBits : 1;
  g->bits = (width + g->passes - 1) / g->passes;
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
// Two pieces a thread where rows of one type start on 16 bytes and fill a warp so.
int pieces_for(int dtype, int dtype_out, int64_t T, int64_t D, bool words) {
  const int per = 16 / elem_bytes_of(dtype);
  return words && T > kFewTokens && dtype == dtype_out && D >= 64 * per ? 2 : 1;
}

// Clusters of 16 are not portable: whether this device runs one, else 8 do.
template <int kCtas, int kSortWarps>
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
  cfg->blockDim = dim3(kSortWarps * 32);
  cfg->dynamicSmemBytes = sort_smem_bytes(kSortWarps);
  cfg->stream = stream;
  cfg->attrs = attr;
  cfg->numAttrs = 2;
  return static_cast<cudaError_t>(configured.get(
      dev,
      [&] {
        cudaError_t r = cudaFuncSetAttribute(embedding_sort_kernel<kCtas, kSortWarps>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(cfg->dynamicSmemBytes));
        if (r == cudaSuccess && kCtas > 8)
          r = cudaFuncSetAttribute(embedding_sort_kernel<kCtas, kSortWarps>,
                                   cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        int fit = 1;
        if (r == cudaSuccess && kCtas > 8)
          r = cudaOccupancyMaxActiveClusters(&fit, embedding_sort_kernel<kCtas, kSortWarps>, cfg);
        if (r == cudaSuccess && fit < 1) r = cudaErrorInvalidConfiguration;
        return static_cast<int>(r);
      },
      [](int r) { return r == static_cast<int>(cudaSuccess) ||
                       r == static_cast<int>(cudaErrorInvalidConfiguration); }));
}
template <int kCtas, int kSortWarps>
cudaError_t launch_sort(const SortArgs& s, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  const cudaError_t e = sort_config<kCtas, kSortWarps>(stream, &cfg, attr);
  if (e == cudaSuccess) return cudaLaunchKernelEx(&cfg, embedding_sort_kernel<kCtas, kSortWarps>, s);
  if (kCtas <= 8) return e;
  cudaGetLastError();
  return launch_sort<(kCtas > 8 ? 8 : kCtas), kSortWarps>(s, stream);
}

template <typename S, typename O, bool kAdd, int kPieces>
cudaError_t launch_sum(const GradArgs<S, O>& a, const Ranges& r, int64_t V, dim3 blocks,
                       cudaStream_t stream) {
  static DeviceOnce configured;
  constexpr int kSmem = SumShape<S, O, kAdd, kPieces>::kSmem;
  const cudaError_t e = set_smem_once(configured, embedding_sum_kernel<S, O, kAdd, kPieces>, kSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(embedding_sum_kernel<S, O, kAdd, kPieces>, blocks, dim3(kThreads), kSmem,
                       stream, a, r, V);
}

template <typename S, typename O>
cudaError_t launch_sum_any(const GradArgs<S, O>& a, const Ranges& r, int64_t T, int64_t V,
                           dim3 blocks, cudaStream_t stream) {
  static DeviceOnce configured;
  const cudaError_t e = set_smem_once(configured, embedding_sum_any_kernel<S, O>, AnyShape::kSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(embedding_sum_any_kernel<S, O>, blocks, dim3(kThreads), AnyShape::kSmem,
                       stream, a, r, T, V);
}

template <typename S, typename O>
int grad_as(const Tokens& k, int64_t D, const void* dY, int64_t lddy, void* dW, int64_t lddw,
            float scale, float beta, const GradPlan& g, char* ws, const CallContext& ctx,
            cudaStream_t stream) {
  const int sms = ctx.sm_count;
  const GradArgs<S, O> a{static_cast<const S*>(dY), lddy,  static_cast<O*>(dW), lddw, D, scale, beta,
                         rows_on(dW, lddw, sizeof(O), 16), ctx.err};
  const bool any_dy = !rows_on(dY, lddy, sizeof(S), 16), any = any_dy || !a.words;
  // the rows without tokens: blocks of four times the bytes of the tokens, which
  // each looks at, and 32 KB at least; two blocks an SM at most where that is more
  const int64_t row_bytes = D * static_cast<int64_t>(sizeof(O));
  const int64_t even = (k.V + static_cast<int64_t>(sms) * 2 - 1) / (static_cast<int64_t>(sms) * 2);
  const int64_t share =
      std::max<int64_t>(1, std::min(even, std::max<int64_t>(32768, 32 * k.T) / row_bytes + 1));
  const int64_t rest = beta == 1.0f ? 0 : (k.V + share - 1) / share;
  if (g.few) {
    const int64_t blocks = k.T * g.slices + rest;
    if (blocks == 0) return GEMM14_OK;
    if (blocks > INT32_MAX) return GEMM14_ERR_INVALID_ARG;
    const auto kernel =
        any_dy ? embedding_grad_few_kernel<S, O, true> : embedding_grad_few_kernel<S, O, false>;
    return finish_launch(launch_kernel(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads),
                                       0, stream, a, k, g.along, g.slices, share),
                         "embedding gradient launch", stream);
  }
  SortArgs s{};
  s.k = k;
  for (int i = 0; i < 2; ++i) s.list[i] = reinterpret_cast<uint2*>(ws + g.place_off[i]);
  s.count = reinterpret_cast<uint32_t*>(ws + g.count_off);
  s.bits = g.bits;
  s.passes = g.passes;
  s.err = ctx.err;
  const cudaError_t e =
      g.ctas == 0 ? launch_kernel(embedding_rank_kernel, dim3(static_cast<unsigned>((k.T + 31) / 32)),
                                  dim3(kRankThreads), 0, stream, k, s.list[0], s.count)
      : g.ctas == 8        ? launch_sort<8, 16>(s, stream)
      : k.T <= kHalfCtas ? launch_sort<16, 16>(s, stream)
                         : launch_sort<16, 32>(s, stream);
  int st = finish_launch(e, "embedding sort launch", stream);
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
                 reinterpret_cast<float*>(ws + g.slots_off), g.slot_ld,
                 static_cast<uint32_t>(g.ranges), g.along, g.slices};
  const dim3 blocks(static_cast<unsigned>(g.blocks));
  constexpr int kTwo = sizeof(O) == sizeof(S) ? 2 : 1;  // (of mixed types one is two words)
  const cudaError_t summed =
      any            ? launch_sum_any<S, O>(a, r, k.T, k.V, blocks, stream)
      : g.pieces > 1 ? beta == 0.0f ? launch_sum<S, O, false, kTwo>(a, r, k.V, blocks, stream)
                                    : launch_sum<S, O, true, kTwo>(a, r, k.V, blocks, stream)
      : beta == 0.0f ? launch_sum<S, O, false, 1>(a, r, k.V, blocks, stream)
                     : launch_sum<S, O, true, 1>(a, r, k.V, blocks, stream);
  st = finish_launch(summed, "embedding gradient launch", stream);
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

size_t gemm14_embedding_backward_workspace_bytes(int dtype, int64_t T, int64_t V, int64_t D,
                                                 int sm_count) {
  if (sm_count <= 0 && current_sm_count(&sm_count) != GEMM14_OK) return 0;
  if (!element_type(dtype) || T < 0 || T > kTrainMaxSize || V < 1 || V > kTrainMaxSize || D < 1 ||
      D > kTrainMaxSize)
    return 0;
  // rows may start anywhere or not, and the gradient be of either type
  size_t most = 0;
  for (int pieces = 1; pieces <= 2; ++pieces) {
    GradPlan g;
    grad_plan(dtype, pieces, T, V, D, sm_count, &g);
    most = std::max(most, g.total);
  }
  return most;
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
  const bool words = rows_on(dY, lddy, elem_bytes_of(dtype), 16) &&
                     rows_on(dW, lddw, elem_bytes_of(dtype_out), 16);
  GradPlan g;
  grad_plan(dtype, pieces_for(dtype, dtype_out, T, D, words), T, V, D, ctx.sm_count, &g);
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
