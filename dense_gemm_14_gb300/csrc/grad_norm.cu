// grad_norm.cu -- the norm of many gradients taken together (and of each), and
// the gradients scaled so that it stays within a limit:
//     N = |scale| sqrt(sum over tensors and elements of g^2),
//     f = scale min(1, max_norm / N),    out = f g.
// One reading of the gradients for the norm, one reading and one writing for
// the scaling: memory-bound, so the whole list goes in one launch a pass,
// however many tensors it has, and the factor never leaves the device.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <memory>
#include <new>

#include "../../include/gemm14.h"
#include "api_internal.h"
#include "checks.h"
#include "elements.cuh"
#include "kernels.h"
#include "plan.h"
#include "ptx.cuh"

namespace gemm14 {
namespace {

// A tensor of the list as the kernels see it: rows of `cols` elements (a dense
// one is a single row). Its elements are numbered in units of kUnitBytes of the
// source, which a warp takes at a time; the list's units are numbered through.
struct Entry {
  const void* src;
  void* dst;
  int64_t rows, cols, ld_src, ld_dst;
  uint32_t first_unit;
  uint16_t type, dst_type;  // gemm14 dtypes
};
// Passed by value: the kernels' parameters hold up to 32764 bytes. start, of the
// longest: the tensor of each block's first unit (a search for it would wait for
// one miss of the constant cache after another).
constexpr int kMostBlocks = 640;
constexpr int kMostEntries = 544;  // of a launch
template <int kN>
struct Table {
  static constexpr bool kStarts = kN == kMostEntries;
  int n;
  uint32_t units;
  bool in_place;  // every output is its gradient
  uint16_t start[kStarts ? kMostBlocks : 1];
  Entry e[kN];
};
// The tensor of unit u, of the block or one behind its first.
template <int kN>
__device__ __forceinline__ int tensor_of(const Table<kN>& t, uint32_t u) {
  if constexpr (Table<kN>::kStarts) {
    int i = t.start[blockIdx.x];
    while (i + 1 < t.n && t.e[i + 1].first_unit <= u) ++i;
    return i;
  } else {
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (t.e[mid].first_unit <= u)
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  }
}

constexpr int kUnitBytes = 4096;
constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 3;  // resident (4: 314 against 302 us for the norm of 1.1e9 bf16 values)
constexpr int kEach = 8;  // pieces of 16 bytes a lane has of a unit

__host__ __device__ inline int type_bytes(int type) { return type == GEMM14_DTYPE_F32 ? 4 : 2; }
__host__ __device__ inline int unit_shift(int type) { return type == GEMM14_DTYPE_F32 ? 10 : 11; }
__host__ __device__ inline int64_t unit_values(int type) { return int64_t(1) << unit_shift(type); }
static_assert((4 << 10) == kUnitBytes && (2 << 11) == kUnitBytes, "a unit's values");
// Units of a row of several (its first may begin up to 7 elements before an aligned
// word) and of a dense tensor (up to 63, before a line of 128 bytes: loads that
// straddle lines took 73 us for 109 packed tensors of 394 MB, 71 so), and the rows
// that share a unit.
__host__ __device__ inline int64_t row_units(int64_t cols, int type) {
  return (cols + 7 + unit_values(type) - 1) >> unit_shift(type);
}
__host__ __device__ inline int64_t unit_rows(int64_t cols, int type) {
  const int64_t r = unit_values(type) / (cols + 7);
  return r > 1 ? r : 1;
}
__host__ inline int64_t entry_units(const Entry& e) {
  if (e.rows == 1) return row_units(e.cols + 56, e.type);
  const int64_t u = row_units(e.cols, e.type);
  return u > 1 ? e.rows * u : (e.rows + unit_rows(e.cols, e.type) - 1) / unit_rows(e.cols, e.type);
}

// Warp w of `warps` takes the units [unit_at(w), unit_at(w + 1)); unit u is warp_of(u)'s.
__device__ __forceinline__ uint32_t unit_at(uint32_t units, uint32_t w, uint32_t warps) {
  return static_cast<uint32_t>(static_cast<uint64_t>(units) * w / warps);
}
__host__ inline uint32_t warp_of(uint32_t units, uint32_t u, uint32_t warps) {
  return static_cast<uint32_t>(((static_cast<uint64_t>(u) + 1) * warps - 1) / units);
}

// Where the sums of the list's tensors lie among the slots (sum_units below):
// tensor i's are [first[i], first[i + 1]).
template <int kN>
struct Parts {
  int n;
  uint32_t first[kN + 1];
};

// What a unit holds of its tensor: rows [row, row + rows) (more than one: whole
// rows, side by side), and of each the part-th stretch of unit_values elements,
// counted from the aligned word that holds the row's first element.
struct Unit {
  int64_t row, part;
  int rows;
};
// Elements between the boundary that units are counted from and a row's first.
template <typename T>
__device__ __forceinline__ int before_of(const Entry& e, const T* row, int bytes) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(row) & ((e.rows == 1 ? 128 : bytes) - 1)) /
         static_cast<int>(sizeof(T));
}
__device__ __forceinline__ Unit unit_of(const Entry& e, uint32_t u) {
  if (e.rows == 1) return Unit{0, u, 1};
  const int64_t per = row_units(e.cols, e.type);
  if (per > 1) {
    const int64_t row = u / per;
    return Unit{row, u - row * per, 1};
  }
  const int64_t share = unit_rows(e.cols, e.type), row = u * share;
  return Unit{row, 0, static_cast<int>(min(share, e.rows - row))};
}
// Lanes that share a row of a unit: all of them, or a power of two that its
// pieces do not fill twice.
__device__ __forceinline__ int lanes_along(const Unit& u, int64_t cols, int per) {
  if (u.rows == 1) return 32;
  int x = 1;
  while (x < 32 && x * per < cols + 7) x *= 2;
  return x;
}

// ---- sums of squares

// A lane squares and adds the values of a unit in fp32 (at most 64 of them),
// then adds that to its sum in fp64. Squares that leave what fp32 holds to 24
// bits (a sum above 2^120, or below 2^-120 and not 0) are formed again in fp64,
// from values read again: no value that the types have overflows or is lost, and
// the fp64 units see one addition for 32 or 64 values.
__device__ __forceinline__ float square_sum(float s, const Pack<float, 4>& p) {
#pragma unroll
  for (int j = 0; j < 4; ++j) s = fmaf(p.x[j], p.x[j], s);
  return s;
}
template <typename S>
__device__ __forceinline__ float square_sum(float s, const Pack<S, 8>& p) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = to_f32(p.x[j]);
    s = fmaf(x, x, s);
  }
  return s;
}

// s, the squares of the values c0, c0 + 1, .. (kPer of them), those `step` further, and
// so on, of [lo, hi), to the lane's sum; bits: what is set in any value.
template <typename S>
__device__ __forceinline__ void add_squares(double& sum, float s, uint32_t bits, const S* row,
                                            int64_t c0, int step, int64_t lo, int64_t hi) {
  constexpr int kPer = 16 / static_cast<int>(sizeof(S));
  if (s <= 0x1p120f && s >= 0x1p-120f) {
    sum += static_cast<double>(s);
  } else if (bits & (sizeof(S) == 4 ? 0x7fffffffu : 0x7fff7fffu)) {
#pragma unroll 1
    for (int64_t c = c0; c < hi; c += step) {
#pragma unroll 1
      for (int64_t j = max(c, lo); j < min(c + kPer, hi); ++j) {
        const double x = static_cast<double>(to_f32(row[j]));
        sum = fma(x, x, sum);
      }
    }
  }
}
__device__ __forceinline__ uint32_t bits_of(const uint4& v) { return v.x | v.y | v.z | v.w; }

// Of a stretch of a row from `from` (below 0 where the row begins in it) on: the
// elements [first, last) in whole pieces, those before and behind them (at most
// kPer - 1 each), which go one a lane. (With every piece looked at element by element
// the two such units of each of 109 tensors cost 7 us of 71.)
struct Stretch {
  int64_t first, last, end;
};
template <int kPer>
__device__ __forceinline__ Stretch stretch_of(int64_t from, int64_t values, int64_t cols) {
  Stretch t;
  t.end = min(from + values, cols);
  t.first = from < 0 ? min(t.end, from + (kPer - 1 - from) / kPer * kPer) : from;
  t.last = t.first + (t.end - t.first) / kPer * kPer;
  return t;
}

template <typename S>
__device__ __forceinline__ void add_unit(double& sum, const Entry& e, const Unit& u, int lane) {
  constexpr int kPer = 16 / static_cast<int>(sizeof(S));
  const S* row = static_cast<const S*>(e.src) + u.row * e.ld_src;
  if (u.rows == 1) {
    const int64_t from = u.part * unit_values(e.type) - before_of(e, row, 16);
    const int64_t c0 = from + lane * kPer;
    Pack<S, kPer> p[kEach];
    Stretch t{from, from + unit_values(e.type), 0};
    if (from >= 0 && t.last <= e.cols) {  // a whole unit
#pragma unroll
      for (int i = 0; i < kEach; ++i) p[i].raw = *reinterpret_cast<const uint4*>(row + c0 + i * 32 * kPer);
    } else {
      t = stretch_of<kPer>(from, unit_values(e.type), e.cols);
      const double x = from < 0 && lane < t.first ? static_cast<double>(to_f32(row[lane])) : 0.0;
      const double y =
          t.last + lane < t.end ? static_cast<double>(to_f32(row[t.last + lane])) : 0.0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int64_t c = c0 + i * 32 * kPer;
        p[i].raw = make_uint4(0u, 0u, 0u, 0u);
        if (c >= t.first && c < t.last) p[i].raw = *reinterpret_cast<const uint4*>(row + c);
      }
      sum = fma(x, x, fma(y, y, sum));
    }
    float s[4] = {};
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      s[i & 3] = square_sum(s[i & 3], p[i]);
      bits |= bits_of(p[i].raw);
    }
    add_squares(sum, (s[0] + s[1]) + (s[2] + s[3]), bits, row, c0, 32 * kPer, t.first, t.last);
    return;
  }
  const int along = lanes_along(u, e.cols, kPer), lx = lane & (along - 1);
  for (int r = lane / along; r < u.rows; r += 32 / along) {
    const S* at = row + r * e.ld_src;
    const int64_t c0 = lx * kPer - before_of(e, at, 16);
    float s = 0.0f;
    uint32_t bits = 0;
#pragma unroll 4
    for (int64_t c = c0; c < e.cols; c += along * kPer) {
      const Pack<S, kPer> p = load_pack<S, kPer, false>(at, c, e.cols, nullptr, nullptr);
      s += square_sum(0.0f, p);
      bits |= bits_of(p.raw);
    }
    add_squares(sum, s, bits, at, c0, along * kPer, int64_t(0), e.cols);
  }
}

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Warp w's units, in order. What they hold of tensor i goes to slot w + i: where
// a warp or a tensor ends, the next sum's slot is one further, so that a tensor's
// slots lie side by side, in order. (Where both end at once a slot is left over,
// and is set to 0.)
template <int kN>
__device__ __forceinline__ void sum_units(const Table<kN>& t, uint32_t w, uint32_t warps, int lane,
                                          double* slots) {
  // what the parameters say comes before the wait for the kernel before this one
  const bool any = w < warps;
  const uint32_t u0 = any ? unit_at(t.units, w, warps) : 0u;
  const uint32_t u1 = any ? unit_at(t.units, w + 1, warps) : 0u;
  int i = any ? tensor_of(t, u0) : 0;
  grid_dependency_wait();
  grid_launch_dependents();
  if (!any) return;
  if (lane == 0 && w > 0 && i > 0 && t.e[i].first_unit == u0) slots[w + i - 1] = 0.0;
  for (uint32_t u = u0; u < u1;) {
    const Entry& e = t.e[i];
    const uint32_t end = min(u1, i + 1 < t.n ? t.e[i + 1].first_unit : t.units);
    double sum = 0.0;
    for (; u < end; ++u) {
      const Unit at = unit_of(e, u - e.first_unit);
      if (e.type == GEMM14_DTYPE_BF16)
        add_unit<__nv_bfloat16>(sum, e, at, lane);
      else if (e.type == GEMM14_DTYPE_F16)
        add_unit<__half>(sum, e, at, lane);
      else
        add_unit<float>(sum, e, at, lane);
    }
    sum = warp_sum(sum);
    if (lane == 0) slots[w + i] = sum;
    if (u < u1) ++i;
  }
}

// ---- from the slots to the norms

struct Finish {
  const double* slots;
  double* totals;      // of the launches so far
  int launch;          // this one's number
  bool last;
  float scale, max_norm;
  float* norm;         // written by the last launch
  float* each;         // of this launch's tensors, or NULL
  double* factor;      // for the scaling, or NULL
};

// The root of s >= 0 (or NaN, infinite): sqrtf of s brought to [1, 4) by a power of
// 4, and one step of Newton's iteration r + (s - r^2) / (2 r), whose correction
// needs no more than fp32: right to some 2^-45, for a handful of fp64 operations in
// place of sqrt's (an SM does two a cycle, so one of a warp's takes 16).
__device__ __forceinline__ double root(double s) {
  if (!(s > 0.0) || s - s != 0.0) return s;
  const int k = ((__double2hiint(s) >> 20) - 1023) & ~1;  // (sums of squares are normal numbers)
  const double m = __hiloint2double(__double2hiint(s) - k * (1 << 20), __double2loint(s));
  const float r = sqrtf(static_cast<float>(m));
  const double rd = static_cast<double>(r);
  const float off = static_cast<float>(fma(-rd, rd, m));
  const double y = rd + static_cast<double>(off * (0.5f / r));
  return __hiloint2double(__double2hiint(y) + k / 2 * (1 << 20), __double2loint(y));
}

// Slots [a, b), every `step`-th from the `from`-th.
__device__ __forceinline__ double slot_sum(const double* slots, uint32_t a, uint32_t b,
                                           uint32_t from, uint32_t step) {
  double s = 0.0;
  for (uint32_t i0 = a + from; i0 < b; i0 += 4 * step) {
    double v[4];
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) v[k] = __ldcg(slots + min(i0 + k * step, b - 1));
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k)
      if (i0 + k * step < b) s += v[k];
  }
  return s;
}
// The sum over the threads of the block's first kFinishThreads, to its warp 0; in
// an order of its own. Every thread of the block calls it.
constexpr int kFinishThreads = 256, kFinishCtas = 8;
__device__ __forceinline__ double block_sum(double v, double* smem) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kWarps = kFinishThreads / 32;
  __syncthreads();
  if (warp < kWarps) {
    v = warp_sum(v);
    if (lane == 0) smem[warp] = v;
  }
  __syncthreads();
  double s = 0.0;
  if (warp == 0) {
    s = lane < kWarps ? smem[lane] : 0.0;
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  }
  return s;
}
__device__ __forceinline__ double load_cluster_f64(uint32_t addr) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
  return v;
}

// The norm of a sum of squares, and the factor that the gradients are scaled by.
// (The norm of finite values is finite here, and clips, also where fp32 has no number
// for it.)
__device__ __forceinline__ double factor_of(const Finish& f, double squares, double* norm) {
  *norm = root(squares) * fabs(static_cast<double>(f.scale));
  const bool over = *norm > static_cast<double>(f.max_norm) && *norm - *norm == 0.0;
  return over ? f.scale * (f.max_norm / *norm) : f.scale;
}

// The norm and the factor, by the first kFinishThreads threads of each CTA of a
// cluster of kFinishCtas, smem: 9 doubles of each.
__device__ __forceinline__ void finish_total(const Finish& f, uint32_t slots, double* smem) {
  const uint32_t rank = cluster_ctarank();
  double mine = 0.0;
  if (threadIdx.x < kFinishThreads)
    mine = slot_sum(f.slots, 0u, slots, rank * kFinishThreads + threadIdx.x,
                    kFinishCtas * kFinishThreads);
  mine = block_sum(mine, smem);
  if (threadIdx.x == 0) smem[kFinishThreads / 32] = mine;
  cluster_sync();
  if (rank == 0 && threadIdx.x < 32) {
    double total = 0.0;
    if (threadIdx.x < kFinishCtas)
      total = load_cluster_f64(mapa_shared(smem_u32(smem + kFinishThreads / 32), threadIdx.x));
#pragma unroll
    for (int o = kFinishCtas / 2; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (threadIdx.x == 0) {
      double all = total;
      for (int l = 0; l < f.launch; ++l) all += f.totals[l];
      f.totals[f.launch] = total;
      if (f.last) {
        double norm;
        const double factor = factor_of(f, all, &norm);
        *f.norm = static_cast<float>(norm);
        if (f.factor) *f.factor = factor;
      }
    }
  }
  cluster_sync();  // no CTA ends while its sum is read; the factor is written
}
// The norms of the tensors block, block + blocks, ..: a warp each, the block's first
// threads for one of many slots. (All of them by one block took 35 us for 109
// tensors.)
template <int kN>
__device__ __forceinline__ void finish_each(const Parts<kN>& t, const Finish& f, int block,
                                            int blocks, double* smem) {
  constexpr uint32_t kLong = 1024;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const auto put = [&](int i, double s) {
    f.each[i] = static_cast<float>(root(s) * fabs(static_cast<double>(f.scale)));
  };
  for (int i = block + warp * blocks; i < t.n; i += warps * blocks) {
    if (t.first[i + 1] - t.first[i] > kLong) continue;
    const double s = warp_sum(slot_sum(f.slots, t.first[i], t.first[i + 1], lane, 32u));
    if (lane == 0) put(i, s);
  }
  for (int i = block; i < t.n; i += blocks) {
    if (t.first[i + 1] - t.first[i] <= kLong) continue;
    double s = 0.0;
    if (threadIdx.x < kFinishThreads)
      s = slot_sum(f.slots, t.first[i], t.first[i + 1], threadIdx.x, kFinishThreads);
    s = block_sum(s, smem);
    if (threadIdx.x == 0) put(i, s);
  }
}

// ---- scaling

// A lane's pieces of a unit: kPer values each, 16 bytes of the source and 16 or 32
// aligned ones of the output, stored at once; the source's word, where it does not
// start on 16 bytes, is read as two and a shift. kEach of them are in flight.
// (As two stores of 16 bytes of fp32 output a clipping of 109 packed fp16 tensors of
// 197 million values takes 316 us, 264 so.)
// With nvcc 13.0 a store of 32 bytes, this one's or that of a ulonglong4_32a, wrote only
// its first element in a function that was not inlined; why is not known. So all that
// stand above one are inlined, and tests hold the build to that and look at every
// element that is stored, at each alignment.
// Products are rounded to fp32 and then to a 16-bit type: within half a step and
// 2^-24 of the value.
template <typename O, int kPer>
union Output {
  O x[kPer];
  uint32_t w[kPer * sizeof(O) / 4];
};
__device__ __forceinline__ void store_output(void* to, const uint32_t (&w)[4]) {
  *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_output(void* to, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
template <typename S, typename O, int kPer>
__device__ __forceinline__ Output<O, kPer> scaled(const Pack<S, kPer>& p, float f) {
  Output<O, kPer> y;
#pragma unroll
  for (int j = 0; j < kPer; ++j) y.x[j] = from_f32<O>(f * to_f32(p.x[j]));
  return y;
}

// The pieces [first, last) of a stretch from c0 on, 32 pieces apart a lane, whole
// units (kWhole) without a look at where they end. (The others' code, run for the
// units that a tensor begins and ends in, spills.)
template <typename S, typename O, bool kAny, bool kWhole>
__device__ __forceinline__ void scale_pieces(const S* src, O* dst, const S* begin, const S* end,
                                             int64_t c0, int64_t first, int64_t last, float f) {
  constexpr int kPer = 16 / static_cast<int>(sizeof(S));
  Pack<S, kPer> p[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int64_t c = c0 + i * 32 * kPer;
    if (!kWhole && (c < first || c >= last)) continue;
    if constexpr (kAny) {
      if (kWhole || words_inside(src + c, 16, begin, end))
        p[i].raw = load16_any(src + c);
      else
        p[i] = load_pack<S, kPer, true>(src, c, last, begin, end);
    } else {
      p[i].raw = *reinterpret_cast<const uint4*>(src + c);
    }
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int64_t c = c0 + i * 32 * kPer;
    if (!kWhole && (c < first || c >= last)) continue;
    store_output(dst + c, scaled<S, O, kPer>(p[i], f).w);
  }
}

template <typename S, typename O>
__device__ __forceinline__ void scale_unit(const Entry& e, const Unit& u, int lane, float f) {
  constexpr int kPer = 16 / static_cast<int>(sizeof(S));
  constexpr int kOut = kPer * static_cast<int>(sizeof(O));
  const S* begin = static_cast<const S*>(e.src);
  const S* end = begin + (e.rows - 1) * e.ld_src + e.cols;
  const S* src = begin + u.row * e.ld_src;
  O* dst = static_cast<O*>(e.dst) + u.row * e.ld_dst;
  if (u.rows == 1) {
    const int64_t from = u.part * unit_values(e.type) - before_of(e, dst, kOut);
    const int64_t c0 = from + lane * kPer, behind = from + unit_values(e.type);
    const bool words = (reinterpret_cast<uintptr_t>(src + from) & 15u) == 0;
    if (from >= 0 && behind <= e.cols) {
      if (words) {
        scale_pieces<S, O, false, true>(src, dst, begin, end, c0, from, behind, f);
        return;
      }
      if (words_inside(src + from, 16, begin, end) && words_inside(src + behind - kPer, 16, begin, end)) {
        scale_pieces<S, O, true, true>(src, dst, begin, end, c0, from, behind, f);
        return;
      }
    }
    const Stretch t = stretch_of<kPer>(from, unit_values(e.type), e.cols);
    const auto one = [&](int64_t c) { dst[c] = from_f32<O>(f * to_f32(src[c])); };
    if (from < 0 && lane < t.first) one(lane);
    if (t.last + lane < t.end) one(t.last + lane);
    if (words)
      scale_pieces<S, O, false, false>(src, dst, begin, end, c0, t.first, t.last, f);
    else
      scale_pieces<S, O, true, false>(src, dst, begin, end, c0, t.first, t.last, f);
    return;
  }
  const int along = lanes_along(u, e.cols, kPer), lx = lane & (along - 1);
  for (int r = lane / along; r < u.rows; r += 32 / along) {
    const S* x = src + r * e.ld_src;
    O* y = dst + r * e.ld_dst;
    const int64_t from = -before_of(e, y, kOut);
    const bool words = (reinterpret_cast<uintptr_t>(x + from) & 15u) == 0;
#pragma unroll 2
    for (int64_t c = from + lx * kPer; c < e.cols; c += along * kPer) {
      const Pack<S, kPer> p = words ? load_pack<S, kPer, false>(x, c, e.cols, begin, end)
                                    : load_pack<S, kPer, true>(x, c, e.cols, begin, end);
      const Output<O, kPer> q = scaled<S, O, kPer>(p, f);
      if (c >= 0 && c + kPer <= e.cols) {
        store_output(y + c, q.w);
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (c + j >= 0 && c + j < e.cols) y[c + j] = q.x[j];
      }
    }
  }
}

// A factor below fp32's normal numbers has fewer than 24 bits there, or is 0, while
// its products with large values are normal numbers: it is multiplied in fp64, an
// element at a time. Limits some 2^126 below the norm alone come here, so it stays out
// of the others' registers. (100 fp32 tensors of 419 MB into others, values of 1e37: 1038 us
// a call, 528 with a factor of 1e-11.)
__device__ __forceinline__ bool small_factor(double by) {
  const float f = static_cast<float>(by);
  return fabsf(f) < 0x1p-126f && static_cast<double>(f) != by;
}
template <typename S, typename O>
__device__ __forceinline__ void scale_small_as(const S* src, O* dst, int64_t n, int lane, double by) {
  for (int64_t c = lane; c < n; c += 32)
    dst[c] = from_f32<O>(static_cast<float>(by * static_cast<double>(to_f32(src[c]))));
}
__device__ __noinline__ void scale_small(const void* src, void* dst, int type, int dst_type,
                                         int64_t n, int lane, double by) {
  if (type == GEMM14_DTYPE_BF16) {
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(src);
    if (dst_type == GEMM14_DTYPE_F32)
      scale_small_as(x, static_cast<float*>(dst), n, lane, by);
    else
      scale_small_as(x, static_cast<__nv_bfloat16*>(dst), n, lane, by);
  } else if (type == GEMM14_DTYPE_F16) {
    const __half* x = static_cast<const __half*>(src);
    if (dst_type == GEMM14_DTYPE_F32)
      scale_small_as(x, static_cast<float*>(dst), n, lane, by);
    else
      scale_small_as(x, static_cast<__half*>(dst), n, lane, by);
  } else {
    scale_small_as(static_cast<const float*>(src), static_cast<float*>(dst), n, lane, by);
  }
}
// (Units are counted from a row's first element here, whatever its address: they are
// enough for that, and those left over are empty.)
__device__ __forceinline__ void scale_small_unit(const Entry& e, const Unit& u, int lane, double by) {
  const int64_t lo = min(e.cols, u.part * unit_values(e.type));
  const int64_t n = min(e.cols - lo, unit_values(e.type));
  for (int64_t r = u.row; r < u.row + u.rows; ++r)
    scale_small(static_cast<const char*>(e.src) + (r * e.ld_src + lo) * type_bytes(e.type),
                static_cast<char*>(e.dst) + (r * e.ld_dst + lo) * type_bytes(e.dst_type), e.type,
                e.dst_type, n, lane, by);
}
template <int kN>
__device__ __forceinline__ void scale_small_units(const Table<kN>& t, uint32_t w, uint32_t warps,
                                                  int lane, double by) {
  int i = 0;
  for (uint32_t u = w; u < t.units; u += warps) {
    while (i + 1 < t.n && t.e[i + 1].first_unit <= u) ++i;
    scale_small_unit(t.e[i], unit_of(t.e[i], u - t.e[i].first_unit), lane, by);
  }
}

// Every warps-th unit from the last down, so that the units at work at any time lie
// side by side: reads and writes of one stretch of memory each.
template <int kN>
__device__ __forceinline__ void scale_units(const Table<kN>& t, uint32_t w, uint32_t warps,
                                            int lane, double by) {
  if (small_factor(by)) {
    scale_small_units(t, w, warps, lane, by);
    return;
  }
  const float f = static_cast<float>(by);
  int i = t.n - 1;
  for (uint32_t left = t.units - w; left > 0; left = left > warps ? left - warps : 0u) {
    const uint32_t u = left - 1u;
    while (t.e[i].first_unit > u) --i;
    const Entry& e = t.e[i];
    if (e.src == e.dst && f == 1.0f) continue;  // nothing changes
    const Unit at = unit_of(e, u - e.first_unit);
    if (e.type == GEMM14_DTYPE_BF16) {
      if (e.dst_type == GEMM14_DTYPE_F32)
        scale_unit<__nv_bfloat16, float>(e, at, lane, f);
      else
        scale_unit<__nv_bfloat16, __nv_bfloat16>(e, at, lane, f);
    } else if (e.type == GEMM14_DTYPE_F16) {
      if (e.dst_type == GEMM14_DTYPE_F32)
        scale_unit<__half, float>(e, at, lane, f);
      else
        scale_unit<__half, __half>(e, at, lane, f);
    } else {
      scale_unit<float, float>(e, at, lane, f);
    }
  }
}

// ---- kernels

template <int kN>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    grad_sum_kernel(const __grid_constant__ Table<kN> t, uint32_t warps, double* slots) {
  sum_units(t, blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), warps, threadIdx.x & 31, slots);
}

// Clusters of kFinishCtas CTAs: the first has the norm, the others those of each.
template <int kN>
__global__ void __launch_bounds__(kFinishThreads)
    grad_finish_kernel(const __grid_constant__ Parts<kN> t, const Finish f) {
  __shared__ double smem[kFinishThreads / 32 + 1];
  grid_dependency_wait();
  grid_launch_dependents();
  if (blockIdx.x < kFinishCtas)
    finish_total(f, t.first[t.n], smem);
  else
    finish_each(t, f, blockIdx.x - kFinishCtas, gridDim.x - kFinishCtas, smem);
}

template <int kN>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    grad_scale_kernel(const __grid_constant__ Table<kN> t, uint32_t warps, const double* factor) {
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const double by = *factor;
  if (t.in_place && static_cast<float>(by) == 1.0f) return;  // nothing changes
  if (w < warps) scale_units(t, w, warps, threadIdx.x & 31, by);
}

// The scaling of a list of few units: each block forms the total itself, which costs
// no more than a launch of grad_finish_kernel does, and saves the host that launch
// (10 tensors of 8 MB: 17.6 us of the host in place so and 20.3 with it, 21.3 and 23.6
// into others; on the GPU alone 8.4 and 7.8, 11.8 and 10.5; of 2 MB 4.5 and 7.0, 7.2 and
// 8.8; of 16 MB 10.7 and 8.8, 14.7 and 12.1).
constexpr int64_t kFewUnits = 4096;
template <int kN>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    grad_total_scale_kernel(const __grid_constant__ Table<kN> t,
                            const __grid_constant__ Parts<kN> parts, uint32_t warps,
                            const Finish f) {
  static_assert(kThreads == kFinishThreads, "a block forms the total");
  __shared__ double smem[kFinishThreads / 32 + 1];
  __shared__ double factor;
  grid_dependency_wait();
  grid_launch_dependents();
  const double total =
      block_sum(slot_sum(f.slots, 0u, parts.first[parts.n], threadIdx.x, kThreads), smem);
  if (threadIdx.x == 0) {
    double norm;
    factor = factor_of(f, total, &norm);
    if (blockIdx.x == 0) *f.norm = static_cast<float>(norm);
  }
  if (f.each) finish_each(parts, f, blockIdx.x, gridDim.x, smem);
  __syncthreads();
  const double by = factor;
  if (t.in_place && static_cast<float>(by) == 1.0f) return;  // nothing changes
  const uint32_t w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (w < warps) scale_units(t, w, warps, threadIdx.x & 31, by);
}

// A short list: one cluster of kSmallCtas CTAs does all of it in one launch, its
// barriers between the passes.
constexpr int kSmallCtas = kFinishCtas, kSmallThreads = 1024, kSmallEntries = 72;
// 4 MB, and 1 MB where they are scaled too. What it saves is the host's time, which such
// calls from a program are bound by: 10 tensors of 1 MB take 13.9 us so and 15.5 as two
// launches, in place 14.6 and 17.1, into others 17.7 and 21.1; of 4 MB the norm 12.1 and
// 15.2. On the GPU alone, as in a graph's replays, the launches are faster: of 1 MB 8.4
// against 6.0 us for the norm, 9.0 against 4.7 in place, 12.0 against 7.0 into others; of
// 4 MB the norm 10.9 against 6.4.
constexpr int64_t kSmallUnits = 1024, kSmallScaled = 256;
template <int kN>
__global__ void __launch_bounds__(kSmallThreads, 1)
    grad_small_kernel(const __grid_constant__ Table<kN> t, const __grid_constant__ Parts<kN> parts,
                      uint32_t warps, double* slots, const Finish f) {
  __shared__ double smem[kFinishThreads / 32 + 1];
  const uint32_t w = blockIdx.x * (kSmallThreads / 32) + (threadIdx.x >> 5);
  sum_units(t, w, warps, threadIdx.x & 31, slots);
  cluster_sync();
  finish_total(f, parts.first[parts.n], smem);
  if (f.each) finish_each(parts, f, blockIdx.x, kSmallCtas, smem);
  if (!f.factor) return;
  if (w < warps) scale_units(t, w, warps, threadIdx.x & 31, __ldcg(f.factor));
}

// ---- the calls

// Bytes of the workspace: the launches' totals, the factor, a launch's slots.
struct Layout {
  size_t totals = 0, factor = 0, slots = 0, total = 0;
};
uint32_t most_warps(int sms) {
  return std::min(static_cast<uint32_t>(sms) * kBlocksPerSm, static_cast<uint32_t>(kMostBlocks)) *
         (kThreads / 32);
}
void layout(int64_t n, int sms, Layout* l) {
  const int64_t launches = (n + kMostEntries - 1) / kMostEntries;
  l->totals = streamk_flag_bytes(sms);
  l->factor = l->totals + round256(static_cast<size_t>(launches) * sizeof(double));
  l->slots = l->factor + 256;
  l->total = l->slots + round256((most_warps(sms) + static_cast<size_t>(kMostEntries)) * sizeof(double));
}

constexpr int64_t kMostTensors = int64_t(1) << 20;
constexpr int64_t kMostSize = int64_t(1) << 40, kMostSpan = int64_t(1) << 43;

bool dense(const gemm14_tensor& g) { return g.rows <= 1 || g.ld == g.cols; }
bool empty(const gemm14_tensor& g) { return g.rows == 0 || g.cols == 0; }

int validate_tensor(const gemm14_tensor& g) {
  if (g.dtype != GEMM14_DTYPE_F32 && g.dtype != GEMM14_DTYPE_BF16 && g.dtype != GEMM14_DTYPE_F16)
    return GEMM14_ERR_INVALID_ARG;
  if (g.rows < 0 || g.cols < 0 || g.rows > kMostSize || g.cols > kMostSize || g.ld > kMostSize)
    return GEMM14_ERR_INVALID_ARG;
  if (empty(g)) return GEMM14_OK;
  if (g.rows > 1 && (g.ld < g.cols || g.rows > kMostSpan / g.ld)) return GEMM14_ERR_INVALID_ARG;
  if (!g.data || !aligned(g.data, type_bytes(g.dtype))) return GEMM14_ERR_INVALID_ARG;
  return GEMM14_OK;
}

Entry entry_of(const gemm14_tensor& g, const gemm14_tensor* out) {
  Entry e{};
  e.type = static_cast<uint16_t>(g.dtype);
  e.dst_type = static_cast<uint16_t>(out ? out->dtype : g.dtype);
  e.rows = 1;  // an empty one is one unit with nothing in it
  if (empty(g)) return e;
  e.src = g.data;
  e.dst = out ? out->data : g.data;
  if (dense(g) && (!out || dense(*out))) {
    e.cols = g.rows * g.cols;
  } else {
    e.rows = g.rows;
    e.cols = g.cols;
    e.ld_src = g.ld;
    e.ld_dst = out ? out->ld : g.ld;
  }
  return e;
}

// ---- tensors that share memory

struct Span {
  uintptr_t begin, end;  // its first byte, and the byte after its last
  const gemm14_tensor* g;
  bool written;
  int64_t i;
};
// Whether two tensors whose spans cross share an element: not where the second lies
// between the first's rows, in one row or in several of the same pitch (columns of
// one matrix). Rows of another pitch between them count as shared.
bool share_elements(const Span& a, const Span& b) {
  const gemm14_tensor &x = *a.g, &y = *b.g;
  const int size = type_bytes(x.dtype);
  if (x.rows <= 1 || (y.rows > 1 && x.ld * size != y.ld * type_bytes(y.dtype))) return true;
  const int64_t pitch = x.ld * size, wide_x = x.cols * size, wide_y = y.cols * type_bytes(y.dtype);
  // b begins no earlier, and where it begins behind a row that is not a's last
  const int64_t off = static_cast<int64_t>(b.begin - a.begin) % pitch;
  return off < wide_x || off + wide_y > pitch;
}
// What is written may share no element with anything else of the lists, its own source aside.
int check_apart(int64_t n, const gemm14_tensor* grads, const gemm14_tensor* outs) {
  const int64_t most = outs ? 2 * n : n;
  std::unique_ptr<Span[]> s(new (std::nothrow) Span[static_cast<size_t>(most > 0 ? most : 1)]);
  if (!s) {
    note_error("gemm14_grad_clip: no host memory for %lld tensors", static_cast<long long>(n));
    return GEMM14_ERR_CUDA;
  }
  int64_t m = 0;
  const auto add = [&](const gemm14_tensor& g, bool written, int64_t i) {
    if (empty(g)) return;
    const uintptr_t b = reinterpret_cast<uintptr_t>(g.data);
    const int64_t values = (g.rows > 1 ? (g.rows - 1) * g.ld : 0) + g.cols;
    s[m++] = Span{b, b + static_cast<uintptr_t>(values * type_bytes(g.dtype)), &g, written, i};
  };
  for (int64_t i = 0; i < n; ++i) {
    const bool in_place = outs && !empty(grads[i]) && outs[i].data == grads[i].data &&
                          outs[i].dtype == grads[i].dtype &&
                          ((dense(outs[i]) && dense(grads[i])) || outs[i].ld == grads[i].ld);
    add(outs ? outs[i] : grads[i], true, i);
    if (outs && !in_place) add(grads[i], false, i);
  }
  const auto before = [](const Span& a, const Span& b) {
    return a.begin != b.begin ? a.begin < b.begin : a.i < b.i;
  };
  if (!std::is_sorted(s.get(), s.get() + m, before)) std::sort(s.get(), s.get() + m, before);
  for (int64_t i = 0; i < m; ++i) {
    for (int64_t j = i + 1; j < m && s[j].begin < s[i].end; ++j) {
      if (!s[i].written && !s[j].written) continue;
      if (!share_elements(s[i], s[j])) continue;
      note_error("gemm14_grad_clip: tensors %lld and %lld share memory that is written",
                 static_cast<long long>(s[i].i), static_cast<long long>(s[j].i));
      return GEMM14_ERR_INVALID_ARG;
    }
  }
  return GEMM14_OK;
}

struct Call {
  int64_t n;
  const gemm14_tensor* grads;
  const gemm14_tensor* outs;  // NULL: none, or in place
  bool clip;
  float scale, max_norm;
  float* norm;
  float* each;
  char* ws;
  Layout l;
  int sms;
  cudaStream_t stream;
};

// One launch's tensors, [i0, i0 + t.n), for blocks of so many warps; returns all warps.
template <int kN>
uint32_t fill(const Call& c, int64_t i0, uint32_t most, uint32_t block_warps, Table<kN>* t) {
  t->n = static_cast<int>(std::min<int64_t>(kN, c.n - i0));
  int64_t units = 0;
  for (int i = 0; i < t->n; ++i) {
    t->e[i] = entry_of(c.grads[i0 + i], c.outs ? c.outs + i0 + i : nullptr);
    t->e[i].first_unit = static_cast<uint32_t>(units);
    units += entry_units(t->e[i]);
  }
  t->units = static_cast<uint32_t>(units);
  t->in_place = true;
  for (int i = 0; i < t->n; ++i) t->in_place = t->in_place && t->e[i].src == t->e[i].dst;
  const uint32_t warps = std::min(t->units, most);
  if (Table<kN>::kStarts) {
    // block b's first unit, units b block_warps / warps rounded down, without a division each
    const uint64_t step = static_cast<uint64_t>(t->units) * block_warps;
    uint64_t u = 0, rest = 0;
    int i = 0;
    for (uint32_t b = 0; b * block_warps < warps; ++b) {
      while (i + 1 < t->n && t->e[i + 1].first_unit <= u) ++i;
      t->start[b] = static_cast<uint16_t>(i);
      u += step / warps;
      rest += step % warps;
      if (rest >= warps) {
        rest -= warps;
        ++u;
      }
    }
  }
  return warps;
}

dim3 blocks_for(uint32_t warps) { return dim3((warps + kThreads / 32 - 1) / (kThreads / 32)); }

template <int kN>
Parts<kN> parts_of(const Table<kN>& t, uint32_t warps) {
  Parts<kN> p;
  p.n = t.n;
  for (int i = 0; i < t.n; ++i) p.first[i] = warp_of(t.units, t.e[i].first_unit, warps) + i;
  p.first[t.n] = warps + static_cast<uint32_t>(t.n) - 1u;
  return p;
}

Finish finish_of(const Call& c, int64_t i0, int n, int launch) {
  Finish f{};
  f.slots = reinterpret_cast<double*>(c.ws + c.l.slots);
  f.totals = reinterpret_cast<double*>(c.ws + c.l.totals);
  f.launch = launch;
  f.last = i0 + n == c.n;
  f.scale = c.scale;
  f.max_norm = c.max_norm;
  f.norm = c.norm;
  f.each = c.each ? c.each + i0 : nullptr;
  f.factor = c.clip ? reinterpret_cast<double*>(c.ws + c.l.factor) : nullptr;
  return f;
}

// launch_kernel for clusters of `ctas` blocks.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, int ctas,
                           cudaStream_t stream, Args&&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <int kN>
int small_call(const Call& c) {
  Table<kN> t;
  const uint32_t warps =
      fill(c, 0, kSmallCtas * kSmallThreads / 32, kSmallThreads / 32, &t);
  return finish_launch(
      launch_cluster(grad_small_kernel<kN>, dim3(kSmallCtas), dim3(kSmallThreads), kSmallCtas,
                     c.stream, t, parts_of(t, warps), warps,
                     reinterpret_cast<double*>(c.ws + c.l.slots), finish_of(c, 0, t.n, 0)),
      "gradient norm launch", c.stream);
}

template <int kN>
int few_units_call(const Call& c) {
  Table<kN> t;
  const uint32_t warps = fill(c, 0, most_warps(c.sms), kThreads / 32, &t);
  const int st = finish_launch(
      launch_kernel(grad_sum_kernel<kN>, blocks_for(warps), dim3(kThreads), 0, c.stream, t, warps,
                    reinterpret_cast<double*>(c.ws + c.l.slots)),
      "gradient norm launch", c.stream);
  if (st != GEMM14_OK) return st;
  return finish_launch(
      launch_kernel(grad_total_scale_kernel<kN>, blocks_for(warps), dim3(kThreads), 0, c.stream, t,
                    parts_of(t, warps), warps, finish_of(c, 0, t.n, 0)),
      "gradient scaling launch", c.stream);
}

template <int kN>
int sum_launch(const Call& c, int64_t i0, int launch) {
  Table<kN> t;
  const uint32_t warps = fill(c, i0, most_warps(c.sms), kThreads / 32, &t);
  const int st = finish_launch(
      launch_kernel(grad_sum_kernel<kN>, blocks_for(warps), dim3(kThreads), 0, c.stream, t, warps,
                    reinterpret_cast<double*>(c.ws + c.l.slots)),
      "gradient norm launch", c.stream);
  if (st != GEMM14_OK) return st;
  // a warp a tensor
  const int each = c.each ? (t.n + kFinishThreads / 32 * kFinishCtas - 1) /
                                (kFinishThreads / 32 * kFinishCtas)
                          : 0;
  return finish_launch(
      launch_cluster(grad_finish_kernel<kN>, dim3((1 + each) * kFinishCtas), dim3(kFinishThreads),
                     kFinishCtas, c.stream, parts_of(t, warps), finish_of(c, i0, t.n, launch)),
      "gradient norm launch", c.stream);
}
template <int kN>
int scale_launch(const Call& c, int64_t i0) {
  Table<kN> t;
  const uint32_t warps = fill(c, i0, most_warps(c.sms), kThreads / 32, &t);
  return finish_launch(launch_kernel(grad_scale_kernel<kN>, blocks_for(warps), dim3(kThreads), 0,
                                     c.stream, t, warps,
                                     reinterpret_cast<const double*>(c.ws + c.l.factor)),
                       "gradient scaling launch", c.stream);
}

// Tables of three sizes: a launch's parameters are copied with it (10 tensors in the
// table of 544: 17.3 us of the host for the norm, 15.9 in that of 16; in three launches
// into others 25.3 and 23.4; 40 tensors 25.1 and 23.7 in that of 72, 41.7 and 39.3).
int run(const Call& c, int64_t units) {
  if (c.n <= kSmallEntries && units <= (c.clip ? kSmallScaled : kSmallUnits))
    return c.n <= 16 ? small_call<16>(c) : small_call<kSmallEntries>(c);
  if (c.clip && c.n <= kSmallEntries && units <= kFewUnits)
    return c.n <= 16 ? few_units_call<16>(c) : few_units_call<kSmallEntries>(c);
  int launch = 0;
  for (int64_t i0 = 0; i0 < c.n; i0 += kMostEntries, ++launch) {
    const int64_t m = c.n - i0;
    const int st = m <= 16   ? sum_launch<16>(c, i0, launch)
                   : m <= 72 ? sum_launch<72>(c, i0, launch)
                             : sum_launch<kMostEntries>(c, i0, launch);
    if (st != GEMM14_OK) return st;
  }
  if (!c.clip) return GEMM14_OK;
  // from the last tensors to the first, for what L2 still holds of them: a list of 43 MB
  // is read again from there (2 to 5 MB of it from DRAM), of 90 MB a third, as the norm's
  // last readings are the ends of all warps' stretches
  for (int64_t i0 = (c.n - 1) / kMostEntries * kMostEntries; i0 >= 0; i0 -= kMostEntries) {
    const int64_t m = c.n - i0;
    const int st = m <= 16   ? scale_launch<16>(c, i0)
                   : m <= 72 ? scale_launch<72>(c, i0)
                             : scale_launch<kMostEntries>(c, i0);
    if (st != GEMM14_OK) return st;
  }
  return GEMM14_OK;
}

bool finite(float x) { return x - x == 0.0f; }

// What the arguments are checked for on the host, before any CUDA call.
const char* fault_of(const Call& c, int64_t* units) {
  if (c.n < 0 || c.n > kMostTensors || (c.n > 0 && !c.grads)) return "the number of tensors";
  if (!finite(c.scale)) return "scale";
  if (c.clip && !(c.max_norm >= 0.0f)) return "max_norm";
  if (!c.norm || !aligned(c.norm, 4) || !aligned(c.each, 4)) return "norm or each";
  if (c.ws && !aligned(c.ws, 16)) return "the workspace's alignment";
  *units = 0;
  for (int64_t i = 0; i < c.n; ++i) {
    const gemm14_tensor& g = c.grads[i];
    if (validate_tensor(g) != GEMM14_OK) return "a gradient";
    if (c.outs) {
      const gemm14_tensor& o = c.outs[i];
      if (validate_tensor(o) != GEMM14_OK || o.rows != g.rows || o.cols != g.cols ||
          (o.dtype != g.dtype && o.dtype != GEMM14_DTYPE_F32))
        return "an output";
    }
    *units += entry_units(entry_of(g, c.outs ? c.outs + i : nullptr));
    if (*units > INT32_MAX) return "the gradients' total size";
  }
  return nullptr;
}

int grad_call(Call c, size_t workspace_bytes, const char* where) {
  int64_t units = 0;
  if (const char* fault = fault_of(c, &units)) {
    note_error("%s: invalid: %s", where, fault);
    return GEMM14_ERR_INVALID_ARG;
  }
  int st = c.clip ? check_apart(c.n, c.grads, c.outs) : GEMM14_OK;
  if (st != GEMM14_OK) return st;
  if ((st = current_sm_count(&c.sms)) != GEMM14_OK) return st;
  if (c.n == 0)
    return finish_launch(cudaMemset2DAsync(c.norm, 4, 0, 4, 1, c.stream), "gradient norm", c.stream);
  layout(c.n, c.sms, &c.l);
  if (!c.ws || workspace_bytes < c.l.total) {
    note_error("%s: %zu bytes of workspace given, %zu needed", where, workspace_bytes, c.l.total);
    return GEMM14_ERR_INVALID_ARG;
  }
  return run(c, units);
}

}  // namespace
}  // namespace gemm14

using namespace gemm14;

extern "C" {

size_t gemm14_grad_workspace_bytes(int64_t n, int sm_count) {
  if (n < 1 || n > kMostTensors) return 0;
  if (sm_count <= 0 && current_sm_count(&sm_count) != GEMM14_OK) return 0;
  Layout l;
  layout(n, sm_count, &l);
  return l.total;
}

int gemm14_grad_norm(int64_t n, const gemm14_tensor* grads, float scale, float* norm, float* each,
                     void* workspace, size_t workspace_bytes, void* stream) {
  Call c{};
  c.n = n;
  c.grads = grads;
  c.scale = scale;
  c.norm = norm;
  c.each = each;
  c.ws = static_cast<char*>(workspace);
  c.stream = static_cast<cudaStream_t>(stream);
  return grad_call(c, workspace_bytes, "gemm14_grad_norm");
}

int gemm14_grad_clip(int64_t n, const gemm14_tensor* grads, const gemm14_tensor* out, float scale,
                     float max_norm, float* norm, float* each, void* workspace,
                     size_t workspace_bytes, void* stream) {
  Call c{};
  c.n = n;
  c.grads = grads;
  c.outs = out;
  c.clip = true;
  c.scale = scale;
  c.max_norm = max_norm;
  c.norm = norm;
  c.each = each;
  c.ws = static_cast<char*>(workspace);
  c.stream = static_cast<cudaStream_t>(stream);
  return grad_call(c, workspace_bytes, "gemm14_grad_clip");
}

}  // extern "C"
