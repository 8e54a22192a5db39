// linear_ce.cu -- softmax cross entropy of a projection's outputs over a large
// vocabulary, without keeping the outputs: with z_t = H[t] W^T (V logits of
// row t), y_t the row's target and g_t the gradient of the caller's objective
// in loss_t,
//     lse_t  = log sum_v exp z_tv          loss_t = lse_t - z_t,y(t)
//     dZ_tv  = (exp(z_tv - lse_t) - [v = y_t]) g_t
//     dH     = dZ W                        dW     = dZ^T H.
//
// 16-bit operands, and fp32 ones in the split-precision mode, run on the
// tensor-core kernel of train_tc.cu. Its epilogues take the logits where they
// are, in tensor memory: the forward pass keeps of each tile a maximum and a sum
// per row, merged at the end; the backward pass forms the logits again from H,
// W and lse, a piece of the vocabulary at a time, writes the piece of dZ (16
// bits, two 16-bit parts for up to 128 rows, or three bf16 parts), and multiplies it into dH (fp32 sums over the
// pieces) and into the piece's rows of dW. What a step reads and writes beside
// its 8 n V D operations of products (n rows that take part; 2 of the 8 form the
// logits again) is small against them from a few hundred rows on, so the
// products bound it; below that, reading W does.
// Rows that take no part are left out before the products: a first kernel
// numbers the others, a second gathers their rows of H, and every later one
// reads their number on the device, so a batch that is mostly prompt costs what
// its answers cost, and nothing that an ignored row holds is ever multiplied.
//
// fp32 operands in the FFMA and TF32 modes take the library's products, a
// piece of fp32 logits at a time, with row kernels between them.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/gemm14.h"
#include "api_internal.h"
#include "kernels.h"
#include "linear_ce_narrow.h"
#include "operand_copy.cuh"
#include "plan.h"
#include "ptx.cuh"
#include "train_tc.h"

namespace gemm14 {
namespace {

constexpr int kThreads = 256;

// Sum of exponentials held as top + log(sum): (m, l) stands for l exp(m).
struct ExpSum {
  float m, l;
};
__device__ __forceinline__ ExpSum merge(ExpSum a, ExpSum b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return {m, a.l + b.l};  // no term above -inf (NaN sums are kept)
  return {m, a.l * __expf(a.m - m) + b.l * __expf(b.m - m)};
}

// ---- rows in use

// The rows that take part are numbered in order: *n of them, row i of them from
// row index[i] of the batch, position[t] = i or -1; and their data: the target
// as a column (-1 where it is no row of W), and for the gradient lse and the
// coefficient. For 16-bit dZ that is g_t / ref * unit with ref = max |g_t|
// over the rows that take part: dZ then lies in [-unit, unit] whatever the
// scale of the objective, and the products are multiplied by *back = ref / unit
// at the end.
struct Rows {
  int* n;
  float* back;
  int* index;
  int* position;
  int* target;
  float* lse;
  float* coef;
};
// What numbering reads; g null: the forward pass.
struct RowsIn {
  const int64_t* targets;
  int64_t ignore;
  const float* lse;
  const float* g;
  int64_t T, V;
  bool relative;
  float unit;
};

__device__ __forceinline__ float sound_ref(float ref) {
  return ref > 0.0f && ref < INFINITY ? ref : 1.0f;
}
// The data of row t of the batch, which takes part as row i.
__device__ __forceinline__ void put_row(const RowsIn& in, const Rows& out, int64_t t, int i,
                                        int64_t y, float g, float ref) {
  const bool sound = y >= 0 && y < in.V;
  out.index[i] = static_cast<int>(t);
  out.target[i] = sound ? static_cast<int>(y) : -1;
  if (in.g) {
    out.lse[i] = in.lse[t];
    out.coef[i] = sound ? g / ref * in.unit : __uint_as_float(0x7fc00000u);
  }
}

// One block: 8192 rows a turn, each thread 8 of them.
constexpr int kRowsPerThread = 8;

__global__ void __launch_bounds__(1024) ce_rows_kernel(const RowsIn in, const Rows out) {
  __shared__ int count[kRowsPerThread * 32];
  __shared__ float part[32];
  __shared__ int total;
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t T = in.T;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t y[kRowsPerThread];
  float k[kRowsPerThread];
  const auto load = [&](int64_t t0) {
#pragma unroll
    for (int j = 0; j < kRowsPerThread; ++j) {
      const int64_t t = t0 + 1024 * j + threadIdx.x;
      y[j] = t < T ? in.targets[t] : in.ignore;
      k[j] = in.g && t < T ? in.g[t] : 1.0f;
    }
  };
  load(0);  // (all there is, for most batches)
  float ref = 0.0f;
  if (in.relative) {
#pragma unroll
    for (int j = 0; j < kRowsPerThread; ++j)
      if (y[j] != in.ignore) ref = fmaxf(ref, fabsf(k[j]));
    for (int64_t t = 1024 * kRowsPerThread + threadIdx.x; t < T; t += 1024)
      if (in.targets[t] != in.ignore) ref = fmaxf(ref, fabsf(in.g[t]));
    for (int o = 16; o; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
    if (lane == 0) part[warp] = ref;
    __syncthreads();
    ref = 0.0f;
    for (int w = 0; w < 32; ++w) ref = fmaxf(ref, part[w]);
  }
  ref = sound_ref(ref);
  int base = 0;
  for (int64_t t0 = 0; t0 < T; t0 += 1024 * kRowsPerThread) {
    if (t0 > 0) load(t0);
    unsigned mask[kRowsPerThread];
#pragma unroll
    for (int j = 0; j < kRowsPerThread; ++j) {
      mask[j] = __ballot_sync(0xffffffffu, y[j] != in.ignore && k[j] != 0.0f);
      if (lane == 0) count[32 * j + warp] = __popc(mask[j]);
    }
    __syncthreads();
    if (warp == 0) {  // exclusive sums of the 256 counts
      int c[kRowsPerThread], sum = 0;
#pragma unroll
      for (int j = 0; j < kRowsPerThread; ++j) {
        c[j] = sum;
        sum += count[kRowsPerThread * lane + j];
      }
      int before = sum;
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      if (lane == 31) total = before;
      before -= sum;
#pragma unroll
      for (int j = 0; j < kRowsPerThread; ++j) count[kRowsPerThread * lane + j] = before + c[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kRowsPerThread; ++j) {
      const int64_t t = t0 + 1024 * j + threadIdx.x;
      if (t >= T) continue;
      const bool used = (mask[j] >> lane) & 1u;
      const int i = base + count[32 * j + warp] + __popc(mask[j] & ((1u << lane) - 1u));
      out.position[t] = used ? i : -1;
      if (used) put_row(in, out, t, i, y[j], k[j], ref);
    }
    base += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    *out.n = base;
    *out.back = ref / in.unit;
  }
}

// The rows of H in use, one after the other (E = float: as three bf16 parts),
// zeros up to the next multiple of 64 rows (a product over the rows reads whole
// k-blocks), and zeros into the rows of dH (where given) that take no part; and
// beside that the first piece of W, where it is copied. Block b < T: row b of the
// batch; the 64 after that: rows past the last; the rest: W.
// kNumber: the rows are not numbered yet. Up to 1024 of them each block counts
// for itself, which takes less than the launch of the kernel that does it once.
constexpr int kSelfNumbered = 1024;

template <typename E, bool kNumber>
__global__ void __launch_bounds__(256)
    ce_gather_kernel(const E* H, int64_t ldh, int64_t D, const RowsIn in, const Rows rows,
                     uint16_t* out, int64_t ldo, int64_t part_stride, E* dH, int64_t lddh,
                     bool vec, const OperandCopy w, int w_blocks) {
  __shared__ float part[8];
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int kParts = sizeof(E) == 4 ? 3 : 1;
  const int64_t T = in.T, b = blockIdx.x;
  if (b >= T + 64) {
    operand_copy(w, static_cast<int>(b - T - 64), w_blocks);
    return;
  }
  int i = -1, n = 0;
  if constexpr (kNumber) {
    int64_t y[4];
    float g[4], ref = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t t = threadIdx.x + 256 * j;
      y[j] = t < T ? in.targets[t] : in.ignore;
      g[j] = in.g && t < T ? in.g[t] : 1.0f;
      if (in.relative && y[j] != in.ignore) ref = fmaxf(ref, fabsf(g[j]));
    }
    for (int o = 16; o; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ref;
    bool mine = false;
    int before = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t t = threadIdx.x + 256 * j;
      const bool used = y[j] != in.ignore && g[j] != 0.0f;
      n += __syncthreads_count(used);
      before += __syncthreads_count(used && t < b);
      mine = __syncthreads_or(used && t == b) || mine;
    }
    ref = 0.0f;
    for (int k = 0; k < 8; ++k) ref = fmaxf(ref, part[k]);
    ref = sound_ref(ref);
    i = mine ? before : -1;
    if (threadIdx.x == 0) {
      if (b < T) {
        rows.position[b] = i;
        if (mine) put_row(in, rows, b, i, in.targets[b], in.g ? in.g[b] : 1.0f, ref);
      }
      if (b == 0) {
        *rows.n = n;
        *rows.back = ref / in.unit;
      }
    }
  } else {
    n = *rows.n;
    if (b < T) i = rows.position[b];
  }
  if (b >= T) {
    const int64_t r = n + (b - T);
    if (r >= (n + 63) / 64 * 64) return;
    for (int p = 0; p < kParts; ++p)
      for (int64_t c = threadIdx.x; c < D; c += blockDim.x)
        out[p * part_stride + r * ldo + c] = 0;
    return;
  }
  if (i < 0) {
    if (dH)
      for (int64_t c = threadIdx.x; c < D; c += blockDim.x) dH[b * lddh + c] = E(0);
    return;
  }
  const E* h = H + b * ldh;
  uint16_t* o = out + i * ldo;
  if constexpr (kParts == 1) {
    const E* end = H + (T - 1) * ldh + D;
    for (int64_t c = 8 * threadIdx.x; c < D; c += 8 * blockDim.x) {
      if (c + 8 <= D && (vec || words_inside(h + c, 16, H, end))) {
        *reinterpret_cast<uint4*>(o + c) =
            vec ? *reinterpret_cast<const uint4*>(h + c) : load16_any(h + c);
      } else {
        for (int j = 0; j < 8 && c + j < D; ++j) o[c + j] = h[c + j];
      }
    }
  } else {
    for (int64_t c = threadIdx.x; c < D; c += blockDim.x) {
      float x = h[c];
      for (int p = 0; p < kParts; ++p)
        o[p * part_stride + c] = __bfloat16_as_ushort(take_part(x, p));
    }
  }
}

// loss and lse of 32 rows of the batch from their rows' parts: lane = row,
// the 32 warps share the parts. position null: row t is row t in use.
__global__ void __launch_bounds__(1024)
    ce_combine_kernel(const float2* part, int64_t part_ld, int parts, const float* target_logit,
                      const int* position, const int64_t* targets, int64_t ignore, int64_t T,
                      int64_t V, float* loss, float* lse) {
  __shared__ ExpSum sums[32][33];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const int64_t y = t < T ? targets[t] : ignore;
  const int64_t i = t >= T || y == ignore ? -1 : position ? position[t] : t;
  ExpSum s{-INFINITY, 0.0f};
  if (i >= 0) {
    constexpr int kAhead = 8;  // loads in flight
    for (int p0 = warp; p0 < parts; p0 += 32 * kAhead) {
      float2 v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        v[u] = p0 + 32 * u < parts ? part[(p0 + 32 * u) * part_ld + i]
                                   : make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) s = merge(s, {v[u].x, v[u].y});
    }
  }
  sums[warp][lane] = s;
  __syncthreads();
  for (int half = 16; half >= 1; half /= 2) {
    if (warp < half) sums[warp][lane] = s = merge(s, sums[warp + half][lane]);
    __syncthreads();
  }
  if (warp != 0 || t >= T) return;
  const float total = s.m + logf(s.l);
  lse[t] = i < 0 ? 0.0f : total;
  loss[t] = i < 0 ? 0.0f
            : y < 0 || y >= V ? __uint_as_float(0x7fc00000u) : total - target_logit[i];
}

// ---- the FFMA and TF32 modes: row passes over a piece of fp32 logits (Z: T x C,
// pitch ldz, columns v0 ..)

struct RowState {  // per row, carried from piece to piece
  float* m;
  float* l;
  float* zy;  // the target's logit
};

__global__ void __launch_bounds__(kThreads)
    ce_stats_kernel(const float* Z, int64_t ldz, int64_t C, int64_t v0, int64_t V,
                    const int64_t* targets, int64_t ignore, RowState state, float* loss, float* lse) {
  __shared__ ExpSum part[kThreads / 32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t t = blockIdx.x;
  const float* z = Z + t * ldz;
  ExpSum s{-INFINITY, 0.0f};
  // a NaN goes into the sum (the maximum would drop it)
  for (int64_t c = threadIdx.x; c < C; c += kThreads) {
    const float x = z[c];
    s = merge(s, {x, x == x ? 1.0f : x});
  }
  for (int o = 16; o; o >>= 1)
    s = merge(s, {__shfl_xor_sync(0xffffffffu, s.m, o), __shfl_xor_sync(0xffffffffu, s.l, o)});
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < kThreads / 32; ++w) s = merge(s, part[w]);
  const int64_t y = targets[t];
  float zy = 0.0f;
  if (v0 > 0) {
    s = merge({state.m[t], state.l[t]}, s);
    zy = state.zy[t];
  }
  if (y >= v0 && y < v0 + C) zy = z[y - v0];
  if (v0 + C < V) {
    state.m[t] = s.m;
    state.l[t] = s.l;
    state.zy[t] = zy;
    return;
  }
  const float total = s.m + logf(s.l);
  const bool off = y == ignore;
  lse[t] = off ? 0.0f : total;
  loss[t] = off ? 0.0f : y < 0 || y >= V ? __uint_as_float(0x7fc00000u) : total - zy;
}

// dZ of a piece in place of the logits.
__global__ void __launch_bounds__(kThreads)
    ce_grad_kernel(float* Z, int64_t ldz, int64_t C, int64_t v0, const int64_t* targets,
                   const float* lse, const float* coef) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t t = blockIdx.x;
  const float k = coef[t], top = lse[t];
  const int64_t y = targets[t] - v0;
  float* z = Z + t * ldz;
  for (int64_t c = threadIdx.x; c < C; c += kThreads)
    z[c] = k == 0.0f ? 0.0f : (__expf(z[c] - top) - (c == y ? 1.0f : 0.0f)) * k;
}

// Each row's coefficient, 0 for a row that takes no part, NaN for a target
// that is no row of W; and H with the rows that take no part set to zero, so
// that nothing they hold (uninitialised padding, a NaN) reaches dW.
__global__ void __launch_bounds__(kThreads)
    ce_masked_kernel(const float* H, int64_t ldh, int64_t D, const int64_t* targets,
                     int64_t ignore, int64_t V, const float* g, float* coef, float* out,
                     int64_t ldo) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t t = blockIdx.x, y = targets[t];
  const float k = y == ignore || g[t] == 0.0f ? 0.0f
                  : y < 0 || y >= V ? __uint_as_float(0x7fc00000u) : g[t];
  for (int64_t c = threadIdx.x; c < D; c += kThreads)
    out[t * ldo + c] = k == 0.0f ? 0.0f : H[t * ldh + c];
  if (threadIdx.x == 0) coef[t] = k;
}

// Zero into the rows of dH that take no part.
__global__ void __launch_bounds__(kThreads)
    ce_clear_kernel(float* dH, int64_t ldd, int64_t D, const float* coef) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t t = blockIdx.x;
  if (coef[t] != 0.0f) return;
  for (int64_t c = threadIdx.x; c < D; c += kThreads) dH[t * ldd + c] = 0.0f;
}

// ---- host side

bool size_ok(int64_t n) { return n >= 0 && n <= kTrainMaxSize; }
int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
int64_t tiles_of(int64_t x) { return (x + 255) / 256; }
// Whether the operands run on the tensor-core kernel: 16-bit ones, and fp32
// ones in the split-precision mode (as three bf16 parts).
bool on_tensor_cores(int dtype) {
  return dtype == GEMM14_DTYPE_BF16 || dtype == GEMM14_DTYPE_F16 ||
         dtype == GEMM14_DTYPE_F32_3XTF32;
}
// TMA can read rows of 16-bit elements at this address and pitch.
bool tma_rows(const void* p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

int validate_ce(int dtype, int64_t T, int64_t V, int64_t D, const void* H, int64_t ldh,
                const void* W, int64_t ldw, const int64_t* targets) {
  if (!size_ok(T) || !size_ok(V) || !size_ok(D) || V < 1 || D < 1) return GEMM14_ERR_INVALID_ARG;
  if (T > 0 && (!targets || !aligned(targets, 8))) return GEMM14_ERR_INVALID_ARG;
  // the product's own checks; the logits (in the workspace) are always sound
  const void* sound = reinterpret_cast<const void*>(uintptr_t(1) << 12);
  return validate_product(dtype, 0, 1, T, V, D, H, ldh, W, ldw, sound, V);
}

// Bytes a piece of logits or dZ, and a piece of W that has to be copied, may take.
constexpr int64_t kPieceBytes = int64_t(384) << 20;

// Rows of W per piece, a multiple of 256 unless one piece takes all: pieces of
// about the same size, `per_row` bytes a row of W within the limit.
int64_t piece_rows(int64_t V, int64_t per_row) {
  const int64_t most = std::max<int64_t>(kPieceBytes / per_row / 256 * 256, 256);
  const int64_t pieces = (V + most - 1) / most;
  return pieces == 1 ? V : round_up((V + pieces - 1) / pieces, 256);
}

// Whether a handful of rows run on the CUDA cores (linear_ce_narrow.cu): fp32
// ones, in the modes that keep the fp32 bound (and no wider than a grid's second
// dimension reaches). The FFMA mode's other side is the library's products: 32 x
// 32768 x 4096, loss and gradients, 1937 us here against 2281, 32 x 100000 x 900
// 866 against 1836. The split mode's is the tensor cores on W's parts. Up to 16
// rows are ahead here (16 x 32768 x 4096 817 us against 1312, 1 row 404 against 1310),
// and 17 to 32 while shared memory holds them (32 x 65536 x 1024 587 against 619,
// x 1536 946 against 934, 17 rows 909 against 933); wider ones are loaded again, in
// slices, for each 32 rows of W, as many bytes as those: 17 x 65536 x 1600 1591
// against 1000, 32 rows 2072 against 999.
bool on_cuda_cores(int dtype, int64_t T, int64_t D) {
  if (T > kNarrowRows || D > kNarrowMaxD) return false;
  return dtype == GEMM14_DTYPE_F32 ||
         (dtype == GEMM14_DTYPE_F32_3XTF32 && (T <= 16 || narrow_in_one_slice(T, D)));
}

struct CeLayout {
  bool narrow = false;
  bool tc = false;
  int64_t C = 0;       // vocabulary rows of a piece
  int64_t ldz = 0;     // pitch of the logits or of dZ
  int64_t ldx = 0;     // pitch of the D-wide buffers
  int parts = 1;       // bf16 parts of an operand
  int dz_parts = 1;    // parts of dZ
  bool few = false;    // the logits come from the kernel for few rows
  int width = 0;       // columns of the logits' tiles, the same for every piece
  bool gather = false; // rows in use are numbered and gathered first
  bool copy_w = false; // pieces of W are copied (unaligned) or split
  int64_t slot_count = 0, tail_count = 0;  // of dH, and of dW's split tiles
  int64_t rows = 0;    // T rounded up to whole tiles
  int64_t stats = 0;   // entries of the statistics, of all pieces
  size_t state = 0, counts = 0, index = 0, position = 0, target = 0, lse = 0, coef = 0, h = 0,
         w = 0, part = 0, z = 0, slots = 0, tail = 0, total = 0;
};

// Parts of a row's statistics that c columns leave: two a tile. Tiles of one
// width for all pieces: a last, smaller piece of c columns would be spread
// better by tiles of its own width (few_width(c), which may be narrower and make
// more of them), but then its parts have no bound in those of the others.
int64_t stat_parts(const CeLayout& l, int64_t c) { return 2 * ((c + l.width - 1) / l.width); }

void ce_layout(int dtype, int64_t T, int64_t V, int64_t D, const void* H, int64_t ldh,
               const void* W, int64_t ldw, bool backward, int sms, CeLayout* l) {
  *l = CeLayout{};
  l->narrow = on_cuda_cores(dtype, T, D);
  l->tc = on_tensor_cores(dtype);
  l->ldx = round_up(D, 8);
  l->rows = round_up(T, 256);
  size_t at = streamk_flag_bytes(sms);
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = round256(at + bytes);
    return here;
  };
  const size_t t4 = static_cast<size_t>(T) * 4;
  if (l->narrow) {
    l->ldz = V;
    if (backward) {
      l->z = take(static_cast<size_t>(T) * l->ldz * 4);
      l->slots = take(static_cast<size_t>(narrow_splits(static_cast<int>(T), V, D, sms)) * T * D * 4);
    } else {
      l->part = take(static_cast<size_t>(narrow_blocks(V, sms)) * T * sizeof(float2));
      l->state = take(t4);
    }
    l->total = at;
    return;
  }
  if (l->tc) {
    l->ldx = round_up(D, 64);  // rows that start on 128-byte lines
    l->parts = dtype == GEMM14_DTYPE_F32_3XTF32 ? 3 : 1;
    l->copy_w = l->parts == 3 || !tma_rows(W, ldw);
    // one tile row of rows costs the same with and without the ignored ones
    l->gather = backward || l->parts == 3 || !tma_rows(H, ldh) || T > TrainShape::BM;
    l->few = T <= FewShape::MAX_ROWS;
    // 16-bit dZ of few rows is held in two parts. Its rounding makes gradients 1.33
    // times as far off as their own does; over many rows that is all, over few it
    // is one row's luck (up to 1.6 times). The parts share the 256 rows of a tile, so
    // dH's products take no longer.
    l->dz_parts = l->parts == 3 ? 3 : l->few ? 2 : 1;
    int64_t per_row = 1;  // (a piece is well within 32 bits in any case)
    if (backward) per_row = l->rows * 2 * l->parts;
    if (l->copy_w) per_row = std::max(per_row, l->ldx * 2 * l->parts);
    l->C = piece_rows(V, per_row);
    l->width = l->few ? few_width(l->C, sms) : TrainShape::BN;
    l->ldz = round_up(l->C, 64);
    if (l->gather) {
      l->counts = take(256);
      l->index = take(t4);
      l->position = take(t4);
      l->target = take(t4);
      l->h = take(static_cast<size_t>(l->rows) * l->ldx * 2 * l->parts);
    }
    if (l->copy_w) l->w = take(static_cast<size_t>(l->C) * l->ldx * 2 * l->parts);
    if (backward) {
      l->lse = take(t4);
      l->coef = take(t4);
      l->z = take(static_cast<size_t>(l->rows) * l->ldz * 2 * l->parts);
      // dH's sums over the pieces, and what dW's split tiles need after them
      const int clusters = std::max(sms / 2, 1);
      l->slot_count = slots_needed(tiles_of(T) * tiles_of(D), (l->C + 63) / 64, clusters, true);
      l->tail_count = slots_needed(2 * tiles_of(l->C) * tiles_of(D), (T + 63) / 64, clusters, false);
      l->slots = take(static_cast<size_t>(l->slot_count) * kSlotBytes);
      l->tail = take(static_cast<size_t>(l->tail_count) * kSlotBytes);
    } else {
      const int64_t full = (V - 1) / l->C;  // pieces before the last
      l->stats = (full * stat_parts(*l, l->C) + stat_parts(*l, V - full * l->C)) * l->rows;
      l->part = take(static_cast<size_t>(l->stats) * sizeof(float2));
      l->state = take(t4);
    }
    l->total = at;
    return;
  }
  l->C = piece_rows(V, 4 * T);
  l->ldz = round_up(l->C, 8);
  const void* own = reinterpret_cast<const void*>(uintptr_t(1) << 12);
  auto need = [&](int ta, int tb, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                  const void* B, int64_t ldb, int64_t ldc) {
    at = std::max(at, gemm14_workspace_bytes_ex(dtype, ta, tb, M, N, K, A, lda, B, ldb, own, ldc,
                                                sms));
  };
  const int64_t last = V - (V - 1) / l->C * l->C;
  for (const int64_t c : {l->C, last}) {
    need(0, 1, T, c, D, H, ldh, W, ldw, l->ldz);
    if (!backward) continue;
    need(0, 0, T, D, c, own, l->ldz, W, ldw, D);
    need(1, 0, c, D, T, own, l->ldz, own, l->ldx, D);
  }
  at = round256(at);
  l->state = take(3 * t4);
  l->z = take(static_cast<size_t>(T) * l->ldz * 4);
  if (backward) {
    l->coef = take(t4);
    l->h = take(static_cast<size_t>(T) * l->ldx * 4);
  }
  l->total = at;
}

int check_room(const char* who, const void* workspace, size_t bytes, size_t need) {
  if (workspace && aligned(workspace, 16) && bytes >= need) return GEMM14_OK;
  note_error("%s: %zu bytes of workspace given, %zu needed (16-byte aligned)", who,
             workspace ? bytes : size_t(0), need);
  return GEMM14_ERR_INVALID_ARG;
}

// Row v of W (elements of eb bytes).
const void* row_of(const void* W, int64_t v, int64_t ld, int eb) {
  return static_cast<const char*>(W) + v * ld * eb;
}

// A call of either direction.
struct CeCall {
  int dtype;
  int64_t T, V, D;
  const void* H;
  int64_t ldh;
  const void* W;
  int64_t ldw;
  const int64_t* targets;
  int64_t ignore;
  char* ws;
  cudaStream_t stream;
  CeLayout l;
  CallContext ctx;
  int clusters = 0;

  bool bf16() const { return dtype != GEMM14_DTYPE_F16; }
  int eb() const { return elem_bytes_of(dtype); }
  template <typename P>
  P* at(size_t off) const { return reinterpret_cast<P*>(ws + off); }

  int launched(cudaError_t e, const char* what) const { return finish_launch(e, what, stream); }

  Rows rows() const {
    return Rows{at<int>(l.counts),   at<float>(l.counts) + 1, at<int>(l.index),
                at<int>(l.position), at<int>(l.target),       at<float>(l.lse),
                at<float>(l.coef)};
  }

  int prepare_tc() {
    clusters = train_max_clusters();
    if (clusters > 0) return GEMM14_OK;
    note_error("linear_ce: clusters of two CTAs cannot run on this device");
    return GEMM14_ERR_CUDA;
  }

  // Numbers and gathers the rows in use, and copies the first piece of W where
  // it has to be.
  int gather(const float* lse, const float* g, void* dH, int64_t lddh) const {
    // fp16's range: dZ is held in units of 2^-15, so that probabilities down
    // to 2^-39 of the largest coefficient are not lost
    const RowsIn in{targets, ignore, lse, g, T, V, g && dtype != GEMM14_DTYPE_F32_3XTF32,
                    dtype == GEMM14_DTYPE_F16 ? 32768.0f : 1.0f};
    const bool number = T <= kSelfNumbered;
    if (!number) {
      const int st = launched(launch_kernel(ce_rows_kernel, dim3(1), dim3(1024), 0, stream, in,
                                            rows()),
                              "linear_ce rows launch");
      if (st != GEMM14_OK) return st;
    }
    const OperandCopy w = w_copy(0, l.copy_w ? std::min(l.C, V) : 0);
    const int w_blocks = l.copy_w ? operand_copy_blocks(w, ctx.sm_count) : 0;
    const dim3 grid(static_cast<unsigned>(T + 64 + w_blocks)), block(256);
    uint16_t* out = at<uint16_t>(l.h);
    const int64_t stride = l.rows * l.ldx;
    const cudaError_t e =
        l.parts == 3
            ? launch_kernel(number ? ce_gather_kernel<float, true> : ce_gather_kernel<float, false>,
                            grid, block, 0, stream, static_cast<const float*>(H), ldh, D, in,
                            rows(), out, l.ldx, stride, static_cast<float*>(dH), lddh, false, w,
                            w_blocks)
            : launch_kernel(
                  number ? ce_gather_kernel<uint16_t, true> : ce_gather_kernel<uint16_t, false>,
                  grid, block, 0, stream, static_cast<const uint16_t*>(H), ldh, D, in, rows(), out,
                  l.ldx, stride, static_cast<uint16_t*>(dH), lddh, tma_rows(H, ldh), w, w_blocks);
    return launched(e, "linear_ce gather launch");
  }

  // The rows of H in use as an operand.
  TrainOperand h_operand() const {
    if (!l.gather) return TrainOperand{H, T, D, ldh, 1, 0};
    return TrainOperand{ws + l.h, l.rows, D, l.ldx, l.parts, l.rows * l.ldx};
  }

  // The copy of c rows of W from v0 as the products read them.
  OperandCopy w_copy(int64_t v0, int64_t c) const {
    return OperandCopy{row_of(W, v0, ldw, eb()), ldw, c, D, ws + l.w, l.ldx, l.C * l.ldx, l.parts};
  }

  // c rows of W from v0 as an operand, copied or split first where they must be
  // (the first piece: by gather, where there is one).
  int w_operand(int64_t v0, int64_t c, TrainOperand* w) const {
    if (!l.copy_w) {
      *w = TrainOperand{row_of(W, v0, ldw, eb()), c, D, ldw, 1, 0};
      return GEMM14_OK;
    }
    *w = TrainOperand{ws + l.w, c, D, l.ldx, l.parts, l.C * l.ldx};
    if (v0 == 0 && l.gather) return GEMM14_OK;
    return launched(launch_operand_copy(w_copy(v0, c), ctx.sm_count, stream),
                    "linear_ce copy launch");
  }

  // Arguments of a product M x N over K, its rows (or its K, n_is_k) being those in use.
  TrainArgs product(int64_t M, int64_t N, int64_t K, bool n_is_k) const {
    TrainArgs a{};
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.n = l.gather ? at<int>(l.counts) : nullptr;
    a.n_is_k = n_is_k;
    a.err = ctx.err;
    a.wait_limit_ns = ctx.wait_limit_ns;
    a.fault = ctx.fault;
    a.alpha = 1.0f;
    a.width = TrainShape::BN;
    return a;
  }

  int run(int mode, bool promote, const TrainOperand& A, bool a_mn, const TrainOperand& B,
          bool b_mn, TrainArgs* a) {
    TrainMaps maps;
    const int st = train_operands(bf16(), A, a_mn, B, b_mn, &maps, a);
    if (st != GEMM14_OK) return st;
    ctx.fault = kFaultNone;  // a test's request applies to the call's first product
    return launched(launch_train_tc(mode, promote, maps, *a, clusters, stream),
                    "linear_ce product launch");
  }

  // A product of few rows with c rows of W, its arguments in a.
  int run_few(int mode, const TrainOperand& w, TrainArgs a) {
    TrainMaps maps;
    const int st = train_operands(bf16(), h_operand(), false, w, false, &maps, &a, few_rows(T),
                                  l.width);
    if (st != GEMM14_OK) return st;
    ctx.fault = kFaultNone;
    return launched(launch_train_few(mode, maps, a, bf16(), l.width, ctx.sm_count, stream),
                    "linear_ce few rows launch");
  }

  // Whether the logits' sums over D are carried in fp32 registers: in both calls,
  // so that dZ is formed from the logits that lse was.
  bool long_logits() const { return D > TrainShape::LOGITS_CHUNK * TrainShape::BK; }

  // Whether a gradient's sums over K are carried in fp32 registers. Written in
  // fp32 they keep fp32's accuracy. Rounded to 16 bits they may be off by a
  // fraction of that rounding: 262144 terms in one truncating accumulator left
  // dH of fp16 2.6 times its rounding off (its largest term came first), 700000
  // of bf16 0.9 times, so 0.16 times is left for as many as may stay there.
  bool long_sum(int64_t K) const {
    const int64_t most = l.parts == 3 ? TrainShape::CHUNK * TrainShape::BK
                         : bf16()     ? int64_t(131072)
                                      : int64_t(16384);
    return K > most;
  }

  // ---- a handful of rows

  NarrowArgs narrow_args() const {
    NarrowArgs a{};
    a.T = static_cast<int>(T);
    a.V = V;
    a.D = D;
    a.H = static_cast<const float*>(H);
    a.ldh = ldh;
    a.W = static_cast<const float*>(W);
    a.ldw = ldw;
    a.targets = targets;
    a.ignore = ignore;
    return a;
  }

  int forward_narrow(float* loss, float* lse) const {
    NarrowArgs a = narrow_args();
    a.part = at<float2>(l.part);
    a.part_ld = T;
    a.target_logit = at<float>(l.state);
    const int st = launched(launch_narrow_stats(a, ctx.sm_count, stream),
                            "linear_ce narrow launch");
    if (st != GEMM14_OK) return st;
    return combine(a.part, T, narrow_blocks(V, ctx.sm_count), a.target_logit, nullptr, loss, lse);
  }

  int backward_narrow(const float* lse, const float* g, void* dH, int64_t lddh, void* dW,
                      int64_t lddw) const {
    NarrowArgs a = narrow_args();
    a.lse = lse;
    a.dloss = g;
    a.dz = at<float>(l.z);
    a.ldz = l.ldz;
    a.sums = at<float>(l.slots);
    a.dH = static_cast<float*>(dH);
    a.lddh = lddh;
    a.dW = static_cast<float*>(dW);
    a.lddw = lddw;
    return launched(launch_narrow_backward(a, ctx.sm_count, stream), "linear_ce narrow launch");
  }

  // The rows' parts to loss and lse.
  int combine(const float2* part, int64_t part_ld, int64_t parts, const float* target_logit,
              const int* position, float* loss, float* lse) const {
    return launched(
        launch_kernel(ce_combine_kernel, dim3(static_cast<unsigned>((T + 31) / 32)), dim3(1024),
                      0, stream, part, part_ld, static_cast<int>(parts), target_logit, position,
                      targets, ignore, T, V, loss, lse),
        "linear_ce combine launch");
  }

  int forward_tc(float* loss, float* lse) {
    int st = prepare_tc();
    if (st != GEMM14_OK) return st;
    if (l.gather && (st = gather(nullptr, nullptr, nullptr, 0)) != GEMM14_OK) return st;
    const Rows r = rows();
    int64_t parts = 0;
    for (int64_t v0 = 0; v0 < V; v0 += l.C) {
      const int64_t c = std::min(l.C, V - v0);
      TrainOperand w;
      if ((st = w_operand(v0, c, &w)) != GEMM14_OK) return st;
      TrainArgs a = product(T, c, D, false);
      a.v0 = static_cast<int>(v0);
      a.target = l.gather ? r.target : nullptr;
      a.target64 = targets;
      a.part = at<float2>(l.part) + parts * l.rows;
      a.part_ld = l.rows;
      a.part_count = l.stats - parts * l.rows;
      a.target_logit = at<float>(l.state);
      st = l.few ? run_few(kTrainStats, w, a)
                 : run(kTrainStats, long_logits(), h_operand(), false, w, false, &a);
      if (st != GEMM14_OK) return st;
      parts += stat_parts(l, c);
    }
    return combine(at<float2>(l.part), l.rows, parts, at<float>(l.state),
                   l.gather ? r.position : nullptr, loss, lse);
  }

  int backward_tc(const float* lse, const float* g, void* dH, int64_t lddh, void* dW,
                  int64_t lddw) {
    int st = prepare_tc();
    if (st != GEMM14_OK) return st;
    if ((st = gather(lse, g, dH, lddh)) != GEMM14_OK) return st;
    const Rows r = rows();
    const bool exact = l.parts == 3;
    const int elem = exact ? kElemF32 : bf16() ? kElemBf16 : kElemF16;
    const bool two = l.dz_parts == 2;  // dZ's second part: rows 128 .. of its tile
    const int64_t z_rows = two ? FewShape::MAX_ROWS : l.rows, g_part = z_rows * l.ldz;
    for (int64_t v0 = 0; v0 < V; v0 += l.C) {
      const int64_t c = std::min(l.C, V - v0);
      TrainOperand w;
      if ((st = w_operand(v0, c, &w)) != GEMM14_OK) return st;
      TrainArgs a = product(T, c, D, false);
      a.v0 = static_cast<int>(v0);
      a.target = r.target;
      a.lse = r.lse;
      a.coef = r.coef;
      a.out = ws + l.z;
      a.ld_out = l.ldz;
      a.out_part = g_part;
      a.elem = exact ? kElemBf16x3 : elem;
      a.out_vec = 1;
      a.out_rows = z_rows;
      a.out_cols = c;
      st = l.few ? run_few(kTrainGrad, w, a)
                 : run(kTrainGrad, long_logits(), h_operand(), false, w, false, &a);
      if (st != GEMM14_OK) return st;
      // (rows past T's last block of 64 are zeros without being read)
      const TrainOperand dz{ws + l.z, round_up(T, 64), c, l.ldz, l.dz_parts, g_part};
      if (dH) {
        a = product(T, D, c, false);
        TrainOperand both = dz;
        if (two) {  // all 256 rows: what is past the rows in use stays in its rows
          both = TrainOperand{ws + l.z, 2 * z_rows, c, l.ldz, 1, 0};
          a.M = static_cast<int>(2 * z_rows);
          a.n = nullptr;
        }
        a.split_k = static_cast<int>(l.C);  // the same plan for every piece
        a.slots = at<float4>(l.slots);
        a.slot_count = l.slot_count;
        a.add = v0 > 0;
        if ((st = run(kTrainSlots, long_sum(c), both, false, w, true, &a)) != GEMM14_OK)
          return st;
      }
      if (dW) {
        a = product(c, D, T, true);
        a.width = tile_width((T + 63) / 64 * (exact ? 6 : 1));
        a.out = static_cast<char*>(dW) + v0 * lddw * eb();
        a.ld_out = lddw;
        a.elem = elem;
        a.out_vec = aligned(dW, 16) && lddw * eb() % 16 == 0;
        a.scale = r.back;
        a.split_k = static_cast<int>(T);
        a.slots = at<float4>(l.tail);
        a.slot_count = l.tail_count;
        a.out_rows = c;
        a.out_cols = D;
        if ((st = run(kTrainOut, long_sum(T), dz, true, h_operand(), true, &a)) !=
            GEMM14_OK)
          return st;
        if (may_split(a, clusters)) {
          const SlotsOut s{false, nullptr, 1.0f, 0.0f, r.back, a.out, lddw, elem, c};
          if ((st = launched(launch_slots_out(a, s, clusters, stream),
                             "linear_ce output launch")) != GEMM14_OK)
            return st;
        }
      }
    }
    if (!dH) return GEMM14_OK;
    TrainArgs a = product(T, D, V, false);
    a.split_k = static_cast<int>(l.C);
    a.terms = exact ? 6 : 1;
    a.slots = at<float4>(l.slots);
    const SlotsOut s{true, r.index, 1.0f, 0.0f, r.back, dH, lddh, elem, T, two ? 1 : 0};
    return launched(launch_slots_out(a, s, clusters, stream), "linear_ce output launch");
  }

  // ---- the FFMA and TF32 modes

  int logits(int64_t v0, int64_t c) const {
    return product_on_stream(dtype, 0, 1, T, c, D, 1.0f, H, ldh, row_of(W, v0, ldw, 4), ldw, 0.0f,
                             at<float>(l.z), l.ldz, ws, l.state, stream);
  }

  int forward_products(float* loss, float* lse) const {
    float* state = at<float>(l.state);
    const RowState rs{state, state + T, state + 2 * T};
    for (int64_t v0 = 0; v0 < V; v0 += l.C) {
      const int64_t c = std::min(l.C, V - v0);
      int st = logits(v0, c);
      if (st == GEMM14_OK)
        st = launched(launch_kernel(ce_stats_kernel, dim3(static_cast<unsigned>(T)),
                                    dim3(kThreads), 0, stream, at<float>(l.z), l.ldz, c, v0, V,
                                    targets, ignore, rs, loss, lse),
                      "linear_ce statistics launch");
      if (st != GEMM14_OK) return st;
    }
    return GEMM14_OK;
  }

  int backward_products(const float* lse, const float* g, void* dH, int64_t lddh, void* dW,
                        int64_t lddw) const {
    const dim3 per_row(static_cast<unsigned>(T)), block(kThreads);
    float* z = at<float>(l.z);
    float* coef = at<float>(l.coef);
    float* h = at<float>(l.h);
    float* dh = static_cast<float*>(dH);
    int st = launched(launch_kernel(ce_masked_kernel, per_row, block, 0, stream,
                                    static_cast<const float*>(H), ldh, D, targets, ignore, V, g,
                                    coef, h, l.ldx),
                      "linear_ce rows launch");
    for (int64_t v0 = 0; v0 < V && st == GEMM14_OK; v0 += l.C) {
      const int64_t c = std::min(l.C, V - v0);
      if ((st = logits(v0, c)) != GEMM14_OK) return st;
      if ((st = launched(launch_kernel(ce_grad_kernel, per_row, block, 0, stream, z, l.ldz, c, v0,
                                       targets, lse, coef),
                         "linear_ce gradient launch")) != GEMM14_OK)
        return st;
      if (dH && (st = product_on_stream(dtype, 0, 0, T, D, c, 1.0f, z, l.ldz,
                                        row_of(W, v0, ldw, 4), ldw, v0 ? 1.0f : 0.0f, dh, lddh, ws,
                                        l.state, stream)) != GEMM14_OK)
        return st;
      if (dW && (st = product_on_stream(dtype, 1, 0, c, D, T, 1.0f, z, l.ldz, h, l.ldx, 0.0f,
                                        static_cast<float*>(dW) + v0 * lddw, lddw, ws, l.state,
                                        stream)) != GEMM14_OK)
        return st;
    }
    if (st != GEMM14_OK || !dH) return st;
    return launched(launch_kernel(ce_clear_kernel, per_row, block, 0, stream, dh, lddh, D, coef),
                    "linear_ce clear launch");
  }
};

}  // namespace
}  // namespace gemm14

using namespace gemm14;

extern "C" {

size_t gemm14_linear_ce_workspace_bytes(int dtype, int backward, int64_t T, int64_t V, int64_t D,
                                        const void* H, int64_t ldh, const void* W, int64_t ldw,
                                        int sm_count) {
  static const int64_t some = 0;
  if (validate_ce(dtype, T, V, D, H, ldh, W, ldw, &some) != GEMM14_OK || T == 0) return 0;
  if (sm_count <= 0 && current_sm_count(&sm_count) != GEMM14_OK) return 0;
  CeLayout l;
  ce_layout(dtype, T, V, D, H, ldh, W, ldw, backward != 0, sm_count, &l);
  return l.total;
}

int gemm14_linear_ce_forward(int dtype, int64_t T, int64_t V, int64_t D, const void* H,
                             int64_t ldh, const void* W, int64_t ldw, const int64_t* targets,
                             int64_t ignore_index, float* loss, float* lse, void* workspace,
                             size_t workspace_bytes, void* stream) {
  CeCall c{dtype,        T, V, D, H, ldh, W, ldw, targets, ignore_index,
           static_cast<char*>(workspace), static_cast<cudaStream_t>(stream)};
  take_request(&c.ctx);
  int st = validate_ce(dtype, T, V, D, H, ldh, W, ldw, targets);
  if (st != GEMM14_OK) return st;
  if (T == 0) return GEMM14_OK;
  if (!loss || !lse || !aligned(loss, 4) || !aligned(lse, 4)) return GEMM14_ERR_INVALID_ARG;
  if ((st = call_device(&c.ctx)) != GEMM14_OK) return st;
  ce_layout(dtype, T, V, D, H, ldh, W, ldw, false, c.ctx.sm_count, &c.l);
  if ((st = check_room("gemm14_linear_ce_forward", workspace, workspace_bytes, c.l.total)) !=
      GEMM14_OK)
    return st;
  if (c.l.narrow) return c.forward_narrow(loss, lse);
  if (c.l.tc) return c.forward_tc(loss, lse);
  give_request(c.ctx);
  return c.forward_products(loss, lse);
}

int gemm14_linear_ce_backward(int dtype, int64_t T, int64_t V, int64_t D, const void* H,
                              int64_t ldh, const void* W, int64_t ldw, const int64_t* targets,
                              int64_t ignore_index, const float* lse, const float* dloss, void* dH,
                              int64_t lddh, void* dW, int64_t lddw, void* workspace,
                              size_t workspace_bytes, void* stream) {
  CeCall c{dtype,        T, V, D, H, ldh, W, ldw, targets, ignore_index,
           static_cast<char*>(workspace), static_cast<cudaStream_t>(stream)};
  take_request(&c.ctx);
  int st = validate_ce(dtype, T, V, D, H, ldh, W, ldw, targets);
  if (st != GEMM14_OK) return st;
  const int eb = elem_bytes_of(dtype);
  if ((dH && (lddh < D || !aligned(dH, eb))) || (dW && (lddw < D || !aligned(dW, eb))))
    return GEMM14_ERR_INVALID_ARG;
  if (T > 0 && (!lse || !dloss || !aligned(lse, 4) || !aligned(dloss, 4)))
    return GEMM14_ERR_INVALID_ARG;
  if (!dW && (!dH || T == 0)) return GEMM14_OK;  // nothing is asked for
  if ((st = call_device(&c.ctx)) != GEMM14_OK) return st;
  if (T == 0)
    return c.launched(cudaMemset2DAsync(dW, static_cast<size_t>(lddw) * eb, 0,
                                        static_cast<size_t>(D) * eb, static_cast<size_t>(V),
                                        c.stream),
                      "cudaMemset2DAsync");
  ce_layout(dtype, T, V, D, H, ldh, W, ldw, true, c.ctx.sm_count, &c.l);
  if ((st = check_room("gemm14_linear_ce_backward", workspace, workspace_bytes, c.l.total)) !=
      GEMM14_OK)
    return st;
  if (c.l.narrow) return c.backward_narrow(lse, dloss, dH, lddh, dW, lddw);
  if (c.l.tc) return c.backward_tc(lse, dloss, dH, lddh, dW, lddw);
  give_request(c.ctx);
  return c.backward_products(lse, dloss, dH, lddh, dW, lddw);
}

}  // extern "C"
