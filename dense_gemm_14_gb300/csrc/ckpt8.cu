// ckpt8.cu -- activations kept in 8 bits for the backward pass, and the
// weight gradient formed from them. The format, per block of 32 consecutive
// columns of a row (the last block of a row may be shorter):
//     scale byte s, q[j] in [-127, 127], a value stands for q[j] 2^(s - 133),
// s the exponent field of the block's largest magnitude as an fp32 (so that
// |x| 2^(133 - s) < 128), at least 7, and 255 for a block that holds an
// infinity or a NaN (every value of it then stands for NaN).
// A power of two as the scale makes q 2^(s - 133) exact in bf16 and fp32 (7
// significant bits, s >= 7 keeps it a normal number), so a product formed from
// the restored values adds no error of its own; a value is off by at most
// half a step of its block, 2^-7 of the block's largest magnitude, or by one
// step where the largest rounds up to 128 and is held at 127.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/gemm14.h"
#include "api_internal.h"
#include "elements.cuh"
#include "kernels.h"
#include "operand_copy.cuh"
#include "plan.h"
#include "ptx.cuh"
#include "train_tc.h"

namespace gemm14 {
namespace {

constexpr int kBlock = 32;       // columns that share a scale
constexpr int kThreads = 256;

// The scale byte of a block whose largest magnitude has these fp32 bits (a
// NaN's bits, sign cleared, compare above every number's).
__device__ __forceinline__ uint32_t scale_byte(uint32_t top_bits) {
  const uint32_t e = top_bits >> 23;
  return e < 7u ? 7u : e;
}
// x in steps of the block: round to nearest even, held within [-127, 127].
// factor = 2^(133 - s); a block of byte 255 is kept as zeros.
__device__ __forceinline__ float scale_factor(uint32_t s) {
  return s == 255u ? 0.0f : __uint_as_float((260u - s) << 23);
}
__device__ __forceinline__ int quantise(float x, float factor) {
  const int q = __float2int_rn(x * factor);
  return max(-127, min(127, q));
}
// Two values at once, each in the low byte of its result: one packed multiply
// and add of 1.5 2^23 rounds x factor to the nearest whole number, ties to even,
// in the low bits of the sum (the product is exact, so there is one rounding).
__device__ __forceinline__ void quantise2(uint32_t a, uint32_t b, float factor, uint32_t& qa,
                                          uint32_t& qb) {
  asm("{\n\t.reg .b64 x, f, m;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 f, {%4, %4};\n\tmov.b64 m, {%5, %5};\n\t"
      "fma.rn.f32x2 x, x, f, m;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=r"(qa), "=r"(qb)
      : "r"(a), "r"(b), "f"(factor), "f"(12582912.0f));
}
// Two whole numbers u = q + 128, each as the fp32 2^23 + u, to q times its
// block's step (less 2^23 + 128 first: the step times that may leave fp32's range).
__device__ __forceinline__ void scale2(uint32_t a, uint32_t b, float step_a, float step_b,
                                       float& xa, float& xb) {
  asm("{\n\t.reg .b64 x, s, o;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 s, {%4, %5};\n\tmov.b64 o, {%6, %6};\n\t"
      "add.rn.f32x2 x, x, o;\n\tmul.rn.f32x2 x, x, s;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(xa), "=f"(xb)
      : "r"(a), "r"(b), "f"(step_a), "f"(step_b), "f"(-8388736.0f));
}
// Four low bytes as one word.
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// The fp32 bits, sign cleared, of the largest magnitude among a piece's values:
// magnitudes of a 16-bit type are ordered as whole numbers, two at a time.
__device__ __forceinline__ uint32_t top_of(const uint4& v, float) {
  return max(max(v.x & 0x7fffffffu, v.y & 0x7fffffffu), max(v.z & 0x7fffffffu, v.w & 0x7fffffffu));
}
__device__ __forceinline__ uint32_t top16(const uint4& v) {
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                              __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}
__device__ __forceinline__ uint32_t top_of(const uint4& v, __nv_bfloat16) {
  return top16(v) << 16;
}
__device__ __forceinline__ uint32_t top_of(const uint4& v, __half) {
  return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(top16(v))))) &
         0x7fffffffu;
}
// 2^(s - 133), NaN for byte 255; bytes below 7, which save never writes, count as 7.
__device__ __forceinline__ float step_of(uint32_t s) {
  return s == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float((max(s, 7u) - 6u) << 23);
}

// A thread's place in a matrix of rows x per_row items taken in order, moved on
// by a fixed step without dividing again.
struct Place {
  int64_t row, item;
  __device__ Place(int64_t i, int64_t per_row) : row(i / per_row), item(i - row * per_row) {}
  __device__ void move(const Place& step, int64_t per_row) {
    row += step.row;
    item += step.item;
    if (item >= per_row) {
      item -= per_row;
      ++row;
    }
  }
};

// Wide forms: a lane moves a piece of 16 bytes of X (8 or 4 values; 4 or 8 lanes
// a block, whose largest magnitude they find with two or three shuffles) and 8
// or 4 bytes of Q. Rows of X that do not start on 16 bytes are read as two
// aligned words and a shift; restore writes the aligned pieces of its rows and
// reads Q with the shift. (Where Q's rows do not start on 8 or 4 bytes, save is
// a warp a block and a lane a column.) The passes should be bound by memory,
// and what held them back was their instructions (21 a value, 72 % of the issue
// slots): so a thread keeps to its place in the rows and steps by whole rows (no
// division, no multiply in the loop), two values share an instruction where
// they can, and q is only clamped where the block's largest value rounds to
// 128. kAhead loads are in flight before the first is used. 16384 x 11008 bf16,
// 547 MB each way: save 140 -> 99 us, restore 93 -> 83 (6.6 TB/s).
constexpr int kUnroll = 8, kAhead = 6;  // (kUnroll: of the element form)

template <typename T>
__host__ __device__ constexpr int piece_values() { return 16 / static_cast<int>(sizeof(T)); }

template <typename T>
union Piece {
  uint4 raw;
  T x[16 / sizeof(T)];
};

// Threads along a row of so many pieces, a power of two: as many as leave each
// kAhead pieces, the block's other threads taking other rows (8 at least: a
// block's lanes stay together); more where the rows are too few for the SMs.
int threads_along(int64_t rows, int64_t pieces, int sms) {
  int x = 8;
  while (x < kThreads && x * kAhead < pieces) x *= 2;
  while (x < kThreads && x < pieces && rows * x < static_cast<int64_t>(sms) * 1024) x *= 2;
  return x;
}

// A piece's values as fp32 bits, and back.
__device__ __forceinline__ void unpack(const Piece<float>& p, uint32_t (&x)[4]) {
  x[0] = p.raw.x;
  x[1] = p.raw.y;
  x[2] = p.raw.z;
  x[3] = p.raw.w;
}
__device__ __forceinline__ void unpack(const Piece<__nv_bfloat16>& p, uint32_t (&x)[8]) {
  const uint32_t w[4] = {p.raw.x, p.raw.y, p.raw.z, p.raw.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = w[j] << 16;
    x[2 * j + 1] = w[j] & 0xffff0000u;
  }
}
__device__ __forceinline__ void unpack(const Piece<__half>& p, uint32_t (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = __float_as_uint(__half2float(p.x[j]));
}
__device__ __forceinline__ void pack(const float (&x)[4], Piece<float>& p) {
#pragma unroll
  for (int j = 0; j < 4; ++j) p.x[j] = x[j];
}
__device__ __forceinline__ void pack(const float (&x)[8], Piece<__nv_bfloat16>& p) {
  uint32_t* w = &p.raw.x;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&v);
  }
}
__device__ __forceinline__ void pack(const float (&x)[8], Piece<__half>& p) {
  uint32_t* w = &p.raw.x;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2 v = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

// kAny: X at any address and pitch.
template <typename T, bool kAny>
__global__ void __launch_bounds__(kThreads)
    ckpt8_save_vec_kernel(const T* X, int64_t ldx, int8_t* Q, int64_t ldq, uint8_t* S, int64_t lds,
                          int64_t rows, uint32_t cols, int along) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int kPer = piece_values<T>(), kLanes = kBlock / kPer;
  const int tx = threadIdx.x & (along - 1), ty = threadIdx.x / along;
  const int64_t row_step = static_cast<int64_t>(gridDim.x) * (kThreads / along);
  // pieces of a row, whole blocks: every lane of a warp goes round as often (the
  // shuffles need every lane of a block)
  const uint32_t pieces = (cols + kBlock - 1) / kBlock * kLanes;
  const uint32_t turns = (pieces + along * kAhead - 1) / (along * kAhead);
  int64_t r = static_cast<int64_t>(blockIdx.x) * (kThreads / along) + ty;
  const int64_t rounds = (rows + row_step - 1) / row_step;
  const T* xr = X + r * ldx;
  const T* end = X + (rows - 1) * ldx + cols;
  int8_t* qr = Q + r * ldq;
  uint8_t* sr = S + r * lds;
  for (int64_t round = 0; round < rounds; ++round) {
    const bool in_rows = r < rows;
    for (uint32_t turn = 0; turn < turns; ++turn) {
      const uint32_t p0 = tx + turn * along * kAhead;
      Piece<T> p[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const uint32_t c = (p0 + u * along) * kPer;
        p[u].raw = make_uint4(0, 0, 0, 0);
        if (in_rows && c + kPer <= cols && (!kAny || words_inside(xr + c, 16, X, end))) {
          p[u].raw = kAny ? load16_any(xr + c) : __ldcs(reinterpret_cast<const uint4*>(xr + c));
        } else if (in_rows && c < cols) {
#pragma unroll
          for (int j = 0; j < kPer; ++j)
            if (c + j < cols) p[u].x[j] = xr[c + j];
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const uint32_t c = (p0 + u * along) * kPer;
        uint32_t top = top_of(p[u].raw, T());
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (!in_rows || c >= cols) continue;
        const uint32_t s = scale_byte(top);
        const float factor = scale_factor(s);
        uint32_t x[kPer], w[kPer / 4];
        unpack(p[u], x);
        if (__uint_as_float(top) * factor >= 127.5f || s == 255u) {
          // the largest rounds to 128, or the block is kept as zeros (an infinity
          // times 0 is no number)
          const float most = s == 255u ? 0.0f : 127.0f / factor;
#pragma unroll
          for (int j = 0; j < kPer; ++j)
            x[j] = s == 255u ? 0u
                             : __float_as_uint(fminf(fmaxf(__uint_as_float(x[j]), -most), most));
        }
#pragma unroll
        for (int k = 0; k < kPer / 4; ++k) {
          uint32_t q[4];
          quantise2(x[4 * k], x[4 * k + 1], factor, q[0], q[1]);
          quantise2(x[4 * k + 2], x[4 * k + 3], factor, q[2], q[3]);
          w[k] = pack4(q[0], q[1], q[2], q[3]);
        }
        int8_t* to = qr + c;
        if (c + kPer <= cols) {
          if constexpr (kPer == 8)
            *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
          else
            *reinterpret_cast<uint32_t*>(to) = w[0];
        } else {
#pragma unroll
          for (int j = 0; j < kPer; ++j)
            if (c + j < cols) to[j] = static_cast<int8_t>(w[j / 4] >> (8 * (j % 4)));
        }
        if ((tx & (kLanes - 1)) == 0) sr[c / kBlock] = static_cast<uint8_t>(s);
      }
    }
    r += row_step;
    xr += row_step * ldx;
    qr += row_step * ldq;
    sr += row_step * lds;
  }
}

// kAny: X and Q at any address and pitch. Column c of a piece is then its
// place in X's aligned words, from -(values before the row in its first word).
// The grid's blocks past `blocks` copy another operand of the product that
// follows, where there is one.
template <typename T, bool kAny>
__global__ void __launch_bounds__(kThreads)
    ckpt8_restore_kernel(const int8_t* Q, int64_t ldq, const uint8_t* S, int64_t lds, T* X,
                         int64_t ldx, int64_t rows, int64_t cols, int along, int blocks,
                         const OperandCopy other) {
  grid_dependency_wait();
  grid_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= blocks) {
    operand_copy(other, blockIdx.x - blocks, gridDim.x - blocks);
    return;
  }
  constexpr int kPer = piece_values<T>();
  const int tx = threadIdx.x & (along - 1), ty = threadIdx.x / along;
  const int64_t row_step = static_cast<int64_t>(blocks) * (kThreads / along);
  int64_t r = static_cast<int64_t>(blockIdx.x) * (kThreads / along) + ty;
  const int8_t* qr = Q + r * ldq;
  const int8_t* end = Q + (rows - 1) * ldq + cols;
  const uint8_t* sr = S + r * lds;
  T* xr = X + r * ldx;
  for (; r < rows; r += row_step, qr += row_step * ldq, sr += row_step * lds, xr += row_step * ldx) {
    const int before =
        kAny ? static_cast<int>(reinterpret_cast<uintptr_t>(xr) & 15u) / static_cast<int>(sizeof(T))
             : 0;
    for (int64_t c0 = tx * kPer - before; c0 < cols; c0 += along * kAhead * kPer) {
      uint32_t w[kAhead][kPer / 4], s[kAhead][kAny ? 2 : 1];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int64_t c = c0 + u * along * kPer;
        s[u][0] = 7u;
        if (kAny) s[u][kAny ? 1 : 0] = 7u;
#pragma unroll
        for (int j = 0; j < kPer / 4; ++j) w[u][j] = 0u;
        if (c >= cols) continue;
        s[u][0] = sr[max(c, int64_t(0)) / kBlock];
        if (kAny) s[u][kAny ? 1 : 0] = sr[min(c + kPer, cols) > 0 ? (min(c + kPer, cols) - 1) / kBlock : 0];
        if (c >= 0 && c + kPer <= cols && (!kAny || words_inside(qr + c, kPer, Q, end))) {
          if constexpr (kPer == 8) {
            const uint2 v = kAny ? load8_any(qr + c) : __ldcs(reinterpret_cast<const uint2*>(qr + c));
            w[u][0] = v.x;
            w[u][1] = v.y;
          } else {
            w[u][0] = kAny ? load4_any(qr + c) : __ldcs(reinterpret_cast<const uint32_t*>(qr + c));
          }
        } else {
#pragma unroll
          for (int j = 0; j < kPer; ++j)
            if (c + j >= 0 && c + j < cols)
              w[u][j / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(qr[c + j])) << (8 * (j % 4));
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int64_t c = c0 + u * along * kPer;
        if (c >= cols) break;
        // a piece holds columns of one block, or (kAny) of two: those from `split` on
        const float step0 = step_of(s[u][0]), step1 = step_of(s[u][kAny ? 1 : 0]);
        const int split = kAny ? kBlock - static_cast<int>(max(c, int64_t(0)) % kBlock) -
                                     static_cast<int>(min(c, int64_t(0)))
                               : kBlock;
        const auto step = [&](int j) { return !kAny || j < split ? step0 : step1; };
        float x[kPer];
#pragma unroll
        for (int k = 0; k < kPer / 4; ++k) {
          const uint32_t v = w[u][k] ^ 0x80808080u;  // q + 128 in each byte
          scale2(__byte_perm(v, 0x4b000000u, 0x7440), __byte_perm(v, 0x4b000000u, 0x7441),
                 step(4 * k), step(4 * k + 1), x[4 * k], x[4 * k + 1]);
          scale2(__byte_perm(v, 0x4b000000u, 0x7442), __byte_perm(v, 0x4b000000u, 0x7443),
                 step(4 * k + 2), step(4 * k + 3), x[4 * k + 2], x[4 * k + 3]);
        }
        Piece<T> p;
        pack(x, p);
        T* to = xr + c;
        if (c >= 0 && c + kPer <= cols) {
          *reinterpret_cast<uint4*>(to) = p.raw;
        } else {
#pragma unroll
          for (int j = 0; j < kPer; ++j)
            if (c + j >= 0 && c + j < cols) to[j] = p.x[j];
        }
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    ckpt8_save_kernel(const T* X, int64_t ldx, int8_t* Q, int64_t ldq, uint8_t* S, int64_t lds,
                      int64_t rows, int64_t cols) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t per_row = (cols + kBlock - 1) / kBlock;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  const Place step(warps, per_row);
  Place at(static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5), per_row);
  while (at.row < rows) {
    float x[kUnroll];
    Place place[kUnroll] = {at, at, at, at, at, at, at, at};
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      place[u] = at;
      const int64_t c = at.item * kBlock + lane;
      x[u] = at.row < rows && c < cols ? to_f32(X[at.row * ldx + c]) : 0.0f;
      at.move(step, per_row);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t r = place[u].row, b = place[u].item, c = b * kBlock + lane;
      if (r >= rows) break;
      const uint32_t s = scale_byte(
          __reduce_max_sync(0xffffffffu, __float_as_uint(x[u]) & 0x7fffffffu));
      if (c < cols)
        Q[r * ldq + c] = static_cast<int8_t>(s == 255u ? 0 : quantise(x[u], scale_factor(s)));
      if (lane == 0) S[r * lds + b] = static_cast<uint8_t>(s);
    }
  }
}

// Blocks for `threads_needed` threads of one item each, at most 8 an SM.
int grid_for(int64_t threads_needed, int sm_count) {
  const int64_t blocks = (threads_needed + kThreads - 1) / kThreads;
  const int64_t cap = static_cast<int64_t>(sm_count) * 8;
  return static_cast<int>(blocks < cap ? blocks : cap);
}

// Whether rows start on `bytes` bytes (elements of `size` bytes).
bool rows_on(const void* p, int64_t ld, int size, int bytes) {
  return aligned(p, bytes) && ld * size % bytes == 0;
}

template <typename T>
cudaError_t save_as(const void* X, int64_t ldx, int8_t* Q, int64_t ldq, uint8_t* S, int64_t lds,
                    int64_t rows, int64_t cols, int sms, cudaStream_t stream) {
  constexpr int kPer = piece_values<T>();
  const int64_t blocks = (cols + kBlock - 1) / kBlock;
  const T* x = static_cast<const T*>(X);
  if (!rows_on(Q, ldq, 1, kPer))
    return launch_kernel(ckpt8_save_kernel<T>, dim3(grid_for(rows * blocks * 32, sms)),
                         dim3(kThreads), 0, stream, x, ldx, Q, ldq, S, lds, rows, cols);
  const int along = threads_along(rows, blocks * kBlock / kPer, sms);
  const auto kernel = rows_on(X, ldx, sizeof(T), 16) ? ckpt8_save_vec_kernel<T, false>
                                                     : ckpt8_save_vec_kernel<T, true>;
  return launch_kernel(kernel, dim3(grid_for(rows * along, sms)), dim3(kThreads), 0, stream, x, ldx,
                       Q, ldq, S, lds, rows, static_cast<uint32_t>(cols), along);
}
template <typename T>
cudaError_t restore_as(const int8_t* Q, int64_t ldq, const uint8_t* S, int64_t lds, void* X,
                       int64_t ldx, int64_t rows, int64_t cols, const OperandCopy& other, int sms,
                       cudaStream_t stream) {
  constexpr int kPer = piece_values<T>();
  T* x = static_cast<T*>(X);
  const bool any = !rows_on(X, ldx, sizeof(T), 16) || !rows_on(Q, ldq, 1, kPer);
  const int64_t pieces = (cols + (any ? kPer - 1 : 0) + kPer - 1) / kPer;
  const int along = threads_along(rows, pieces, sms);
  const auto kernel = any ? ckpt8_restore_kernel<T, true> : ckpt8_restore_kernel<T, false>;
  const int blocks = grid_for(rows * along, sms);
  const int more = other.rows > 0 ? operand_copy_blocks(other, sms) : 0;
  return launch_kernel(kernel, dim3(blocks + more), dim3(kThreads), 0, stream, Q, ldq, S, lds, x,
                       ldx, rows, cols, along, blocks, other);
}

// other: an operand to copy beside it (rows = 0: none).
cudaError_t launch_restore(int dtype, const int8_t* Q, int64_t ldq, const uint8_t* S, int64_t lds,
                           void* X, int64_t ldx, int64_t rows, int64_t cols,
                           const OperandCopy& other, int sms, cudaStream_t stream) {
  switch (dtype) {
    case GEMM14_DTYPE_BF16:
      return restore_as<__nv_bfloat16>(Q, ldq, S, lds, X, ldx, rows, cols, other, sms, stream);
    case GEMM14_DTYPE_F16:
      return restore_as<__half>(Q, ldq, S, lds, X, ldx, rows, cols, other, sms, stream);
    default: return restore_as<float>(Q, ldq, S, lds, X, ldx, rows, cols, other, sms, stream);
  }
}

bool size_ok(int64_t n) { return n >= 0 && n <= INT32_MAX; }
int64_t at_least_one(int64_t n) { return n > 1 ? n : 1; }

// X, Q and S of save and restore.
int validate_ckpt8(int dtype, int64_t rows, int64_t cols, const void* X, int64_t ldx,
                   const void* Q, int64_t ldq, const void* S, int64_t lds) {
  if (dtype != GEMM14_DTYPE_F32 && dtype != GEMM14_DTYPE_BF16 && dtype != GEMM14_DTYPE_F16)
    return GEMM14_ERR_INVALID_ARG;
  if (!size_ok(rows) || !size_ok(cols)) return GEMM14_ERR_INVALID_ARG;
  if (ldx < at_least_one(cols) || ldq < at_least_one(cols) ||
      lds < at_least_one((cols + kBlock - 1) / kBlock))
    return GEMM14_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return GEMM14_OK;
  if (!X || !Q || !S || !aligned(X, elem_bytes_of(dtype))) return GEMM14_ERR_INVALID_ARG;
  return GEMM14_OK;
}

// ---- the weight gradient of a handful of rows, on the CUDA cores

// dW = alpha dY^T X (+ beta dW) of T <= 16 rows reads and writes dW and little
// else, so memory bounds it: a thread holds its 4 columns of X, from the
// checkpoint, in registers and goes down dW with 4 kT fp32 FMAs (two to an
// instruction) for each 16 bytes, dY's values coming from shared memory, the next
// rows of dW in flight meanwhile (without that, and with single FMAs, it took
// 37.6 us for the 29.5 below). One launch and no copy of X or dY, against two or
// three on the tensor cores, whose epilogue moves dW at 3.9 TB/s: 16 x 4096 x 4096
// fp16, added, 36.4 -> 29.5 us (4.6 TB/s with the launch).
// `along` threads (a power of two, 32 at least) side by side take 4 along
// columns, the block's others other rows. kVec: dW's rows start on 16 bytes, and
// a thread's columns lie together; else they lie `along` apart, so that a warp's
// accesses do. Sums of T products in fp32.
constexpr int kNarrowRows = 16;
constexpr int kNarrowDown = 64;  // rows of dW between two loads of dY
constexpr int kNarrowAhead = 4;  // rows of dW in flight beside the 4 at work

__device__ __forceinline__ void fma2(uint64_t& s, uint64_t d, uint64_t x) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(s) : "l"(d), "l"(x));
}
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  return static_cast<uint64_t>(__float_as_uint(b)) << 32 | __float_as_uint(a);
}

template <typename T, int kT, bool kVec, bool kAdd>
__global__ void __launch_bounds__(kThreads, 2)
    ckpt8_wgrad_narrow_kernel(const T* dY, int64_t lddy, const int8_t* Q, int64_t ldq,
                              const uint8_t* S, int64_t lds, float* dW, int64_t lddw, int rows,
                              int64_t N, int64_t K, float alpha, float beta, int along,
                              int64_t across, int64_t share) {
  __shared__ __align__(16) float2 dy[kNarrowDown][kT];  // each value twice
  grid_dependency_wait();
  grid_launch_dependents();
  const int tx = threadIdx.x & (along - 1), ty = threadIdx.x / along;
  const int step = kThreads / along;
  const int64_t part = blockIdx.x / across, n_begin = part * share;
  const int64_t n_end = min(N, n_begin + share);
  const int64_t c0 = (blockIdx.x - part * across) * (4 * static_cast<int64_t>(along));
  int64_t col[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) col[j] = c0 + (kVec ? 4 * tx + j : tx + j * along);
  const bool q_words = kVec && col[3] < K && ((reinterpret_cast<uintptr_t>(Q) | ldq) & 3) == 0;
  uint64_t x[kT][2];
  {
    uint32_t q[kT], sc[kT][kVec ? 1 : 4];
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      q[t] = 0u;
#pragma unroll
      for (int j = 0; j < (kVec ? 1 : 4); ++j) sc[t][j] = 7u;
      if (t >= rows) continue;
      if (q_words) {
        q[t] = *reinterpret_cast<const uint32_t*>(Q + t * ldq + col[0]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (col[j] < K)
            q[t] |= static_cast<uint32_t>(static_cast<uint8_t>(Q[t * ldq + col[j]])) << (8 * j);
      }
#pragma unroll
      for (int j = 0; j < (kVec ? 1 : 4); ++j)
        if (col[j] < K) sc[t][j] = S[t * lds + col[j] / kBlock];
    }
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = to_f32(from_f32<T>(static_cast<float>(static_cast<int8_t>(q[t] >> (8 * j))) *
                                  step_of(sc[t][kVec ? 0 : j])));
      x[t][0] = pair_of(v[0], v[1]);
      x[t][1] = pair_of(v[2], v[3]);
    }
  }
  for (int64_t n0 = n_begin; n0 < n_end; n0 += kNarrowDown) {
    const int down = static_cast<int>(min(static_cast<int64_t>(kNarrowDown), n_end - n0));
    float old[kNarrowAhead][4];
    const auto load = [&](int u0) {
#pragma unroll
      for (int a = 0; a < kNarrowAhead; ++a) {
        const int u = u0 + a * step;
        const float* from = dW + (n0 + u) * lddw;
        if (kVec && u < down && col[3] < K) {
          const float4 v = __ldcs(reinterpret_cast<const float4*>(from + col[0]));
          old[a][0] = v.x;
          old[a][1] = v.y;
          old[a][2] = v.z;
          old[a][3] = v.w;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) old[a][j] = u < down && col[j] < K ? from[col[j]] : 0.0f;
        }
      }
    };
    if constexpr (kAdd) load(ty);
    __syncthreads();
    for (int i = threadIdx.x; i < kNarrowDown * kT; i += kThreads) {
      const int v = i % kNarrowDown, t = i / kNarrowDown;
      const float d = t < rows && n0 + v < n_end ? to_f32(dY[t * lddy + n0 + v]) : 0.0f;
      dy[v][t] = make_float2(d, d);
    }
    __syncthreads();
    for (int u0 = ty; u0 < down; u0 += kNarrowAhead * step) {
      float was[kNarrowAhead][4];
      if constexpr (kAdd) {
#pragma unroll
        for (int a = 0; a < kNarrowAhead; ++a)
#pragma unroll
          for (int j = 0; j < 4; ++j) was[a][j] = old[a][j];
        load(u0 + kNarrowAhead * step);
      }
#pragma unroll
      for (int a = 0; a < kNarrowAhead; ++a) {
        const int u = u0 + a * step;
        if (u >= down) break;
        uint64_t s2[2] = {0u, 0u};
        const ulonglong2* d = reinterpret_cast<const ulonglong2*>(dy[u]);
#pragma unroll
        for (int t = 0; t < kT; t += 2) {
          const ulonglong2 two = d[t / 2];
          fma2(s2[0], two.x, x[t][0]);
          fma2(s2[1], two.x, x[t][1]);
          fma2(s2[0], two.y, x[t + 1][0]);
          fma2(s2[1], two.y, x[t + 1][1]);
        }
        float s[4] = {__uint_as_float(static_cast<uint32_t>(s2[0])),
                      __uint_as_float(static_cast<uint32_t>(s2[0] >> 32)),
                      __uint_as_float(static_cast<uint32_t>(s2[1])),
                      __uint_as_float(static_cast<uint32_t>(s2[1] >> 32))};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[j] *= alpha;
          if constexpr (kAdd) s[j] = fmaf(beta, was[a][j], s[j]);
        }
        float* to = dW + (n0 + u) * lddw;
        if (kVec && col[3] < K) {
          *reinterpret_cast<float4*>(to + col[0]) = make_float4(s[0], s[1], s[2], s[3]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (col[j] < K) to[col[j]] = s[j];
        }
      }
    }
  }
}

// Whether dW's rows start on 16 bytes.
bool wide_rows(const float* dW, int64_t lddw) { return aligned(dW, 16) && lddw % 4 == 0; }

// Up to 16 rows, which is what a thread's registers hold (4096 x 4096 fp16, added,
// 16 rows: 29.8 us against 36.8 on the tensor cores, which take as long for 17 to
// 48), and half as many where dW takes 4-byte accesses (bf16 4001 x
// 4099, added: 5 rows 42.6 us against 52.5, 16 rows 61.4 against 53.7; 4096 x 4096:
// 5 rows 30.7 against 39.6, 16 rows 34.1 against 39.5, with cold caches). TF32 asks
// for the tensor cores' rounding of dY, and keeps it.
bool wgrad_narrow(int dtype, int64_t T, const float* dW, int64_t lddw) {
  return T <= (wide_rows(dW, lddw) ? kNarrowRows : kNarrowRows / 2) && dtype != GEMM14_DTYPE_TF32;
}

template <typename T, int kT, bool kVec, bool kAdd>
cudaError_t launch_narrow_wgrad(const T* dY, int64_t lddy, const int8_t* Q, int64_t ldq,
                                const uint8_t* S, int64_t lds, float* dW, int64_t lddw, int rows,
                                int64_t N, int64_t K, float alpha, float beta, int sms,
                                cudaStream_t stream) {
  int along = 32;
  while (along < kThreads && 4 * along < K) along *= 2;
  const int64_t across = (K + 4 * along - 1) / (4 * along);
  // one wave of blocks, each with rows enough for its threads
  const int64_t blocks = static_cast<int64_t>(sms) * 2;
  const int64_t least = kNarrowAhead / 2 * (kThreads / along);
  int64_t splits = blocks / across > 1 ? blocks / across : 1;
  if (splits > (N + least - 1) / least) splits = (N + least - 1) / least;
  const int64_t share = (N + splits - 1) / splits, parts = (N + share - 1) / share;
  return launch_kernel(ckpt8_wgrad_narrow_kernel<T, kT, kVec, kAdd>,
                       dim3(static_cast<unsigned>(parts * across)), dim3(kThreads), 0, stream, dY,
                       lddy, Q, ldq, S, lds, dW, lddw, rows, N, K, alpha, beta, along, across,
                       share);
}
template <typename T>
cudaError_t narrow_wgrad_as(const void* dY, int64_t lddy, const int8_t* Q, int64_t ldq,
                            const uint8_t* S, int64_t lds, float* dW, int64_t lddw, int64_t rows,
                            int64_t N, int64_t K, float alpha, float beta, int sms,
                            cudaStream_t stream) {
  const bool vec = wide_rows(dW, lddw), add = beta != 0.0f;
  const auto run = [&](auto kernel) {
    return kernel(static_cast<const T*>(dY), lddy, Q, ldq, S, lds, dW, lddw,
                  static_cast<int>(rows), N, K, alpha, beta, sms, stream);
  };
  if (rows <= 4)
    return run(vec ? add ? launch_narrow_wgrad<T, 4, true, true> : launch_narrow_wgrad<T, 4, true, false>
                   : add ? launch_narrow_wgrad<T, 4, false, true> : launch_narrow_wgrad<T, 4, false, false>);
  if (rows <= 8)
    return run(vec ? add ? launch_narrow_wgrad<T, 8, true, true> : launch_narrow_wgrad<T, 8, true, false>
                   : add ? launch_narrow_wgrad<T, 8, false, true> : launch_narrow_wgrad<T, 8, false, false>);
  return run(add ? launch_narrow_wgrad<T, 16, true, true> : launch_narrow_wgrad<T, 16, true, false>);
}

// ---- the weight gradient: restored values (and dY, where it is copied) in the
// workspace, then a product

// 16-bit dY, and fp32 dY in the split-precision mode (as three bf16 parts),
// run on the tensor-core kernel of train_tc.cu; the FFMA and TF32 modes on the
// library's products, with the values restored in fp32.
struct WgradLayout {
  bool narrow = false;     // a handful of rows, on the CUDA cores (no workspace)
  bool tc = false;
  int parts = 1;           // bf16 parts of dY
  bool copy_dy = false;    // dY is copied (unaligned) or split
  int64_t ldx = 0, lddy = 0;
  int64_t slot_count = 0;  // for split tiles
  size_t x_off = 0, dy_off = 0, slots_off = 0, total = 0;
};

void wgrad_layout(int dtype, int64_t T, int64_t N, int64_t K, const void* dY, int64_t lddy,
                  const float* dW, int64_t lddw, int sms, WgradLayout* l) {
  *l = WgradLayout{};
  l->narrow = wgrad_narrow(dtype, T, dW, lddw);
  if (l->narrow) return;
  l->tc = dtype != GEMM14_DTYPE_F32 && dtype != GEMM14_DTYPE_TF32;
  size_t at = streamk_flag_bytes(sms);
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = round256(at + bytes);
    return here;
  };
  if (!l->tc) {
    l->ldx = (K + 3) / 4 * 4;
    const void* notional = reinterpret_cast<const void*>(uintptr_t(1) << 12);
    const size_t product = gemm14_workspace_bytes_ex(dtype, 1, 0, N, K, T, dY, lddy, notional,
                                                     l->ldx, dW, lddw, sms);
    at = round256(product > at ? product : at);
    l->x_off = take(static_cast<size_t>(T) * l->ldx * 4);
    l->total = at;
    return;
  }
  l->parts = dtype == GEMM14_DTYPE_F32_3XTF32 ? 3 : 1;
  l->copy_dy = l->parts == 3 || !aligned(dY, 16) || lddy % 8 != 0;
  l->ldx = (K + 7) / 8 * 8;
  l->lddy = l->copy_dy ? (N + 7) / 8 * 8 : lddy;
  l->x_off = take(static_cast<size_t>(T) * l->ldx * 2);
  if (l->copy_dy) l->dy_off = take(static_cast<size_t>(T) * l->lddy * 2 * l->parts);
  const int clusters = sms > 1 ? sms / 2 : 1;
  l->slot_count = slots_needed(((N + 255) / 256) * ((K + 127) / 128), (T + 63) / 64, clusters,
                               false);
  l->slots_off = take(static_cast<size_t>(l->slot_count) * kSlotBytes);
  l->total = at;
}

bool product_size_ok(int64_t T, int64_t N, int64_t K) {
  return T >= 0 && N >= 0 && K >= 0 && T <= kTrainMaxSize && N <= kTrainMaxSize &&
         K <= kTrainMaxSize;
}

int validate_wgrad(int dtype, int64_t T, int64_t N, int64_t K, const void* dY, int64_t lddy,
                   const int8_t* Q, int64_t ldq, const uint8_t* S, int64_t lds, const float* dW,
                   int64_t lddw) {
  if (!product_size_ok(T, N, K)) return GEMM14_ERR_INVALID_ARG;
  if (ldq < at_least_one(K) || lds < at_least_one((K + kBlock - 1) / kBlock))
    return GEMM14_ERR_INVALID_ARG;
  const bool reads = T > 0 && N > 0 && K > 0;
  // the product's own checks; its second operand (in the workspace) is always sound
  const void* sound = reinterpret_cast<const void*>(uintptr_t(1) << 12);
  const int st = validate_product(dtype, 1, 0, N, K, T, dY, lddy, sound, at_least_one(K), dW, lddw);
  if (st != GEMM14_OK) return st;
  if (reads && (!Q || !S)) return GEMM14_ERR_INVALID_ARG;
  return GEMM14_OK;
}

int wgrad_tc(int dtype, int64_t T, int64_t N, int64_t K, float alpha, const void* dY,
             int64_t lddy, float beta, float* dW, int64_t lddw, char* ws, const WgradLayout& l,
             const CallContext& ctx, cudaStream_t stream) {
  int st;
  const int clusters = train_max_clusters();
  if (clusters <= 0) {
    note_error("gemm14_ckpt8_wgrad: clusters of two CTAs cannot run on this device");
    return GEMM14_ERR_CUDA;
  }
  const void* dy = l.copy_dy ? ws + l.dy_off : dY;
  TrainArgs a{};
  a.M = static_cast<int>(N);
  a.N = static_cast<int>(K);
  a.K = static_cast<int>(T);
  a.width = tile_width((T + 63) / 64 * (l.parts == 3 ? 3 : 1));
  a.split_k = a.K;
  a.err = ctx.err;
  a.wait_limit_ns = ctx.wait_limit_ns;
  a.fault = ctx.fault;
  a.alpha = alpha;
  a.beta = beta;
  a.out = dW;
  a.ld_out = lddw;
  a.elem = kElemF32;
  a.out_vec = wide_rows(dW, lddw);
  a.slots = reinterpret_cast<float4*>(ws + l.slots_off);
  a.slot_count = l.slot_count;
  a.out_rows = N;
  a.out_cols = K;
  TrainMaps maps;
  const TrainOperand A{dy, T, N, l.lddy, l.parts, T * l.lddy};
  const TrainOperand B{ws + l.x_off, T, K, l.ldx, 1, 0};
  if ((st = train_operands(dtype != GEMM14_DTYPE_F16, A, true, B, true, &maps, &a)) != GEMM14_OK)
    return st;
  const bool promote = T > TrainShape::CHUNK * TrainShape::BK;
  st = finish_launch(launch_train_tc(kTrainOut, promote, maps, a, clusters, stream),
                     "ckpt8 product launch", stream);
  if (st != GEMM14_OK || !may_split(a, clusters)) return st;
  const SlotsOut s{false, nullptr, alpha, beta, nullptr, dW, lddw, kElemF32, N};
  return finish_launch(launch_slots_out(a, s, clusters, stream), "ckpt8 output launch", stream);
}

}  // namespace
}  // namespace gemm14

using namespace gemm14;

extern "C" {

int gemm14_ckpt8_save(int dtype, int64_t rows, int64_t cols, const void* X, int64_t ldx, int8_t* Q,
                      int64_t ldq, uint8_t* S, int64_t lds, void* stream_ptr) {
  int st = validate_ckpt8(dtype, rows, cols, X, ldx, Q, ldq, S, lds);
  if (st != GEMM14_OK || rows == 0 || cols == 0) return st;
  int sms = 0;
  if ((st = current_sm_count(&sms)) != GEMM14_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  const cudaError_t e =
      dtype == GEMM14_DTYPE_BF16
          ? save_as<__nv_bfloat16>(X, ldx, Q, ldq, S, lds, rows, cols, sms, stream)
      : dtype == GEMM14_DTYPE_F16 ? save_as<__half>(X, ldx, Q, ldq, S, lds, rows, cols, sms, stream)
                                  : save_as<float>(X, ldx, Q, ldq, S, lds, rows, cols, sms, stream);
  return finish_launch(e, "ckpt8 save launch", stream);
}

int gemm14_ckpt8_restore(int dtype, int64_t rows, int64_t cols, const int8_t* Q, int64_t ldq,
                         const uint8_t* S, int64_t lds, void* X, int64_t ldx, void* stream_ptr) {
  int st = validate_ckpt8(dtype, rows, cols, X, ldx, Q, ldq, S, lds);
  if (st != GEMM14_OK || rows == 0 || cols == 0) return st;
  int sms = 0;
  if ((st = current_sm_count(&sms)) != GEMM14_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  return finish_launch(
      launch_restore(dtype, Q, ldq, S, lds, X, ldx, rows, cols, OperandCopy{}, sms, stream),
      "ckpt8 restore launch", stream);
}

size_t gemm14_ckpt8_wgrad_workspace_bytes(int dtype, int64_t T, int64_t N, int64_t K,
                                          const void* dY, int64_t lddy, const float* dW,
                                          int64_t lddw, int sm_count) {
  if (sm_count <= 0 && current_sm_count(&sm_count) != GEMM14_OK) return 0;
  const void* sound = reinterpret_cast<const void*>(uintptr_t(1) << 12);
  if (!product_size_ok(T, N, K) ||
      validate_product(dtype, 1, 0, N, K, T, dY, lddy, sound, at_least_one(K), dW, lddw) !=
          GEMM14_OK ||
      T == 0 || N == 0 || K == 0)
    return 0;
  WgradLayout l;
  wgrad_layout(dtype, T, N, K, dY, lddy, dW, lddw, sm_count, &l);
  return l.total;
}

int gemm14_ckpt8_wgrad(int dtype, int64_t T, int64_t N, int64_t K, float alpha, const void* dY,
                       int64_t lddy, const int8_t* Q, int64_t ldq, const uint8_t* S, int64_t lds,
                       float beta, float* dW, int64_t lddw, void* workspace,
                       size_t workspace_bytes, void* stream_ptr) {
  CallContext ctx;
  take_request(&ctx);
  int st = validate_wgrad(dtype, T, N, K, dY, lddy, Q, ldq, S, lds, dW, lddw);
  if (st != GEMM14_OK) return st;
  if (workspace && !aligned(workspace, 16)) return GEMM14_ERR_INVALID_ARG;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if (T == 0 || N == 0 || K == 0 || alpha == 0.0f)  // no product term: dW = beta dW
    return product_on_stream(dtype, 1, 0, N, K, 0, alpha, nullptr, at_least_one(N), nullptr,
                             at_least_one(K), beta, dW, lddw, nullptr, 0, stream);
  if ((st = call_device(&ctx)) != GEMM14_OK) return st;
  const int sms = ctx.sm_count;
  WgradLayout l;
  wgrad_layout(dtype, T, N, K, dY, lddy, dW, lddw, sms, &l);
  if (l.narrow) {
    const auto launch = dtype == GEMM14_DTYPE_BF16  ? narrow_wgrad_as<__nv_bfloat16>
                        : dtype == GEMM14_DTYPE_F16 ? narrow_wgrad_as<__half>
                                                    : narrow_wgrad_as<float>;
    return finish_launch(launch(dY, lddy, Q, ldq, S, lds, dW, lddw, T, N, K, alpha, beta, sms,
                                stream),
                         "ckpt8 narrow product launch", stream);
  }
  if (!workspace || workspace_bytes < l.total) {
    note_error("gemm14_ckpt8_wgrad: %zu bytes of workspace given, %zu needed", workspace_bytes,
               l.total);
    return GEMM14_ERR_INVALID_ARG;
  }
  char* ws = static_cast<char*>(workspace);
  void* X = ws + l.x_off;
  const int kept_as = !l.tc ? GEMM14_DTYPE_F32 : l.parts == 3 ? GEMM14_DTYPE_BF16 : dtype;
  const OperandCopy dy{dY, lddy, l.copy_dy ? T : 0, N, ws + l.dy_off, l.lddy, T * l.lddy, l.parts};
  const cudaError_t e = launch_restore(kept_as, Q, ldq, S, lds, X, l.ldx, T, K, dy, sms, stream);
  if (e != cudaSuccess) return finish_launch(e, "ckpt8 restore launch", stream);
  if (l.tc) return wgrad_tc(dtype, T, N, K, alpha, dY, lddy, beta, dW, lddw, ws, l, ctx, stream);
  give_request(ctx);
  return product_on_stream(dtype, 1, 0, N, K, T, alpha, dY, lddy, X, l.ldx, beta, dW, lddw,
                           workspace, l.x_off, stream);
}

}  // extern "C"
