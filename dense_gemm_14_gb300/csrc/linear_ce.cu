// linear_ce.cu -- softmax cross entropy of a projection's outputs over a large
// vocabulary, without keeping the outputs: with z_t = H[t] W^T (V logits of
// row t), y_t the row's target and g_t the gradient of the caller's objective
// in loss_t,
//     lse_t  = log sum_v exp z_tv          loss_t = lse_t - z_t,y(t)
//     dZ_tv  = (exp(z_tv - lse_t) - [v = y_t]) g_t
//     dH     = dZ W                        dW     = dZ^T H.
// The logits exist only a piece of the vocabulary at a time: the forward pass
// folds each piece into a running maximum and sum per row, the backward pass
// forms each piece again from H, W and lse_t, turns it into dZ and multiplies
// it into dH (summed over the pieces in fp32) and into the piece's rows of dW.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/gemm14.h"
#include "api_internal.h"
#include "kernels.h"
#include "plan.h"
#include "ptx.cuh"

namespace gemm14 {
namespace {

constexpr int kThreads = 256;

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

// Sum of exponentials held as top + log(sum): (m, l) stands for l exp(m).
struct ExpSum {
  float m, l;
};
__device__ __forceinline__ ExpSum merge(ExpSum a, ExpSum b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return {m, a.l + b.l};  // no term above -inf (NaN sums are kept)
  return {m, a.l * __expf(a.m - m) + b.l * __expf(b.m - m)};
}

// ---- row passes over a piece of logits (Z: T x C, pitch ldz, columns v0 ..)

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

// dZ of a piece, as fp32 in place of the logits or rounded to 16 bits beside them.
template <typename G>
__global__ void __launch_bounds__(kThreads)
    ce_grad_kernel(const float* Z, int64_t ldz, G* out, int64_t ldg, int64_t C, int64_t v0,
                   const int64_t* targets, const float* lse, const float* coef) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t t = blockIdx.x;
  const float k = coef[t], top = lse[t];
  const int64_t y = targets[t] - v0;
  for (int64_t c = threadIdx.x; c < C; c += kThreads) {
    float d = 0.0f;
    if (k != 0.0f) d = (__expf(Z[t * ldz + c] - top) - (c == y ? 1.0f : 0.0f)) * k;
    out[t * ldg + c] = from_f32<G>(d);
  }
}

// ---- before and after the backward products

// Each row's coefficient g_t, 0 for a row that takes no part and NaN for a
// target that is no row of W. For 16-bit dZ it is g_t / ref * unit with
// ref = max |g_t| over the rows that take part: dZ then lies in [-unit, unit]
// whatever the scale of the objective, and the products are multiplied by
// ref / unit (*back) at the end. One block.
__global__ void __launch_bounds__(1024)
    ce_coef_kernel(const int64_t* targets, int64_t ignore, const float* g, int64_t T, int64_t V,
                   bool relative, float unit, float* coef, float* back) {
  __shared__ float part[32];
  grid_dependency_wait();
  grid_launch_dependents();
  float ref = 0.0f;
  if (relative) {
    for (int64_t t = threadIdx.x; t < T; t += blockDim.x)
      if (targets[t] != ignore) ref = fmaxf(ref, fabsf(g[t]));
    for (int o = 16; o; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ref;
    __syncthreads();
    ref = 0.0f;
    for (int w = 0; w < 32; ++w) ref = fmaxf(ref, part[w]);
  }
  if (!(ref > 0.0f && ref < INFINITY)) ref = 1.0f;
  for (int64_t t = threadIdx.x; t < T; t += blockDim.x) {
    const int64_t y = targets[t];
    const float k = y < 0 || y >= V ? __uint_as_float(0x7fc00000u) : g[t] / ref * unit;
    coef[t] = y == ignore ? 0.0f : k;
  }
  if (threadIdx.x == 0) *back = ref / unit;
}

// H with the rows that take no part set to zero, so that nothing they hold
// (uninitialised padding, a NaN) reaches dW.
template <typename E>
__global__ void __launch_bounds__(kThreads)
    ce_rows_kernel(const E* H, int64_t ldh, const float* coef, E* out, int64_t ldo, int64_t D) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t t = blockIdx.x;
  const bool off = coef[t] == 0.0f;
  for (int64_t c = threadIdx.x; c < D; c += kThreads)
    out[t * ldo + c] = off ? E(0) : H[t * ldh + c];
}

// out = x * back, rows with coefficient 0 set to zero (coef null: none).
template <typename E>
__global__ void __launch_bounds__(kThreads)
    ce_out_kernel(const float* X, int64_t ldx, const float* coef, const float* back, E* out,
                  int64_t ldo, int64_t cols) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t t = blockIdx.x;
  const bool off = coef && coef[t] == 0.0f;
  const float k = *back;
  for (int64_t c = threadIdx.x; c < cols; c += kThreads)
    out[t * ldo + c] = from_f32<E>(off ? 0.0f : X[t * ldx + c] * k);
}

// ---- host side

bool size_ok(int64_t n) { return n >= 0 && n <= INT32_MAX; }
bool is_16bit(int dtype) { return dtype == GEMM14_DTYPE_BF16 || dtype == GEMM14_DTYPE_F16; }

int validate_ce(int dtype, int64_t T, int64_t V, int64_t D, const void* H, int64_t ldh,
                const void* W, int64_t ldw, const int64_t* targets) {
  if (!size_ok(T) || !size_ok(V) || !size_ok(D) || V < 1 || D < 1) return GEMM14_ERR_INVALID_ARG;
  if (T > 0 && (!targets || !aligned(targets, 8))) return GEMM14_ERR_INVALID_ARG;
  // the product's own checks; the logits (in the workspace) are always sound
  const void* sound = reinterpret_cast<const void*>(uintptr_t(1) << 12);
  return validate_product(dtype, 0, 1, T, V, D, H, ldh, W, ldw, sound, V);
}

struct CeLayout {
  int64_t C = 0;       // vocabulary rows of a piece
  int64_t ldz = 0;     // pitch of the logits (fp32) and of dZ
  int64_t ldx = 0;     // pitch of the D-wide buffers
  size_t state = 0, coef = 0, back = 0, z = 0, g = 0, rows = 0, dh = 0, dw = 0, total = 0;
};

// Bytes of logits a piece may take: 256 MiB, a piece of 8192 columns for 8192 rows.
constexpr int64_t kPieceBytes = int64_t(256) << 20;

void ce_layout(int dtype, int64_t T, int64_t V, int64_t D, const void* H, int64_t ldh,
               const void* W, int64_t ldw, bool backward, int sms, CeLayout* l) {
  const int eb = elem_bytes_of(dtype);
  int64_t C = kPieceBytes / (4 * T) / 256 * 256;
  C = std::max<int64_t>(C, 256);
  l->C = std::min(C, V);
  l->ldz = (l->C + 7) / 8 * 8;
  l->ldx = (D + 7) / 8 * 8;
  const void* own = reinterpret_cast<const void*>(uintptr_t(1) << 12);
  size_t product = streamk_flag_bytes(sms);
  auto need = [&](int ta, int tb, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                  const void* B, int64_t ldb, int64_t ldc) {
    product = std::max(product, gemm14_workspace_bytes_ex(dtype, ta, tb, M, N, K, A, lda, B, ldb,
                                                          own, ldc, sms));
  };
  const int64_t last = V - (V - 1) / l->C * l->C;
  for (const int64_t c : {l->C, last}) {
    need(0, 1, T, c, D, H, ldh, W, ldw, l->ldz);
    if (!backward) continue;
    need(0, 0, T, D, c, own, l->ldz, W, ldw, l->ldx);
    need(1, 0, c, D, T, own, l->ldz, own, l->ldx, l->ldx);
  }
  size_t at = round256(product);
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = round256(at + bytes);
    return here;
  };
  l->state = take(static_cast<size_t>(T) * 3 * sizeof(float));
  l->z = take(static_cast<size_t>(T) * l->ldz * sizeof(float));
  if (backward) {
    l->coef = take(static_cast<size_t>(T) * sizeof(float));
    l->back = take(sizeof(float));
    l->g = is_16bit(dtype) ? take(static_cast<size_t>(T) * l->ldz * eb) : l->z;
    l->rows = take(static_cast<size_t>(T) * l->ldx * eb);
    l->dh = take(static_cast<size_t>(T) * l->ldx * sizeof(float));
    l->dw = take(static_cast<size_t>(l->C) * l->ldx * sizeof(float));
  }
  l->total = at;
}

size_t ce_workspace(int dtype, int64_t T, int64_t V, int64_t D, const void* H, int64_t ldh,
                    const void* W, int64_t ldw, bool backward, int sms) {
  CeLayout l;
  ce_layout(dtype, T, V, D, H, ldh, W, ldw, backward, sms, &l);
  return l.total;
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

template <typename E>
cudaError_t out_rows(const float* X, int64_t ldx, const float* coef, const float* back, void* out,
                     int64_t ldo, int64_t rows, int64_t cols, cudaStream_t stream) {
  return launch_kernel(ce_out_kernel<E>, dim3(static_cast<unsigned>(rows)), dim3(kThreads), 0,
                       stream, X, ldx, coef, back, static_cast<E*>(out), ldo, cols);
}
cudaError_t out_rows(int dtype, const float* X, int64_t ldx, const float* coef, const float* back,
                     void* out, int64_t ldo, int64_t rows, int64_t cols, cudaStream_t stream) {
  switch (dtype) {
    case GEMM14_DTYPE_BF16:
      return out_rows<__nv_bfloat16>(X, ldx, coef, back, out, ldo, rows, cols, stream);
    case GEMM14_DTYPE_F16:
      return out_rows<__half>(X, ldx, coef, back, out, ldo, rows, cols, stream);
    default: return out_rows<float>(X, ldx, coef, back, out, ldo, rows, cols, stream);
  }
}

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
  return ce_workspace(dtype, T, V, D, H, ldh, W, ldw, backward != 0, sm_count);
}

int gemm14_linear_ce_forward(int dtype, int64_t T, int64_t V, int64_t D, const void* H,
                             int64_t ldh, const void* W, int64_t ldw, const int64_t* targets,
                             int64_t ignore_index, float* loss, float* lse, void* workspace,
                             size_t workspace_bytes, void* stream_ptr) {
  int st = validate_ce(dtype, T, V, D, H, ldh, W, ldw, targets);
  if (st != GEMM14_OK) return st;
  if (T == 0) return GEMM14_OK;
  if (!loss || !lse || !aligned(loss, 4) || !aligned(lse, 4)) return GEMM14_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = current_sm_count(&sms)) != GEMM14_OK) return st;
  CeLayout l;
  ce_layout(dtype, T, V, D, H, ldh, W, ldw, false, sms, &l);
  if ((st = check_room("gemm14_linear_ce_forward", workspace, workspace_bytes, l.total)) !=
      GEMM14_OK)
    return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  char* ws = static_cast<char*>(workspace);
  const int eb = elem_bytes_of(dtype);
  float* z = reinterpret_cast<float*>(ws + l.z);
  float* state = reinterpret_cast<float*>(ws + l.state);
  const RowState rs{state, state + T, state + 2 * T};
  for (int64_t v0 = 0; v0 < V; v0 += l.C) {
    const int64_t c = std::min(l.C, V - v0);
    if ((st = product_on_stream(dtype, 0, 1, T, c, D, 1.0f, H, ldh, row_of(W, v0, ldw, eb), ldw,
                                0.0f, z, l.ldz, workspace, l.state, stream)) != GEMM14_OK)
      return st;
    if ((st = finish_launch(launch_kernel(ce_stats_kernel, dim3(static_cast<unsigned>(T)),
                                          dim3(kThreads), 0, stream, z, l.ldz, c, v0, V, targets,
                                          ignore_index, rs, loss, lse),
                            "linear_ce statistics launch", stream)) != GEMM14_OK)
      return st;
  }
  return GEMM14_OK;
}

int gemm14_linear_ce_backward(int dtype, int64_t T, int64_t V, int64_t D, const void* H,
                              int64_t ldh, const void* W, int64_t ldw, const int64_t* targets,
                              int64_t ignore_index, const float* lse, const float* dloss, void* dH,
                              int64_t lddh, void* dW, int64_t lddw, void* workspace,
                              size_t workspace_bytes, void* stream_ptr) {
  int st = validate_ce(dtype, T, V, D, H, ldh, W, ldw, targets);
  if (st != GEMM14_OK) return st;
  const int eb = elem_bytes_of(dtype);
  if ((dH && (lddh < D || !aligned(dH, eb))) || (dW && (lddw < D || !aligned(dW, eb))))
    return GEMM14_ERR_INVALID_ARG;
  if (T > 0 && (!lse || !dloss || !aligned(lse, 4) || !aligned(dloss, 4)))
    return GEMM14_ERR_INVALID_ARG;
  if (!dW && (!dH || T == 0)) return GEMM14_OK;  // nothing is asked for
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if (T == 0) {
    int sms = 0;
    if ((st = current_sm_count(&sms)) != GEMM14_OK) return st;
    return finish_launch(cudaMemset2DAsync(dW, static_cast<size_t>(lddw) * eb, 0,
                                           static_cast<size_t>(D) * eb, static_cast<size_t>(V),
                                           stream),
                         "cudaMemset2DAsync", stream);
  }
  int sms = 0;
  if ((st = current_sm_count(&sms)) != GEMM14_OK) return st;
  CeLayout l;
  ce_layout(dtype, T, V, D, H, ldh, W, ldw, true, sms, &l);
  if ((st = check_room("gemm14_linear_ce_backward", workspace, workspace_bytes, l.total)) !=
      GEMM14_OK)
    return st;
  char* ws = static_cast<char*>(workspace);
  float* z = reinterpret_cast<float*>(ws + l.z);
  float* coef = reinterpret_cast<float*>(ws + l.coef);
  float* back = reinterpret_cast<float*>(ws + l.back);
  float* dh = reinterpret_cast<float*>(ws + l.dh);
  float* dw = reinterpret_cast<float*>(ws + l.dw);
  void* rows = ws + l.rows;
  void* g = ws + l.g;
  const bool half = is_16bit(dtype);
  // fp16's range: dZ is held in units of 2^-15, so that probabilities down to
  // 2^-39 of the largest coefficient are not lost
  const float unit = dtype == GEMM14_DTYPE_F16 ? 32768.0f : 1.0f;
  const dim3 per_row(static_cast<unsigned>(T)), block(kThreads);
  if ((st = finish_launch(launch_kernel(ce_coef_kernel, dim3(1), dim3(1024), 0, stream, targets,
                                        ignore_index, dloss, T, V, half, unit, coef, back),
                          "linear_ce coefficient launch", stream)) != GEMM14_OK)
    return st;
  const cudaError_t e =
      half ? launch_kernel(ce_rows_kernel<uint16_t>, per_row, block, 0, stream,
                           static_cast<const uint16_t*>(H), ldh, coef,
                           static_cast<uint16_t*>(rows), l.ldx, D)
           : launch_kernel(ce_rows_kernel<float>, per_row, block, 0, stream,
                           static_cast<const float*>(H), ldh, coef, static_cast<float*>(rows),
                           l.ldx, D);
  if ((st = finish_launch(e, "linear_ce rows launch", stream)) != GEMM14_OK) return st;
  for (int64_t v0 = 0; v0 < V; v0 += l.C) {
    const int64_t c = std::min(l.C, V - v0);
    const void* w = row_of(W, v0, ldw, eb);
    if ((st = product_on_stream(dtype, 0, 1, T, c, D, 1.0f, H, ldh, w, ldw, 0.0f, z, l.ldz,
                                workspace, l.state, stream)) != GEMM14_OK)
      return st;
    const cudaError_t eg =
        dtype == GEMM14_DTYPE_BF16
            ? launch_kernel(ce_grad_kernel<__nv_bfloat16>, per_row, block, 0, stream, z, l.ldz,
                            static_cast<__nv_bfloat16*>(g), l.ldz, c, v0, targets, lse, coef)
        : dtype == GEMM14_DTYPE_F16
            ? launch_kernel(ce_grad_kernel<__half>, per_row, block, 0, stream, z, l.ldz,
                            static_cast<__half*>(g), l.ldz, c, v0, targets, lse, coef)
            : launch_kernel(ce_grad_kernel<float>, per_row, block, 0, stream, z, l.ldz,
                            static_cast<float*>(g), l.ldz, c, v0, targets, lse, coef);
    if ((st = finish_launch(eg, "linear_ce gradient launch", stream)) != GEMM14_OK) return st;
    if (dH && (st = product_on_stream(dtype, 0, 0, T, D, c, 1.0f, g, l.ldz, w, ldw,
                                      v0 ? 1.0f : 0.0f, dh, l.ldx, workspace, l.state, stream)) !=
                  GEMM14_OK)
      return st;
    if (!dW) continue;
    if ((st = product_on_stream(dtype, 1, 0, c, D, T, 1.0f, g, l.ldz, rows, l.ldx, 0.0f, dw, l.ldx,
                                workspace, l.state, stream)) != GEMM14_OK)
      return st;
    void* out = static_cast<char*>(dW) + v0 * lddw * eb;
    if ((st = finish_launch(out_rows(dtype, dw, l.ldx, nullptr, back, out, lddw, c, D, stream),
                            "linear_ce output launch", stream)) != GEMM14_OK)
      return st;
  }
  if (!dH) return GEMM14_OK;
  return finish_launch(out_rows(dtype, dh, l.ldx, coef, back, dH, lddh, T, D, stream),
                       "linear_ce output launch", stream);
}

}  // extern "C"
