// api_internal.h -- what the entry points outside api.cu (host_path.cu,
// ckpt8.cu, linear_ce.cu) use of the C-ABI layer. Nothing here crosses the
// library boundary.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace gemm14 {

// gemm14_gemm_ex on `stream` with device pointers (its own checks included).
int product_on_stream(int dtype, int transa, int transb, int64_t M, int64_t N, int64_t K,
                      float alpha, const void* A, int64_t lda, const void* B, int64_t ldb,
                      float beta, float* C, int64_t ldc, void* workspace,
                      size_t workspace_bytes, cudaStream_t stream);

// The argument checks of gemm14_gemm_ex; the pointers may be host pointers.
int validate_product(int dtype, int transa, int transb, int64_t M, int64_t N, int64_t K,
                     const void* A, int64_t lda, const void* B, int64_t ldb, const void* C,
                     int64_t ldc);

// Workspace bytes with which such a call on these device operands would use
// the stream-K schedule on the current device (0: it would not split); for
// TF32 and 3xTF32 also the room for their K-major copies and lo parts.
size_t product_workspace_bytes(int dtype, int transa, int transb, int64_t M, int64_t N, int64_t K,
                               const void* A, int64_t lda, const void* B, int64_t ldb,
                               const void* C, int64_t ldc);

// Bytes per element of A and B for a gemm14_dtype (4 or 2).
int operand_bytes(int dtype);

// Share of the worker slots kept busy by such a call on the current device,
// with dense device operands (pitches rounded to 16 bytes) and a workspace:
// 1 when it runs the stream-K schedule, else tiles / (waves x workers).
double schedule_efficiency(int dtype, int transa, int transb, int64_t M, int64_t N, int64_t K);

// The current device's index, checked as by every entry point (a gemm14_status).
int current_device_index(int* device);

// Reads and clears the current device's error word once its kernels are
// known to be done: GEMM14_OK, GEMM14_ERR_TIMEOUT or GEMM14_ERR_CUDA.
int take_device_error();

// The current device's SM count, checked as by every entry point (a gemm14_status).
int current_sm_count(int* sm_count);

// What a call's own kernels need: this thread's pending gemm14_debug_inject
// request, which the call takes at its start, whatever its outcome (take_request;
// give_request hands it on to the products the call is made of), and the current
// device (call_device, a gemm14_status).
struct CallContext {
  int sm_count = 0;
  unsigned* err = nullptr;              // the device error word
  unsigned long long wait_limit_ns = 0;
  int fault = 0;
};
void take_request(CallContext* c);
void give_request(const CallContext& c);
int call_device(CallContext* c);

// A row-major rows x cols matrix of 16-bit elements (pitch ld) as a tensor map
// of boxes 64 columns wide and box_rows high, 128-byte swizzle, zeros out of range.
int map_16bit(CUtensorMap* map, bool bf16, const void* base, int64_t rows, int64_t cols,
              int64_t ld, int box_rows);

// The status of a launch on `stream`: a CUDA failure is recorded as this
// thread's last error; with GEMM14_DEBUG set, the device error word is read.
int finish_launch(cudaError_t e, const char* what, cudaStream_t stream);

// Records a message (printf-style) as this thread's last error text.
void note_error(const char* format, ...);

// Records a CUDA failure as this thread's last error text.
void note_cuda_error(const char* what, cudaError_t e);

}  // namespace gemm14
