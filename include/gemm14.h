/*
 * gemm14.h -- C ABI of the GB300 (sm_103a) dense GEMM library libgemm14.so.
 *
 * Operation (all entry points): C = A * B with
 *     C[i][j] = sum_{k < K} A[i][k] * B[k][j],   0 <= i < M, 0 <= j < N,
 * the matrix product of gpu-hpc-book ch.06 "高级 cuda 特性 —— 从矩阵乘法(gemm)说起"
 * (Advanced CUDA features, starting from GEMM; opening section and
 * "缓存缺失与带宽约束分析" item (4)) and of "Kernel 优化指南" (cuda-kernel-academy
 * module 02), "GEMM 优化路径", Level 1, whose kernels take (M, N, K) and
 * row-major pointers; this interface adds leading dimensions and a stream.
 *
 * Layout: A, B and C are row-major. Element (i, k) of A is A[i * lda + k];
 * (k, j) of B is B[k * ldb + j]; (i, j) of C is C[i * ldc + j]. Leading
 * dimensions are counted in elements: lda >= K, ldb >= N, ldc >= N (each at
 * least 1). C is overwritten (alpha, beta and stored transposes: see
 * gemm14_gemm_ex); A and B are only read. C must not overlap A or B.
 * Reads of A and B stay inside each one's storage span, from its first
 * element to the last element of its last row; the 16-bit software loader
 * (operands TMA cannot address) may read padding elements between rows inside
 * that span, whose values it does not use.
 *
 * Pointers are DEVICE pointers in the current CUDA device's address space
 * (e.g. torch CUDA tensors' data_ptr()). `stream` is a cudaStream_t (NULL =
 * legacy default stream). Calls are asynchronous: the work is enqueued on
 * `stream` and the function returns without synchronising. The caller owns
 * every buffer; the library allocates and frees no device memory and keeps no
 * pointer after it returns.
 *
 * Degenerate sizes: M == 0 or N == 0 returns GEMM14_OK and launches nothing;
 * K == 0 sets the M x N block of C to zero (the empty sum).
 *
 * Errors: every entry point returns a gemm14_status and never aborts, prints
 * or exits. Invalid arguments are detected on the host before any CUDA call.
 * A device-side failure (a bounded wait inside a kernel that expired) is
 * recorded in a device error word and reported by gemm14_check_device_error.
 *
 * Only compute capability 10.3 (GB300) is supported; any other device gives
 * GEMM14_ERR_UNSUPPORTED_DEVICE. Sizes up to 2^31 - 1 per dimension.
 * Thread safety: all entry points are reentrant.
 */
#ifndef GEMM14_H
#define GEMM14_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gemm14_status {
  GEMM14_OK = 0,
  GEMM14_ERR_INVALID_ARG = 1,        /* negative or too large size, ld too small, NULL
                                        pointer with a non-empty extent, misaligned
                                        element pointer, bad dtype */
  GEMM14_ERR_UNSUPPORTED_DEVICE = 2, /* no CUDA device, or it is not compute capability 10.3 */
  GEMM14_ERR_CUDA = 3,               /* a CUDA runtime/driver call failed; see
                                        gemm14_last_error_string() */
  GEMM14_ERR_TIMEOUT = 4,            /* a kernel's bounded wait expired (device-side) */
  GEMM14_ERR_DEVICE_CHECK = 5        /* a device-side bounds check failed and its access was
                                        skipped (only a library built with
                                        GEMM14_DEVICE_CHECKS runs these checks) */
} gemm14_status;

/*
 * Element types and arithmetic, for gemm14_gemm_ex and the planning queries:
 *   F32        fp32 inputs, fp32 FMAs on the CUDA cores (gemm_f32);
 *   BF16, F16  16-bit inputs, fp32 accumulation on the tensor cores;
 *   TF32       fp32 inputs rounded to tf32 on the tensor cores (gemm_tf32_f32acc);
 *   F32_3XTF32 fp32 inputs, split tf32 arithmetic on the tensor cores that
 *              meets the fp32 bound (gemm_f32_3xtf32).
 */
enum {
  GEMM14_DTYPE_F32 = 0,
  GEMM14_DTYPE_BF16 = 1,
  GEMM14_DTYPE_F16 = 2,
  GEMM14_DTYPE_TF32 = 3,
  GEMM14_DTYPE_F32_3XTF32 = 4
};

/*
 * fp32 inputs, fp32 FFMA accumulation on the CUDA cores, fp32 output.
 * A, B, C: 4-byte aligned. The fast loader (TMA) is used when A and B are
 * 16-byte aligned and lda, ldb are multiples of 4; otherwise an equivalent
 * cp.async loader is used (same results). 16-byte stores are used for C when
 * C is 16-byte aligned and ldc is a multiple of 4.
 * A product whose 128 x 256 output tiles would fill at most half the SMs runs
 * on 64 x 64 tiles instead, the k range of each tile split over a cluster of
 * up to 8 CTAs and added up in a fixed order on chip (no workspace): its last
 * bits may differ from the large tiles' (another summation order), within the
 * same bound, and are the same with or without a workspace.
 * Follows the register-tiled, shared-memory-tiled kernels of gpu-hpc-book
 * ch.06, "矩阵乘法中的分块与数据复用" (Shared Memory Tiling, Register Tiling).
 */
int gemm_f32(int64_t M, int64_t N, int64_t K, const float* A, int64_t lda, const float* B,
             int64_t ldb, float* C, int64_t ldc, void* stream);

/*
 * bf16 inputs (raw bfloat16 bit patterns), fp32 accumulation on the tensor
 * cores (tcgen05), fp32 output. Inputs are rounded to bf16 by the caller.
 * A, B: 2-byte aligned; C: 4-byte aligned. The fast loader (TMA) reads each
 * operand that is 16-byte aligned with a leading dimension that is a multiple
 * of 8; a software loader fills the same shared-memory tiles for the other
 * operand(s) (same results, slower).
 * The tensor-core path of "Kernel 优化指南", "Level 4: Tensor Cores (WMMA)"
 * (half-precision inputs, float accumulator), and of gpu-hpc-book ch.06,
 * "Tensor Cores".
 */
int gemm_bf16_f32acc(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                     const void* B, int64_t ldb, float* C, int64_t ldc, void* stream);

/* As gemm_bf16_f32acc with IEEE binary16 (fp16) inputs. */
int gemm_f16_f32acc(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B,
                    int64_t ldb, float* C, int64_t ldc, void* stream);

/*
 * fp32 inputs on the tensor cores (tcgen05 kind::tf32, fp32 accumulation in
 * tensor memory), fp32 output. TF32 is the pages' tensor-core format for fp32
 * data (gpu-hpc-book ch.06, "Tensor Cores": fp32's 8 exponent bits, 10
 * fraction bits).
 *   gemm_tf32_f32acc: every input is read as tf32 the way the tensor cores
 *     read an fp32 operand, tf32(x) = x with its 13 low fraction bits
 *     cleared (truncation toward zero), and the products of those values are
 *     summed in fp32: against the truncated inputs, the fp32 bound; against
 *     the fp32 inputs |C - A B| <= 4e-3 (|A||B|) element-wise.
 *   gemm_f32_3xtf32: each input x is split into hi = tf32(x) and lo = x - hi
 *     (exact), and C = hi(A) hi(B) + hi(A) lo(B) + lo(A) hi(B) summed in fp32
 *     (the split-precision scheme known as 3xTF32): within the fp32 bound,
 *     |C - A B| <= 1e-5 (|A||B|), at tensor-core speed. Through
 *     gemm14_gemm_ex with a workspace of gemm14_workspace_bytes_ex bytes, lo(A)
 *     and lo(B) are first written into the workspace (with K-major copies of
 *     operands stored otherwise) and the product runs as three k sums, lo(A)
 *     hi(B), hi(A) lo(B), hi(A) hi(B), on CTA pairs: the same bound, other
 *     bits (another order of the same terms).
 * Arguments, layout and rules as gemm_f32. A and B 16-byte aligned with lda,
 * ldb multiples of 4 run on CTA pairs of tensor-core SMs (256 x 256 tiles);
 * other operands run on gemm_f32's kernel, whose exact fp32 products meet both
 * bounds. Infinite inputs give NaN where a product would be infinite (lo =
 * inf - inf), and a NaN whose payload lies only in the 13 low fraction bits
 * is read as an infinity; finite inputs whose products overflow behave as in
 * gemm_f32.
 */
int gemm_tf32_f32acc(int64_t M, int64_t N, int64_t K, const float* A, int64_t lda,
                     const float* B, int64_t ldb, float* C, int64_t ldc, void* stream);
int gemm_f32_3xtf32(int64_t M, int64_t N, int64_t K, const float* A, int64_t lda,
                    const float* B, int64_t ldb, float* C, int64_t ldc, void* stream);

/*
 * Stream-K variants. Same operation and arguments as gemm_f32 /
 * gemm_bf16_f32acc / gemm_f16_f32acc, plus a caller-owned DEVICE workspace.
 * With a workspace of at least gemm14_workspace_bytes(...) bytes, the one-SM
 * kernels split the k-blocks of the last wave and a half of output tiles
 * evenly over all SMs instead of leaving SMs idle in a partial last wave, or,
 * for products of fewer tiles than half the SMs, spread all their k-blocks
 * over the SMs (16-bit tiles over at most 4 SMs each, with 16 or more
 * k-blocks apiece) (the "stream-K" schedule): a tile shared by several SMs is finished by the
 * SM holding its first k-blocks, which adds the others' partial sums from the
 * workspace in a fixed order, so results are deterministic run to run (they
 * may differ in the last bits from the data-parallel schedule, which sums a
 * tile's k-blocks in one run). With workspace == NULL, a smaller workspace, a
 * product whose tiles fill whole waves, or one with between half and all of
 * a wave of tiles (where splitting measured slower), the call is exactly the
 * plain entry point. The CTA-pair kernel (wide 16-bit products) splits in the
 * same way with a cluster of two SMs as the worker.
 * workspace: 16-byte aligned (else GEMM14_ERR_INVALID_ARG), zero-filled
 * before its first use. Its first bytes (one 4-byte word per SM, rounded up
 * to 256 bytes) hold publication flags that only ever contain zero or the
 * number of a finished call, so a workspace may be reused by any later call,
 * of any shape, without clearing; it must not be used by two calls that may
 * run at the same time. Each flag is cleared by the one tile owner that waits
 * for it, so a call captured in a CUDA graph (its number fixed at capture) may
 * be replayed any number of times.
 * Re-pitching: an operand TMA cannot read (base or row pitch not a multiple
 * of 16 bytes) is first copied into the workspace with a 16-byte pitch when
 * the workspace has gemm14_workspace_bytes_ex(...) bytes for this call's
 * operands; the product then runs on the TMA loaders (the same kernels, and
 * the same bits, as for aligned operands). The copies lie after the stream-K
 * region, never over the flag words. With less room the call reads such an
 * operand as it is, with the element-wise loaders.
 */
int gemm_f32_ws(int64_t M, int64_t N, int64_t K, const float* A, int64_t lda, const float* B,
                int64_t ldb, float* C, int64_t ldc, void* workspace, size_t workspace_bytes,
                void* stream);
int gemm_bf16_f32acc_ws(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                        const void* B, int64_t ldb, float* C, int64_t ldc, void* workspace,
                        size_t workspace_bytes, void* stream);
int gemm_f16_f32acc_ws(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                       const void* B, int64_t ldb, float* C, int64_t ldc, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * gemm_bf16_f32acc without any device allocation by the caller or the
 * library. The pages have no counterpart to this entry point; it exists for
 * callers that may not allocate device memory: code inside a framework whose
 * memory pool has reserved the GPU and owns every allocation, plug-ins that
 * must not touch the allocator, and latency-critical paths that cannot take
 * the implicit device synchronisation of cudaMalloc / cudaFree. The caller
 * passes A, B and C exactly as for gemm_bf16_f32acc; the stream-K scratch
 * that gemm_bf16_f32acc_ws would take from the caller comes instead from a
 * 20 MiB array built into the library, which every GPU that loads the library
 * holds until the process exits. Operands that TMA cannot read are re-pitched
 * into the same array when they fit beside the split's region, as the
 * workspace entry points do with theirs. It calls no cudaMalloc, cudaFree or
 * other allocating routine.
 * Limit: a product whose split needs more than the 20 MiB returns
 * GEMM14_ERR_INVALID_ARG, and gemm14_last_error_string() says how many bytes
 * were needed (gemm_bf16_f32acc then computes it unsplit, with no scratch).
 * The largest split is one 128 x 256 fp32 slot per SM plus a flag word each,
 * so this happens only on GPUs with more than 159 SMs; on 152 SMs every
 * product runs, split exactly as gemm_bf16_f32acc_ws would split it.
 * Products that need no scratch run as gemm_bf16_f32acc.
 * Set-up: the first call on each device looks up the array's device address
 * and clears its flag words on the caller's stream; make that first call
 * before any stream capture. Every call shares the one array, which keeps the
 * last call's contents (only its flag words must start at zero, and calls
 * leave them holding finished calls' numbers): calls that may overlap on the
 * GPU race with each other and must not be issued.
 */
int gemm_bf16_f32acc_noalloc(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                             const void* B, int64_t ldb, float* C, int64_t ldc, void* stream);

/*
 * The extended product, for every element type and arithmetic (dtype =
 * GEMM14_DTYPE_*):
 *     C = alpha * op(A) * op(B) + beta * C,
 * op(A) an M x K matrix and op(B) a K x N matrix. It generalises the
 * accumulate form of the pages' asynchronous tensor-core MMA (gpu-hpc-book
 * ch.06 "高级 cuda 特性 —— 从矩阵乘法(gemm)说起", "Tensor Cores" / "wgmma":
 * D = A * B + D with either operand optionally transposed and D scaled by
 * 0 or 1) to any fp32 alpha and beta.
 * Storage (row-major throughout):
 *   transa = 0: A is stored M x K, op(A)[i][k] = A[i * lda + k], lda >= K;
 *   transa = 1: A is stored K x M, op(A)[i][k] = A[k * lda + i], lda >= M;
 *   transb = 0: B is stored K x N, op(B)[k][j] = B[k * ldb + j], ldb >= N;
 *   transb = 1: B is stored N x K, op(B)[k][j] = B[j * ldb + k], ldb >= K;
 *   C is M x N, C[i * ldc + j], ldc >= N. Any other transa / transb value is
 *   GEMM14_ERR_INVALID_ARG.
 * Arithmetic: the sum over k is formed exactly as by gemm_f32 /
 * gemm_bf16_f32acc / gemm_f16_f32acc (bit-identical for alpha = 1,
 * beta = 0, with the same workspace; 3xTF32 with a workspace sums its terms
 * in another order, see gemm_f32_3xtf32); then each element is written as
 * alpha * sum (beta == 0) or as fmaf(alpha, sum, beta * C) in fp32.
 * beta == 0: C is not read (NaN or infinity in C does not propagate).
 * K == 0 or alpha == 0: A and B are not read; C becomes beta * C (beta == 1
 * launches nothing, beta == 0 zeroes C).
 * Loaders: operands take TMA under the same alignment rules as the plain
 * entry points (16-byte aligned, pitches multiples of 16 bytes) in either
 * storage, and the equivalent software loader otherwise.
 * workspace / workspace_bytes: as for the *_ws calls (NULL, 0 allowed),
 * re-pitching included; gemm14_workspace_bytes_ex gives the bytes for these
 * operands (for TMA-addressable ones it equals gemm14_workspace_bytes(dtype,
 * M, N, K, ...), which does not depend on transa / transb).
 * Other rules (device pointers, stream, errors, degenerate sizes) as above.
 */
int gemm14_gemm_ex(int dtype, int transa, int transb, int64_t M, int64_t N, int64_t K,
                   float alpha, const void* A, int64_t lda, const void* B, int64_t ldb,
                   float beta, float* C, int64_t ldc, void* workspace, size_t workspace_bytes,
                   void* stream);

/*
 * Workspace bytes that let the *_ws call of this dtype and shape use the
 * stream-K schedule on a GPU with sm_count SMs (sm_count <= 0: the current
 * device's). 0 means the call would not split tiles (whole waves, or
 * between half and one wave of tiles) or the arguments are invalid. Assumes operands
 * TMA can address (16-byte aligned, pitches multiple of 16 bytes).
 */
size_t gemm14_workspace_bytes(int dtype, int64_t M, int64_t N, int64_t K, int sm_count);

/*
 * Workspace bytes for a gemm14_gemm_ex (or *_ws) call on exactly these
 * operands: the stream-K region as above, plus, for an operand TMA cannot
 * read, room for its copy with a 16-byte pitch (so that the call re-pitches
 * it); for TF32 and 3xTF32, room for K-major copies of operands stored
 * otherwise, and for 3xTF32 room for lo(A) and lo(B). Pointers are only inspected for their alignment, never dereferenced;
 * no CUDA call is made when sm_count > 0. 0: the call needs no workspace, or
 * the arguments are invalid.
 */
size_t gemm14_workspace_bytes_ex(int dtype, int transa, int transb, int64_t M, int64_t N,
                                 int64_t K, const void* A, int64_t lda, const void* B,
                                 int64_t ldb, const void* C, int64_t ldc, int sm_count);

/* Static text for a status code (never NULL). */
const char* gemm14_status_string(int status);

/* Text of the last CUDA failure seen by this thread ("" if none). */
const char* gemm14_last_error_string(void);

/*
 * Synchronises `stream`, then reads and clears the current device's error
 * word. Returns GEMM14_ERR_DEVICE_CHECK if a kernel of a checked build
 * skipped an access its bounds checks rejected since the last check, else
 * GEMM14_ERR_TIMEOUT if a kernel recorded an expired wait,
 * GEMM14_ERR_CUDA if the synchronisation failed, else OK.
 */
int gemm14_check_device_error(void* stream);

/*
 * Host-buffer product: C = alpha * op(A) op(B) + beta * C, as gemm14_gemm_ex,
 * with A, B and C in HOST memory, computed on the current device. The library
 * copies the operands in, runs the product and copies C back, on three
 * streams of its own (copies in, kernels, copies out), with device buffers
 * from a memory pool of its own. This call is the exception to the rules
 * above on pointers, ownership and allocation.
 *
 * Pipelining: op(A) is sent in `panels` row panels (0: the library's choice;
 * stored K x M A, transa = 1: one panel), after all of B; panel p is computed
 * once it is in and copied out once computed, while panel p + 1 goes in.
 * Consecutive calls pipeline in the same way: a call's operands go in while
 * earlier calls compute and copy out.
 *
 * Asynchrony: the call enqueues the work and returns; *ticket (not NULL)
 * names it for gemm14_host_wait. Until that wait returns, the caller must not
 * change A, B or C, nor read C. Pinned host memory (cudaHostAlloc, or pinned
 * torch tensors) gives asynchronous copies at the link's rate; pageable
 * memory works but CUDA stages its copies through pinned buffers.
 *
 * Ordering: a call whose A, B (or C when beta != 0) overlaps the C of a call
 * still in flight waits, on the device, for that call's C to be back in host
 * memory. Calls are otherwise ordered only by their streams: products run in
 * call order, and copies out finish in call order.
 *
 * Errors: invalid arguments (as gemm14_gemm_ex, with NULL host pointers where
 * they are read) are reported before anything is enqueued, with *ticket
 * untouched. Transfer or launch failures give GEMM14_ERR_CUDA. Degenerate
 * sizes enqueue nothing (M == 0 or N == 0; beta == 1 with K == 0 or
 * alpha == 0) and still return a ticket.
 * Memory: the pool keeps its buffers for reuse for the life of the process.
 */
int gemm14_gemm_host(int dtype, int transa, int transb, int64_t M, int64_t N, int64_t K,
                     float alpha, const void* A, int64_t lda, const void* B, int64_t ldb,
                     float beta, float* C, int64_t ldc, int panels, uint64_t* ticket);

/*
 * Blocks until the call named by `ticket` has its C in host memory. Returns
 * GEMM14_OK, GEMM14_ERR_TIMEOUT if a kernel of the device recorded an expired
 * wait (the device error word, read and cleared as by
 * gemm14_check_device_error), GEMM14_ERR_CUDA if the work failed, or
 * GEMM14_ERR_INVALID_ARG for a ticket never issued. A ticket already waited
 * for returns GEMM14_OK at once.
 */
int gemm14_host_wait(uint64_t ticket);

/* Waits for every host-buffer call in flight (on every device), as gemm14_host_wait. */
int gemm14_host_synchronize(void);

/*
 * Softmax cross entropy of a projection's outputs, without keeping them: with
 * z_t = H[t] W^T the V logits of row t (H is T x D, W is V x D, a row per
 * entry of the vocabulary),
 *     lse[t]  = log sum_v exp z_tv,      loss[t] = lse[t] - z_t,targets[t].
 * The logits are formed and folded away in pieces of the vocabulary; no buffer
 * of T x V values exists. Each row's statistics are held in fp32.
 * dtype: the element type of H and W and the arithmetic of the products, as
 * for gemm14_gemm_ex (F32, BF16, F16, TF32, F32_3XTF32). F32_3XTF32 here
 * splits each fp32 value into three bf16 parts (their sum is the value to 24
 * bits) and sums the six products of parts above 2^-24 of the whole: the fp32
 * bound, at tensor-core speed; an infinite input gives NaN. As the tensor cores'
 * accumulators add with truncation, sums leave them for fp32 registers: logits
 * every 512 terms or fewer, fp32 gradients and gemm14_ckpt8_wgrad every 1024, and
 * so 16-bit gradients of more than 16384 (F16) or 131072 (BF16) terms. Up to
 * 32 rows of F32 run as fp32 FMAs on the CUDA cores, and so do up to 16 of
 * F32_3XTF32, or 32 where D <= 1536.
 * loss and lse: T fp32.
 * targets: T int64 on the device. A row whose target is ignore_index takes no
 * part: its loss and lse are 0 and nothing its row of H holds is used. Any
 * other target outside [0, V) gives a loss of NaN. A NaN or +infinity among a
 * row's logits makes that row's results NaN and no other's. A logit of -infinity
 * stands for a probability of 0: the target's gives a loss of +infinity, a row of
 * nothing else an lse of -infinity and a loss of NaN. (Where W holds infinities,
 * gradients multiply them, by 0 too, which is NaN.)
 * workspace: caller-owned, 16-byte aligned, zero-filled before its first use
 * (one kept for the *_ws calls serves, and the other way round),
 * gemm14_linear_ce_workspace_bytes(...) bytes at least; a smaller one is
 * GEMM14_ERR_INVALID_ARG, and gemm14_last_error_string says how many are
 * needed. (A forward call keeps 8 bytes for each row and 128 columns, T V / 16 bytes
 * of it; the rest is bounded by pieces of the vocabulary.) A call is several launches that hand data on through it: host
 * threads that share a workspace, on one stream too, make their calls one after
 * the other (a lock around the call; the work itself stays asynchronous).
 * Sizes: T >= 0 (0: nothing is done), V >= 1, D >= 1, each at most
 * 2^31 - 256, ldh >= D, ldw >= D. Other rules (device pointers, stream, errors) as above.
 */
int gemm14_linear_ce_forward(int dtype, int64_t T, int64_t V, int64_t D, const void* H,
                             int64_t ldh, const void* W, int64_t ldw, const int64_t* targets,
                             int64_t ignore_index, float* loss, float* lse, void* workspace,
                             size_t workspace_bytes, void* stream);

/*
 * Its gradients: with dloss[t] the gradient of the caller's objective in
 * loss[t] (any reduction or weighting: 1/n for a mean over n rows) and
 *     dZ_tv = (exp(z_tv - lse[t]) - [v == targets[t]]) dloss[t],
 *     dH = dZ W  (T x D, pitch lddh),      dW = dZ^T H  (V x D, pitch lddw),
 * written in the element type of H and W. The logits are formed again, a piece
 * of the vocabulary at a time, from H, W and the forward call's lse. dH or dW
 * may be NULL: that gradient is not formed. Rows that take no part (target
 * ignore_index, or dloss[t] == 0) get dH[t] = 0 and add nothing to dW, also
 * when their rows of H hold NaN; a target outside [0, V) makes its row of dH
 * and all of dW NaN. T == 0 sets dW to zero.
 * dH and dW must not overlap each other, H or W.
 * Rounding: 16-bit dtypes hold dZ in that type (of up to 128 rows in two parts
 * of it), relative to the largest |dloss[t]|, for the two products, which accumulate in fp32; each gradient is
 * rounded once to the type. fp32 dtypes hold dZ in fp32.
 * Arguments and workspace as for the forward call.
 */
int gemm14_linear_ce_backward(int dtype, int64_t T, int64_t V, int64_t D, const void* H,
                              int64_t ldh, const void* W, int64_t ldw, const int64_t* targets,
                              int64_t ignore_index, const float* lse, const float* dloss, void* dH,
                              int64_t lddh, void* dW, int64_t lddw, void* workspace,
                              size_t workspace_bytes, void* stream);

/*
 * Workspace bytes of the forward (backward == 0) or backward call on exactly
 * these operands (pointers are only inspected for NULL and alignment; no CUDA
 * call is made when sm_count > 0). 0: T == 0, or the arguments are invalid.
 */
size_t gemm14_linear_ce_workspace_bytes(int dtype, int backward, int64_t T, int64_t V, int64_t D,
                                        const void* H, int64_t ldh, const void* W, int64_t ldw,
                                        int sm_count);

/*
 * Activations kept in 8 bits for the backward pass. Each block of 32
 * consecutive columns of a row (the last of a row may be shorter) has a scale
 * byte s, and each value a whole number q in [-127, 127]; the value kept is
 *     q * 2^(s - 133),
 * s the exponent field of the block's largest magnitude (as an fp32), at least
 * 7; q = x * 2^(133 - s) rounded to nearest, ties to even, and held at +-127.
 * So a value is off by at most 2^-7 of its block's largest magnitude (by
 * 2^-6 where it rounds to 128 and is held). s = 255: the block held an infinity
 * or a NaN; all of it is restored as NaN.
 *   save:    X (rows x cols, pitch ldx, dtype F32, BF16 or F16) -> Q (pitch
 *            ldq >= cols) and S (rows x ceil(cols / 32), pitch lds);
 *   restore: Q and S -> X in any of the three types (exact in F32 and BF16;
 *            F16 rounds, which is exact too for what was saved from F16).
 * Bases and pitches of 16 bytes give the fastest accesses; any are allowed.
 * rows or cols of 0: nothing is done. Other rules as above.
 */
int gemm14_ckpt8_save(int dtype, int64_t rows, int64_t cols, const void* X, int64_t ldx, int8_t* Q,
                      int64_t ldq, uint8_t* S, int64_t lds, void* stream);
int gemm14_ckpt8_restore(int dtype, int64_t rows, int64_t cols, const int8_t* Q, int64_t ldq,
                         const uint8_t* S, int64_t lds, void* X, int64_t ldx, void* stream);

/*
 * The weight gradient of a projection y = x W^T from its input kept in 8 bits:
 *     dW = alpha * dY^T X + beta * dW,
 * dY a T x N matrix (pitch lddy) of dtype, X the T x K values that Q and S
 * (pitches ldq, lds, as written by gemm14_ckpt8_save) stand for, dW an N x K
 * fp32 matrix (pitch lddw). dtype selects dY's element type and the product's
 * arithmetic as for gemm14_linear_ce_forward; with 16-bit types and F32_3XTF32
 * X enters the product exactly (F16: rounded where it leaves fp16's range) and
 * sums are fp32.
 * beta == 0: dW is not read; alpha == 0 or T == 0: dY and the checkpoint are
 * not read. Up to 16 rows (8 where dW's rows do not start on 16 bytes) run as
 * fp32 FMAs on the CUDA cores, TF32 aside, and need no workspace; otherwise
 * workspace: as for the *_ws calls, but needed:
 * gemm14_ckpt8_wgrad_workspace_bytes(...) bytes at least. Sizes at most
 * 2^31 - 256.
 */
int gemm14_ckpt8_wgrad(int dtype, int64_t T, int64_t N, int64_t K, float alpha, const void* dY,
                       int64_t lddy, const int8_t* Q, int64_t ldq, const uint8_t* S, int64_t lds,
                       float beta, float* dW, int64_t lddw, void* workspace,
                       size_t workspace_bytes, void* stream);

/* Its workspace bytes on these operands (0: none needed, or invalid arguments). */
size_t gemm14_ckpt8_wgrad_workspace_bytes(int dtype, int64_t T, int64_t N, int64_t K,
                                          const void* dY, int64_t lddy, const float* dW,
                                          int64_t lddw, int sm_count);

/*
 * Rows of a table looked up by token: out[t] = scale * W[tokens[t]], t < T.
 * W: V x D (pitch ldw) of dtype F32, BF16 or F16; out: T x D (pitch ldo) of
 * dtype_out, any of the three; values are multiplied in fp32 and rounded once to
 * dtype_out. tokens: T integers of token_bytes (4 or 8) bytes on the device. The
 * row of a token that is ignore_index is 0 (so it is where that is a row of the
 * table), of any other token outside [0, V) it is NaN.
 * Bases and pitches of 16 bytes give the fastest accesses; any are allowed. out
 * must not overlap W or the tokens. T == 0: nothing is done. Sizes at most
 * 2^31 - 256, V and D at least 1; scale must be finite.
 */
int gemm14_embedding_forward(int dtype, int dtype_out, int64_t T, int64_t V, int64_t D,
                             const void* W, int64_t ldw, const void* tokens, int token_bytes,
                             int64_t ignore_index, float scale, void* out, int64_t ldo,
                             void* stream);

/*
 * The gradient of a lookup in its table:
 *     dW[v] = scale * sum over {t < T : tokens[t] == v} of dY[t]  +  beta * dW[v].
 * dY: T x D (pitch lddy) of dtype F32, BF16 or F16; dW: V x D (pitch lddw) of
 * dtype_out, dtype or F32. Places whose token is ignore_index or outside [0, V)
 * add nothing, whatever their rows of dY hold. beta == 0: dW is not read, rows
 * without tokens are set to 0. beta == 1 (the gradient that is there is added to,
 * the output projection's where the two are tied, gemm14_linear_ce_backward):
 * rows without tokens are neither read nor written.
 * Sums are fp32, in an order that the tokens and the sizes fix (a call repeats
 * bit for bit); each value of dW is rounded once.
 * workspace: caller-owned, 16-byte aligned, of
 * gemm14_embedding_backward_workspace_bytes(...) bytes at least (0: none needed);
 * its contents do not matter, and one kept for other calls serves. A call is
 * several launches that hand data on through it, as for the linear cross entropy.
 * dW must not overlap dY or the tokens. T == 0: dW = beta * dW.
 */
int gemm14_embedding_backward(int dtype, int dtype_out, int64_t T, int64_t V, int64_t D,
                              const void* dY, int64_t lddy, const void* tokens, int token_bytes,
                              int64_t ignore_index, float scale, float beta, void* dW, int64_t lddw,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Its workspace bytes (0: none needed, or invalid arguments); no CUDA call is made
 * when sm_count > 0. */
size_t gemm14_embedding_backward_workspace_bytes(int dtype, int64_t T, int64_t V, int64_t D,
                                                 int sm_count);

/* A gradient in a list of them: rows x cols elements of dtype F32, BF16 or F16 on
 * the device, rows of pitch ld (not looked at where rows <= 1). rows or cols of 0:
 * it holds nothing, and data may be NULL. */
typedef struct gemm14_tensor {
  void* data;
  int64_t rows, cols, ld;
  int dtype;
} gemm14_tensor;

/*
 * The norm of n gradients taken together, N = |scale| sqrt(sum of g^2 over all
 * elements of all of them), and, where each is not NULL, that of each: norm (one
 * fp32) and each (n fp32) on the device; grads on the host, read before the call
 * returns. scale: out of a loss scale, 1 / it. Squares are summed in fp32 over at
 * most 64 values, those sums in fp64, and values whose squares fp32 does not hold
 * are squared in fp64: values of any size add what they should. A call repeats bit
 * for bit. Infinities give an infinite norm (so does a norm beyond fp32's largest
 * number), NaN gives NaN. n == 0: *norm = 0.
 * n at most 2^20; scale must be finite.
 * workspace: caller-owned, 16-byte aligned, gemm14_grad_workspace_bytes(n, ...)
 * bytes at least; its contents do not matter, and one kept for other calls serves.
 */
int gemm14_grad_norm(int64_t n, const gemm14_tensor* grads, float scale, float* norm, float* each,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * The same, and the gradients scaled so that their norm is at most max_norm:
 *     out = f g,   f = scale * min(1, max_norm / N),
 * written over them (out NULL) or into n tensors of the same sizes, each of its
 * gradient's dtype or F32. The factor is worked out on the device, in fp64, and
 * held in fp32 (in fp64 where it is below fp32's normal numbers); products are fp32,
 * rounded to the output's type. Where an element is infinite or NaN nothing is
 * clipped: f = scale, and *norm, infinite or NaN, says so. Where all are finite N is
 * finite, and clips, also beyond fp32's largest number, where *norm is infinite for
 * want of another. f == 1 in place: nothing is written. max_norm >= 0 (infinity: only
 * scale).
 * What is written must share no element with any other tensor of the lists (the
 * same tensor twice in a list is GEMM14_ERR_INVALID_ARG; an output may be its own
 * gradient, with the same layout). Tensors may lie between another's rows: a single
 * row, or rows of the same pitch in bytes; of another pitch they are refused. Each
 * pair of n such columns of a matrix is looked at on the host.
 */
int gemm14_grad_clip(int64_t n, const gemm14_tensor* grads, const gemm14_tensor* out, float scale,
                     float max_norm, float* norm, float* each, void* workspace,
                     size_t workspace_bytes, void* stream);

/* Workspace bytes of the two calls on n tensors (0: n is 0 or invalid). */
size_t gemm14_grad_workspace_bytes(int64_t n, int sm_count);

/* Launch plan chosen for a call (host-side only; no CUDA call is made). */
typedef struct gemm14_plan {
  int kernel;     /* 1 = fp32 SIMT (FFMA), 2 = tcgen05 on one SM per tile,
                     3 = tcgen05 on CTA pairs (two SMs per 256 x 256 tile),
                     4 = tcgen05 kind::tf32 on CTA pairs (TF32 / 3xTF32),
                     5 = kernel 3 with kind::tf32 MMAs (TF32, A stored M x K and B
                         stored N x K: both read as stored),
                     6 = fp32 FFMA on 64 x 64 tiles, the k range of each tile split
                         over a cluster of grid / tiles CTAs (products whose
                         128 x 256 tiles would fill at most half the SMs; with a
                         workspace, only those of at most 2^30 FLOP),
                     0 = no launch */
  int loader;     /* 1 = TMA (kernel 6: 16-byte cp.async), 2 = software loader
                     (cp.async for fp32; kernel 6: 4-byte cp.async); kernel 2
                     only: 3 = software loader for A and TMA for B, 4 = TMA for
                     A and software loader for B; 0 = none */
  int bm, bn, bk; /* output tile rows x columns, k-block depth */
  int stages;     /* shared-memory ring depth (kernel 4: operand stages the converter
                     warps fill, 4 for TF32 and 2 for 3xTF32) */
  int threads;    /* threads per CTA */
  int smem_bytes; /* dynamic shared memory per CTA */
  int vec_store;  /* 1 if C takes 16-byte stores */
  int64_t tiles;  /* output tiles */
  int grid;       /* CTAs launched (persistent: min(tiles, sm_count); for kernel 3,
                     2 x min(tiles, sm_count / 2); for kernel 6, tiles x the
                     cluster size) */
} gemm14_plan;

/*
 * Fills *plan with what the matching gemm_* call would launch on a GPU with
 * `sm_count` SMs. Validates arguments exactly like the entry points (pointers
 * are only inspected for NULL and alignment, never dereferenced). Returns a
 * gemm14_status; makes no CUDA call.
 */
int gemm14_plan_gemm(int dtype, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                     const void* B, int64_t ldb, const void* C, int64_t ldc, int sm_count,
                     gemm14_plan* plan);

/* As gemm14_plan_gemm for a gemm14_gemm_ex call with these transposes. */
int gemm14_plan_gemm_ex(int dtype, int transa, int transb, int64_t M, int64_t N, int64_t K,
                        const void* A, int64_t lda, const void* B, int64_t ldb, const void* C,
                        int64_t ldc, int sm_count, gemm14_plan* plan);

/*
 * The 16-bit entry points compute 256 x 256 output tiles on pairs of SMs
 * (a cluster of two CTAs sharing each tile's B operand) when the operands are
 * TMA-addressable and M, N > 128; otherwise tiles on one SM, of 128 rows, or
 * of 64 rows when the 128-row tiles would be fewer than the SMs. The kernels
 * accumulate in the same order and give bit-identical results.
 * gemm14_set_pair_kernel(0) restricts all later calls in the process to the
 * one-SM kernel, (1) allows pairs again (the default); returns the previous
 * setting. If pairs cannot be launched on the device the library falls back
 * to the one-SM kernel by itself.
 */
int gemm14_set_pair_kernel(int enable);

/*
 * Failure-detection hook for tests. The NEXT gemm_* call made by this thread
 * runs with the given fault mode and per-wait time limit, then both reset:
 *   fault 0 = none; 1 = the kernel's producer never loads its first shared-
 *   memory stage, so every wait for that stage expires after wait_limit_ns,
 *   the kernel records GEMM14_ERR_TIMEOUT in the device error word, drains
 *   its in-flight copies and exits; C is left incomplete.
 *   wait_limit_ns = 0 keeps the default limit (2 s).
 * No fault makes the GPU fault, trap or hang: waits are bounded, the context
 * stays usable, and gemm14_check_device_error reports the timeout.
 * The fp32 small-product kernel (plan kernel 6) synchronises only through
 * block and cluster barriers, with no mbarrier wait to expire: a call that
 * runs on it consumes the request and computes C as usual; so do
 * gemm14_linear_ce_* calls of fp32 rows that run on the CUDA cores and
 * gemm14_ckpt8_wgrad calls of up to 16 rows. (gemm14_ckpt8_save and _restore, gemm14_embedding_* and
 * gemm14_grad_* wait for nothing but barriers and leave the request to the next call.)
 * Returns GEMM14_ERR_INVALID_ARG for an unknown mode.
 */
int gemm14_debug_inject(int fault, uint64_t wait_limit_ns);

/*
 * The number of the CUDA graph capture that `stream` is part of (distinct for
 * every capture of the process), 0: it is not being captured. A workspace that
 * is made during a capture, and zero-filled in the graph, serves the calls of
 * that capture on that stream and no others: this tells them apart.
 */
uint64_t gemm14_capture_id(void* stream);

/* Library version, major * 10000 + minor * 100 + patch. */
int gemm14_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GEMM14_H */
