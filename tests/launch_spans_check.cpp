// Host check of what the training calls' launches are told to write: the
// library's own objects, linked with a CUDA runtime that records launches in
// place of running them. Over a sweep of sizes, types and pitches, in one and
// in several pieces of the vocabulary, every buffer that a launch of the tensor
// core kernels fills lies inside the workspace that the query asked for, holds
// what its tiles leave, and lies apart from the buffers that have to survive it.
//
//     launch_spans_check        (exit status 0: all spans are sound)
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <map>
#include <string>
#include <vector>

#include <cuda_runtime.h>

#include "../../include/gemm14.h"
#include "train_tc.h"

using namespace gemm14;

// ---- the recording runtime

namespace {
struct Launch {
  std::string name;
  TrainArgs args;      // of the tensor core kernels
  int few_width = 0;   // of the kernel for few rows
  const void* part = nullptr;  // of ce_combine_kernel
  int64_t part_ld = 0;
  int parts = 0;
  OperandCopy copy{};  // of operand_copy_kernel
};
std::map<const void*, std::string>& kernels() {
  static std::map<const void*, std::string> k;
  return k;
}
std::vector<Launch> g_launches;
unsigned g_err;
int fake_encode() { return 0; }
}  // namespace

extern "C" {
void** __cudaRegisterFatBinary(void*) { static void* h; return &h; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, void*, void*,
                            void*, void*, int*) {
  kernels()[host] = name;
}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
unsigned __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return 0; }
cudaError_t __cudaGetKernel(cudaKernel_t*, const void*) { return cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) {
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void* func, void** a) {
  Launch l;
  l.name = kernels()[func];
  const auto has = [&](const char* s) { return l.name.find(s) != std::string::npos; };
  if (has("train_tc_kernel") || has("train_few_kernel"))
    std::memcpy(static_cast<void*>(&l.args), a[1], sizeof l.args);
  if (has("train_few_kernel")) l.few_width = *static_cast<int*>(a[2]);
  if (has("ce_combine_kernel")) {
    l.part = *static_cast<void**>(a[0]);
    l.part_ld = *static_cast<int64_t*>(a[1]);
    l.parts = *static_cast<int*>(a[2]);
  }
  if (has("operand_copy_kernel")) std::memcpy(static_cast<void*>(&l.copy), a[0], sizeof l.copy);
  g_launches.push_back(l);
  return cudaSuccess;
}
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3 : 152;
  return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void** p, const void*) { *p = &g_err; return cudaSuccess; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *p = reinterpret_cast<void*>(&fake_encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t*) {
  *n = 76;
  return cudaSuccess;
}
const char* cudaGetErrorString(cudaError_t) { return "recorded"; }
cudaError_t cudaMemset2DAsync(void*, size_t, int, size_t, size_t, cudaStream_t) { return cudaSuccess; }
// what the host-buffer runtime uses; not called here
cudaError_t cudaEventCreateWithFlags(cudaEvent_t*, unsigned) { return cudaErrorUnknown; }
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaErrorUnknown; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaErrorUnknown; }
cudaError_t cudaEventSynchronize(cudaEvent_t) { return cudaErrorUnknown; }
cudaError_t cudaFreeAsync(void*, cudaStream_t) { return cudaErrorUnknown; }
cudaError_t cudaMallocFromPoolAsync(void**, size_t, cudaMemPool_t, cudaStream_t) { return cudaErrorUnknown; }
cudaError_t cudaMemPoolCreate(cudaMemPool_t*, const cudaMemPoolProps*) { return cudaErrorUnknown; }
cudaError_t cudaMemPoolSetAttribute(cudaMemPool_t, cudaMemPoolAttr, void*) { return cudaErrorUnknown; }
cudaError_t cudaMemcpy(void*, const void*, size_t, cudaMemcpyKind) { return cudaErrorUnknown; }
cudaError_t cudaMemcpy2DAsync(void*, size_t, const void*, size_t, size_t, size_t, cudaMemcpyKind,
                              cudaStream_t) {
  return cudaErrorUnknown;
}
cudaError_t cudaMemset(void*, int, size_t) { return cudaErrorUnknown; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaErrorUnknown; }
cudaError_t cudaStreamCreateWithFlags(cudaStream_t*, unsigned) { return cudaErrorUnknown; }
cudaError_t cudaStreamGetCaptureInfo(cudaStream_t, cudaStreamCaptureStatus*, unsigned long long*,
                                     cudaGraph_t*, const cudaGraphNode_t**, const cudaGraphEdgeData**,
                                     size_t*) {
  return cudaErrorUnknown;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaErrorUnknown; }
cudaError_t cudaStreamWaitEvent(cudaStream_t, cudaEvent_t, unsigned) { return cudaErrorUnknown; }
}

// ---- the checks

namespace {
constexpr int kSms = 152, kClusters = 76;
// addresses that are never dereferenced
char* const kWorkspace = reinterpret_cast<char*>(uintptr_t(1) << 44);
char* const kH = reinterpret_cast<char*>(uintptr_t(1) << 40);
char* const kW = reinterpret_cast<char*>(uintptr_t(1) << 41);
char* const kOut = reinterpret_cast<char*>(uintptr_t(1) << 42);

struct Case {
  int dtype, backward;
  int64_t T, V, D, pad_h, pad_w;
};

struct Span {
  const char* begin;
  const char* end;
  bool inside(const Span& o) const { return begin >= o.begin && end <= o.end && begin <= end; }
  bool apart(const Span& o) const { return end <= o.begin || o.end <= begin; }
};
Span span(const void* p, int64_t bytes) {
  const char* b = static_cast<const char*>(p);
  return {b, b + bytes};
}

long g_pieces, g_multi;

bool fail(const Case& c, const char* what) {
  std::printf("%s: dtype %d %s T %ld V %ld D %ld pads %ld %ld\n", what, c.dtype,
              c.backward ? "backward" : "forward", (long)c.T, (long)c.V, (long)c.D, (long)c.pad_h,
              (long)c.pad_w);
  return false;
}

// The slots that a launch's tiles take (whatever number of rows is in use).
int64_t slots_taken(const TrainArgs& a, bool all) {
  int64_t most = 0;
  const int sizes = a.n ? (a.n_is_k ? a.K : a.M) : 1;
  for (int i = 0; i <= (a.n ? 8 : 0); ++i) {
    const int n = static_cast<int>(static_cast<int64_t>(sizes) * i / 8);
    const int M = a.n && !a.n_is_k ? n : a.M;
    const int k = a.n && a.n_is_k ? std::min(n, a.split_k) : a.split_k;
    const int tiles = (M + 255) / 256 * ((a.N + a.width - 1) / a.width), blocks = (k + 63) / 64;
    const TilePlan p = plan_tiles(tiles, blocks, blocks * a.terms, kClusters);
    if (tiles == 0 || (!all && p.direct == p.tiles)) continue;
    most = std::max<int64_t>(
        most, slot_of(p, all, tiles - 1, p.direct == p.tiles ? 0 : p.splits - 1) + 1);
  }
  return most;
}

bool check(const Case& c) {
  const int64_t eb = c.dtype == GEMM14_DTYPE_F32_3XTF32 ? 4 : 2;
  const int64_t ldh = c.D + c.pad_h, ldw = c.D + c.pad_w;
  const size_t bytes = gemm14_linear_ce_workspace_bytes(c.dtype, c.backward, c.T, c.V, c.D, kH, ldh,
                                                        kW, ldw, kSms);
  if (bytes == 0) return fail(c, "no workspace");
  const Span ws = span(kWorkspace, static_cast<int64_t>(bytes));
  float* loss = reinterpret_cast<float*>(kOut);
  const int64_t* targets = reinterpret_cast<const int64_t*>(kOut + (1 << 30));
  float* g = reinterpret_cast<float*>(kOut + (1 << 29));
  g_launches.clear();
  const int st =
      c.backward
          ? gemm14_linear_ce_backward(c.dtype, c.T, c.V, c.D, kH, ldh, kW, ldw, targets, -100, loss,
                                      g, kOut + (int64_t(1) << 36), c.D, kOut + (int64_t(1) << 38),
                                      c.D, kWorkspace, bytes, nullptr)
          : gemm14_linear_ce_forward(c.dtype, c.T, c.V, c.D, kH, ldh, kW, ldw, targets, -100, loss,
                                     g, kWorkspace, bytes, nullptr);
  if (st != GEMM14_OK) return fail(c, gemm14_last_error_string());

  int64_t parts = 0, columns = 0, pieces = 0;
  const char* first = nullptr;
  for (const Launch& l : g_launches) {
    const TrainArgs& a = l.args;
    const bool few = l.few_width != 0;
    const auto mode = [&](int m) {
      const std::string tc = "train_tc_kernelILi" + std::to_string(m) + "E";
      const std::string fw = "train_few_kernelILi" + std::to_string(m) + "E";
      return l.name.find(tc) != std::string::npos || l.name.find(fw) != std::string::npos;
    };
    if (mode(kTrainStats)) {
      const int64_t w = few ? l.few_width : a.width, tiles = (a.N + w - 1) / w;
      const Span used = span(a.part, 2 * tiles * a.part_ld * 8);
      if (first == nullptr) first = used.begin;
      if (a.v0 != columns) return fail(c, "a piece of the vocabulary is left out");
      if (used.begin != first + parts * a.part_ld * 8) return fail(c, "statistics leave a gap");
      if (!used.inside(ws)) return fail(c, "statistics past the workspace");
      if (!used.apart(span(a.target_logit, c.T * 4))) return fail(c, "statistics over the targets' logits");
      if (a.part_count < 2 * tiles * a.part_ld) return fail(c, "statistics past their bounds check");
      if (!span(a.part, a.part_count * 8).inside(ws) ||
          !span(a.part, a.part_count * 8).apart(span(a.target_logit, c.T * 4)))
        return fail(c, "the bounds check of the statistics passes their buffer");
      if (!span(a.target_logit, c.T * 4).inside(ws)) return fail(c, "targets' logits past the workspace");
      parts += 2 * tiles;
      columns += a.N;
      ++pieces;
    } else if (mode(kTrainGrad)) {
      const int64_t dz_parts = a.elem == kElemBf16x3 ? 3 : few ? 2 : 1;
      const Span dz = span(a.out, ((dz_parts - 1) * a.out_part + a.out_rows * a.ld_out) * 2);
      if (a.v0 != columns) return fail(c, "a piece of the vocabulary is left out");
      if (!dz.inside(ws)) return fail(c, "dZ past the workspace");
      if (a.ld_out < a.N || a.out_rows < a.M) return fail(c, "dZ does not hold the piece");
      if (dz_parts > 1 && a.out_part < a.out_rows * a.ld_out) return fail(c, "dZ's parts overlap");
      columns += a.N;
      ++pieces;
    } else if (mode(kTrainSlots) || mode(kTrainOut)) {
      const Span slots = span(a.slots, a.slot_count * kSlotBytes);
      if (!slots.inside(ws)) return fail(c, "slots past the workspace");
      if (slots_taken(a, mode(kTrainSlots)) > a.slot_count) return fail(c, "too few slots");
      if (mode(kTrainSlots) && (a.add != 0) != (pieces > 1)) return fail(c, "slots added to wrongly");
    } else if (l.part) {
      if (l.part != first || l.parts != parts) return fail(c, "other statistics are merged than were left");
      if (!span(l.part, l.parts * l.part_ld * 8).inside(ws)) return fail(c, "merged statistics past the workspace");
    } else if (l.copy.rows) {
      const Span to = span(l.copy.dst, ((l.copy.parts - 1) * l.copy.part_stride +
                                        l.copy.rows * l.copy.ld_dst) * 2);
      if (!to.inside(ws)) return fail(c, "a copy past the workspace");
    }
  }
  if (columns != c.V) return fail(c, "columns are missing");
  g_pieces += pieces;
  g_multi += pieces > 1;
  (void)eb;
  return true;
}
}  // namespace

// Whether a forward call runs on the tensor cores.
bool on_tensor_cores(int dtype, int64_t T, int64_t V, int64_t D) {
  const size_t bytes =
      gemm14_linear_ce_workspace_bytes(dtype, 0, T, V, D, kH, D, kW, D, kSms);
  g_launches.clear();
  if (gemm14_linear_ce_forward(dtype, T, V, D, kH, D, kW, D,
                               reinterpret_cast<const int64_t*>(kOut + (1 << 30)), -100,
                               reinterpret_cast<float*>(kOut), reinterpret_cast<float*>(kOut + 4096),
                               kWorkspace, bytes, nullptr) != GEMM14_OK)
    return false;
  for (const Launch& l : g_launches)
    if (l.name.find("train_") != std::string::npos) return true;
  return false;
}

int main() {
  // fp32 rows: on the CUDA cores up to 32, in split arithmetic while that is the faster side
  for (int64_t T : {1, 8, 16, 17, 24, 32})
    for (int64_t D : {64, 1536, 1537, 4096, 12000}) {
      if (on_tensor_cores(GEMM14_DTYPE_F32, T, 5000, D)) return 3;
      if (on_tensor_cores(GEMM14_DTYPE_F32_3XTF32, T, 5000, D) != (T > 16 && D > 1536)) return 4;
    }
  long calls = 0, bad = 0;
  const auto run = [&](const Case& c) {
    ++calls;
    if (!check(c)) ++bad;
    return bad < 20;
  };
  // sizes of ordinary vocabularies and widths, split operands and copied ones
  for (int64_t V : {32000, 32768, 39168, 49152, 50257, 50304, 65536, 99584, 102400, 116740, 128000,
                    128256, 131072, 151936, 200064, 256000, 262144})
    for (int64_t D : {64, 513, 768, 1024, 1536, 1728, 2048, 2560, 4096, 5120, 8192})
      for (int64_t T : {1, 33, 64, 100, 128, 129, 300, 2048, 8192})
        for (int dtype : {GEMM14_DTYPE_BF16, GEMM14_DTYPE_F16, GEMM14_DTYPE_F32_3XTF32})
          for (int64_t pad : {0, 1}) {
            if (dtype == GEMM14_DTYPE_F32_3XTF32 && T <= 32) continue;  // the CUDA cores'
            for (int backward : {0, 1})
              if (!run({dtype, backward, T, V, D, 0, pad})) return 1;
          }
  // any size: a fixed sequence
  uint64_t state = 88172645463325252ull;
  const auto next = [&](int64_t low, int64_t high) {
    state ^= state << 13;
    state ^= state >> 7;
    state ^= state << 17;
    return low + static_cast<int64_t>(state % static_cast<uint64_t>(high - low + 1));
  };
  for (int i = 0; i < 20000; ++i) {
    const int dtype = i % 3 == 0 ? GEMM14_DTYPE_BF16 : i % 3 == 1 ? GEMM14_DTYPE_F16 : GEMM14_DTYPE_F32_3XTF32;
    const int64_t low = dtype == GEMM14_DTYPE_F32_3XTF32 ? 33 : 1;
    const int64_t T = i % 2 ? next(low, 128) : next(129, 1 << next(8, 16));
    if (!run({dtype, i % 5 == 0, T, next(1, 1 << next(8, 20)), next(1, 1 << next(4, 13)), next(0, 2),
              next(0, 2)}))
      return 1;
  }
  std::printf("%ld calls, %ld pieces, %ld calls of several, %ld bad\n", calls, g_pieces, g_multi, bad);
  return bad != 0 ? 1 : g_multi < 1000 ? 2 : 0;
}
