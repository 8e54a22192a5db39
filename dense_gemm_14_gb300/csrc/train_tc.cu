// train_tc.cu -- the training products on CTA pairs: tcgen05.mma.cta_group::2,
// 256 x 256 tiles of bf16 / fp16 operands (or of fp32 ones held as bf16 parts),
// fp32 accumulation, and epilogues that fold a tile away or turn it into the
// next product's operand instead of writing its sums (train_tc.h).
//
// Roles per CTA (320 threads, cluster of 2, persistent over tiles), as on the
// library's pair kernel: warp 0 loads this CTA's 128 rows of A and 128 columns
// of B by TMA into a ring of 6 stages, one lane of the leader's warp 1 issues
// the pair's MMAs into one of two 256-column accumulators, and warps 2..9
// drain the other: two warps for each quarter of the lanes, a thread holding
// one row's 128 columns, so that a row's maximum and sum need no exchange
// between threads.
//
// Measured (GB300): 4096 x 65536 x 4096 bf16 losses 1224 us, 1.80 PFLOP/s; a whole
// step of loss and gradients runs at 1.55 to 1.60, the power limit. About 9 us of
// each launch are its start and its last tile's epilogue.
//
// Long sums (kPromote): the accumulator is drained every CHUNK k-blocks (logits:
// LOGITS_CHUNK) into 128 fp32 registers a thread and starts again from zero while
// the MMAs go on in the other one.
//
// Every wait is bounded (ptx.cuh); a CTA that gives up raises its peer's abort
// flag, and both meet at a cluster barrier before TMEM is freed.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "api_internal.h"
#include "kernels.h"
#include "operand_copy.cuh"
#include "ptx.cuh"
#include "train_tc.h"

namespace gemm14 {
namespace {

using S = TrainShape;

constexpr float kLog2e = 1.44269504088896340736f;

struct TrainSmem {
  uint64_t full[S::STAGES];   // leader: both CTAs' bytes of a stage have landed
  uint64_t empty[S::STAGES];  // each CTA: the pair's MMAs finished reading the stage
  uint64_t acc_full[2];       // each CTA: accumulator b holds a finished sum
  uint64_t acc_empty[2];      // leader: all 16 epilogue warps drained accumulator b
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(TrainSmem) <= 256, "barrier block of the training kernel");

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The items of a launch, tiles in groups of 8 tile rows so that neighbouring
// clusters share A and B in L2.
struct Work {
  int M, N, K;        // in use
  int tiles_n, tiles_m, kblocks;
  TilePlan plan;

  __device__ Work(const TrainArgs& args, int clusters) {
    const int n = args.n ? *args.n : 0;
    N = args.N;
    M = args.n && !args.n_is_k ? min(n, args.M) : args.M;
    K = args.n && args.n_is_k ? min(n, args.K) : args.K;
    tiles_m = (M + S::BM - 1) / S::BM;
    tiles_n = (N + args.width - 1) / args.width;
    kblocks = (K + S::BK - 1) / S::BK;
    const int split_k = args.n && args.n_is_k ? min(n, args.split_k) : args.split_k;
    const int split_blocks = (split_k + S::BK - 1) / S::BK;
    plan = plan_tiles(tiles_m * tiles_n, split_blocks, split_blocks * args.terms, clusters);
  }
  __device__ int items() const {
    return plan.direct + (plan.tiles - plan.direct) * plan.splits;
  }
  __device__ void tile_at(int t, int& tm, int& tn) const {
    constexpr int kGroupM = 8;
    const int first = t / (kGroupM * tiles_n) * kGroupM;
    const int gm = min(tiles_m - first, kGroupM);
    const int r = t - first * tiles_n;
    tm = first + r % gm;
    tn = r / gm;
  }
  // Item i: tile t (tm, tn), k-blocks kb0 .. kb1 of it, range `split` of them.
  __device__ void get(int i, int& t, int& split, int& kb0, int& kb1) const {
    if (i < plan.direct) {
      t = i;
      split = 0;
      kb0 = 0;
      kb1 = kblocks;
    } else {
      const int tail = plan.tiles - plan.direct;
      split = (i - plan.direct) / tail;
      t = plan.direct + (i - plan.direct) - split * tail;
      kb0 = static_cast<int>(static_cast<int64_t>(kblocks) * split / plan.splits);
      kb1 = static_cast<int>(static_cast<int64_t>(kblocks) * (split + 1) / plan.splits);
    }
  }
};

// ---- epilogue pieces. `x` holds 32 consecutive columns (col0 ..) of this
// thread's row; `buf` is the warp's 32 x 128-byte staging block, its 16-byte
// pieces spread over the banks (row r's piece p at p ^ (r & 7)).

__device__ __forceinline__ uint32_t stage_at(uint32_t buf, int row, int piece) {
  return buf + static_cast<uint32_t>(row * 128 + (((piece ^ row) & 7) << 4));
}
__device__ __forceinline__ void stage_put(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 stage_get(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The bounds checks of `width` elements of the output at row r, column c.
__device__ __forceinline__ bool out_ok(const TrainArgs& a, int64_t r, int64_t c, int width) {
  return dev_check(c_span_ok(r * a.ld_out + c, a.ld_out, a.out_rows, a.out_cols, width), a.err);
}

// The warp's staged block, rows row0 .. +31, to global memory: 8 lanes write a
// row's 128 bytes. n_cols: elements of the row segment inside the matrix.
__device__ __forceinline__ void stage_out16(const TrainArgs& args, uint32_t buf, uint16_t* out,
                                            int row0, int rows, int64_t col0, int n_cols,
                                            int lane) {
  const int64_t ld = args.ld_out;
  if (!args.out_vec) {
    // rows at any address: a row at a time, lanes on neighbouring elements
#pragma unroll 4
    for (int r = 0; r < 32; ++r) {
      if (row0 + r >= rows) break;
      uint16_t* to = out + static_cast<int64_t>(row0 + r) * ld + col0;
#pragma unroll
      for (int c = lane; c < 64; c += 32) {
        if (c >= n_cols || !out_ok(args, row0 + r, col0 + c, 1)) continue;
        uint16_t v;
        asm volatile("ld.shared.u16 %0, [%1];"
                     : "=h"(v)
                     : "r"(stage_at(buf, r, c >> 3) + 2 * (c & 7))
                     : "memory");
        to[c] = v;
      }
    }
    return;
  }
  const int p = lane & 7;
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const int r = g * 4 + (lane >> 3);
    if (row0 + r >= rows || p * 8 >= n_cols) continue;
    const uint4 v = stage_get(stage_at(buf, r, p));
    uint16_t* to = out + static_cast<int64_t>(row0 + r) * ld + col0 + p * 8;
    if (!out_ok(args, row0 + r, col0 + p * 8, min(8, n_cols - p * 8))) continue;
    if ((p + 1) * 8 <= n_cols) {
      *reinterpret_cast<uint4*>(to) = v;
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (p * 8 + j < n_cols) to[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j % 2)));
    }
  }
}
// fp32, + beta times what is there: all 8 rows' old values are asked for before
// the first is used (one by one, a tile took 32 round trips to memory: 93 us for
// a 4096 x 4096 gradient of 16 rows, against 27 with them together).
__device__ __forceinline__ void stage_out32(const TrainArgs& args, uint32_t buf, int row0,
                                            int rows, int64_t col0, int n_cols, int lane) {
  float* out = static_cast<float*>(args.out);
  const int64_t ld = args.ld_out;
  const bool vec = args.out_vec != 0;
  const float beta = args.beta;
  const int p = lane & 7;
  const bool whole = vec && (p + 1) * 4 <= n_cols;
  float4 old[8];
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const int r = row0 + g * 4 + (lane >> 3);
    old[g] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (beta == 0.0f || r >= rows || p * 4 >= n_cols) continue;
    if (!out_ok(args, r, col0 + p * 4, min(4, n_cols - p * 4))) continue;
    const float* from = out + static_cast<int64_t>(r) * ld + col0 + p * 4;
    if (whole) {
      old[g] = *reinterpret_cast<const float4*>(from);
    } else {
      float* o = &old[g].x;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (p * 4 + j < n_cols) o[j] = from[j];
    }
  }
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const int r = g * 4 + (lane >> 3);
    if (row0 + r >= rows || p * 4 >= n_cols) continue;
    const uint4 u = stage_get(stage_at(buf, r, p));
    float4 v = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z),
                           __uint_as_float(u.w));
    if (beta != 0.0f)
      v = make_float4(fmaf(beta, old[g].x, v.x), fmaf(beta, old[g].y, v.y),
                      fmaf(beta, old[g].z, v.z), fmaf(beta, old[g].w, v.w));
    if (!out_ok(args, row0 + r, col0 + p * 4, min(4, n_cols - p * 4))) continue;
    float* to = out + static_cast<int64_t>(row0 + r) * ld + col0 + p * 4;
    if (whole) {
      *reinterpret_cast<float4*>(to) = v;
    } else {
      const float* e = &v.x;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (p * 4 + j < n_cols) to[j] = e[j];
    }
  }
}

// Row state of the epilogues that work on logits.
struct RowData {
  int y;              // target's column relative to the tile half, or out of [0, 128)
  float lse, coef;    // gradient
  float m, l, zy;     // statistics
};

// kDzParts: 16-bit parts of a dZ of 16-bit operands (kTrainGrad).
template <int kMode, int kChunks = 4, int kDzParts = 1>
struct Epilogue {
  const TrainArgs& args;
  int M, N, lane, row0, row, half, rank;
  int64_t slot;       // of this item, < 0: the tile is written to its place
  int col_half;       // first column of this thread's kChunks x 32
  uint32_t buf;
  RowData d;
  float factor;

  __device__ void begin() {
    if (kMode == kTrainStats || kMode == kTrainGrad) {
      d.y = -1;
      d.lse = 0.0f;
      d.coef = 0.0f;
      if (row < M) {
        if (args.target) {
          d.y = args.target[row];
        } else {
          const int64_t y = args.target64[row];
          d.y = y >= 0 && y < INT_MAX ? static_cast<int>(y) : -1;
        }
        d.y = d.y < 0 ? -1 : d.y - args.v0 - col_half;
        if (kMode == kTrainGrad) {
          d.lse = args.lse[row];
          d.coef = args.coef[row];
        }
      }
      d.m = -INFINITY;
      d.l = 0.0f;
      d.zy = 0.0f;
    }
    if (kMode == kTrainOut) {
      factor = args.alpha * (args.scale ? *args.scale : 1.0f);
      // the old values are asked for before the sums are ready
      if (args.beta != 0.0f && slot < 0 && row < M) {
        const float* from = static_cast<const float*>(args.out) +
                            static_cast<int64_t>(row) * args.ld_out + col_half;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          if (col_half + 32 * c < N)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(from + 32 * c));
      }
    }
  }

  // Columns 32 c .. of the half, in registers.
  __device__ void chunk(int c, float (&x)[32]) {
    const int col0 = col_half + 32 * c;
    if (kMode == kTrainStats) {
      if (col0 + 32 > N) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (col0 + j >= N) x[j] = -INFINITY;
      }
      float m = d.m;
#pragma unroll
      for (int j = 0; j < 32; ++j) m = fmaxf(m, x[j]);
      // nothing above -inf so far: any finite base gives the sum's zeros
      const float base = m == -INFINITY ? 0.0f : m;
      float l = d.l * exp2_approx((d.m - base) * kLog2e);
#pragma unroll
      for (int j = 0; j < 32; ++j) l += exp2_approx((x[j] - base) * kLog2e);
      d.m = m;
      d.l = l;
      const int y = d.y - 32 * c;
      if (y >= 0 && y < 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j == y) d.zy = x[j];
      }
    } else if (kMode == kTrainGrad) {
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] = exp2_approx((x[j] - d.lse) * kLog2e);
      const int y = d.y - 32 * c;
      if (y >= 0 && y < 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j == y) x[j] -= 1.0f;
      }
      // a row past the last in use, or one of coefficient 0, is exactly 0
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] = d.coef == 0.0f ? 0.0f : x[j] * d.coef;
      store16(c, x);
    } else if (kMode == kTrainSlots || slot >= 0) {
      const int64_t at = slot_index(slot, rank, half, c, 0, row - (row0 & ~127));
      if (!dev_check(slot_span_ok(at, slot, kSlotBytes / 16, args.slot_count, 1) &&
                         slot_span_ok(at + 128 * 7, slot, kSlotBytes / 16, args.slot_count, 1),
                     args.err))
        return;
      float4* s = args.slots + at;
      float4 old[8];
#pragma unroll
      for (int v = 0; v < 8; ++v)
        old[v] = kMode == kTrainSlots && args.add ? __ldcg(s + 128 * v)
                                                  : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int v = 0; v < 8; ++v)
        __stcg(s + 128 * v, make_float4(old[v].x + x[4 * v], old[v].y + x[4 * v + 1],
                                        old[v].z + x[4 * v + 2], old[v].w + x[4 * v + 3]));
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] *= factor;
      if (args.elem == kElemF32) {
        __syncwarp();
#pragma unroll
        for (int p = 0; p < 8; ++p)
          stage_put(stage_at(buf, lane, p),
                    make_uint4(__float_as_uint(x[4 * p]), __float_as_uint(x[4 * p + 1]),
                               __float_as_uint(x[4 * p + 2]), __float_as_uint(x[4 * p + 3])));
        __syncwarp();
        stage_out32(args, buf, row0, M, col0, min(32, N - col0), lane);
      } else {
        store16(c, x);
      }
    }
  }

  // 16-bit output: two chunks of 32 columns share a staged block of 64.
  __device__ void store16(int c, float (&x)[32]) {
    const int parts = args.elem == kElemBf16x3 ? 3 : kDzParts;
    // kTrainGrad writes whole tile rows (zeros past the rows in use): its
    // buffer has them
    const int rows = kMode == kTrainGrad ? INT_MAX : M;
    if (parts == 1) {
      if ((c & 1) == 0) __syncwarp();
      const int p0 = (c & 1) * 4;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        uint4 v;
        if (args.elem == kElemF16)
          v = make_uint4(pack_f16(x[8 * p], x[8 * p + 1]), pack_f16(x[8 * p + 2], x[8 * p + 3]),
                         pack_f16(x[8 * p + 4], x[8 * p + 5]), pack_f16(x[8 * p + 6], x[8 * p + 7]));
        else
          v = make_uint4(pack_bf16(x[8 * p], x[8 * p + 1]), pack_bf16(x[8 * p + 2], x[8 * p + 3]),
                         pack_bf16(x[8 * p + 4], x[8 * p + 5]),
                         pack_bf16(x[8 * p + 6], x[8 * p + 7]));
        stage_put(stage_at(buf, lane, p0 + p), v);
      }
      if ((c & 1) == 0 && c + 1 < kChunks) return;
      __syncwarp();
      const int col0 = col_half + 64 * (c >> 1);
      stage_out16(args, buf, static_cast<uint16_t*>(args.out), row0, rows, col0,
                  min(c & 1 ? 64 : 32, N - col0), lane);
      return;
    }
    // parts of each value: the nearest, then the nearest to what is left
    const int col0 = col_half + 32 * c;
    for (int part = 0; part < parts; ++part) {
      __syncwarp();
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float& a = x[8 * p + 2 * k];
          float& b = x[8 * p + 2 * k + 1];
          if (kDzParts == 2 && args.elem == kElemF16) {
            w[k] = pack_f16(a, b);
            a -= __half2float(__ushort_as_half(static_cast<unsigned short>(w[k])));
            b -= __half2float(__ushort_as_half(static_cast<unsigned short>(w[k] >> 16)));
          } else {
            w[k] = pack_bf16(a, b);
            a -= __uint_as_float(w[k] << 16);
            b -= __uint_as_float(w[k] & 0xffff0000u);
          }
        }
        stage_put(stage_at(buf, lane, p), make_uint4(w[0], w[1], w[2], w[3]));
      }
      __syncwarp();
      stage_out16(args, buf, static_cast<uint16_t*>(args.out) + part * args.out_part, row0, rows,
                  col0, min(32, N - col0), lane);
    }
  }

  __device__ void end(int tn) {
    if (kMode == kTrainStats && row < M) {
      const int64_t at = (static_cast<int64_t>(tn) * 2 + half) * args.part_ld + row;
      if (!dev_check(index_ok(at, args.part_count), args.err)) return;
      args.part[at] = make_float2(d.m, d.l);
      if (d.y >= 0 && d.y < 32 * kChunks && col_half + d.y < N) args.target_logit[row] = d.zy;
    }
  }
};

// kWidth: columns of a tile, args.width.
template <int kMode, bool kPromote, int kWidth>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(S::THREADS, 1)
    train_tc_kernel(const __grid_constant__ TrainMaps maps, const TrainArgs args) {
  constexpr int kChunk =
      kMode == kTrainStats || kMode == kTrainGrad ? S::LOGITS_CHUNK : S::CHUNK;
  constexpr int kHalf = kWidth / 2;  // a CTA's columns of B, and a warp's of D
  constexpr int kChunks = kHalf / 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = align1024(smem_raw);
  uint8_t* out_stage = tiles + S::STAGES * S::STAGE_BYTES;
  TrainSmem& sm = *reinterpret_cast<TrainSmem*>(out_stage + S::EPI_WARPS * S::OUT_BUF_BYTES);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cid = static_cast<int>(cluster_id_x());
  const int ncl = static_cast<int>(cluster_count_x());
  const WaitCtx wc{args.err, &sm.abort_flag, args.wait_limit_ns,
                   mapa_shared(smem_u32(&sm.abort_flag), rank ^ 1u)};
  uint32_t prod_it = 0;
  bool mma_issued = false;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.acc_full[b], 1);
      mbar_init(&sm.acc_empty[b], 2 * S::EPI_WARPS);
    }
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.a[0]);
    tma_prefetch_desc(&maps.b[0]);
  }
  cluster_sync();
  if (warp == 1) {
    tmem_alloc_pair(&sm.tmem_base, S::TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t tmem_base = sm.tmem_base;

  // Both CTAs of a pair, and all their roles, work out the same plan.
  const Work work(args, ncl);
  const int M = work.M;
  const int items = work.items();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      bool ok = true;
      for (int i = cid; i < items && ok; i += ncl) {
        int t, split, tm, tn, kb0, kb1;
        work.get(i, t, split, kb0, kb1);
        work.tile_at(t, tm, tn);
        const int m0 = tm * S::BM + static_cast<int>(rank) * 128;
        const int n0 = tn * kWidth + static_cast<int>(rank) * kHalf;
        const int step = kPromote ? kChunk : kb1 - kb0;
        for (int c0 = kb0; c0 < kb1 && ok; c0 += step) {
          const int c1 = min(c0 + step, kb1);
          for (int term = 0; term < args.terms && ok; ++term) {
            const uint32_t code = args.term_code >> (4 * term);
            const CUtensorMap* ma = &maps.a[code & 3];
            const CUtensorMap* mb = &maps.b[(code >> 2) & 3];
            for (int kb = c0; kb < c1; ++kb, ++prod_it) {
              const uint32_t s = prod_it % S::STAGES, ph = (prod_it / S::STAGES) & 1;
              if (!mbar_wait(&sm.empty[s], ph ^ 1, wc)) { ok = false; break; }
              // Failure-detection tests: the first stage is never loaded.
              if (args.fault == kFaultSkipFirstStage && prod_it == 0) continue;
              uint8_t* a_st = tiles + s * S::STAGE_BYTES;
              uint8_t* b_st = a_st + S::A_BYTES;
              const uint32_t full_leader = mapa_shared(smem_u32(&sm.full[s]), 0);
              if (leader) mbar_arrive_expect_tx(&sm.full[s], 2 * (S::A_BYTES + kHalf * 128));
              if (!args.a_mn) {
                tma_load_2d_pair(a_st, ma, kb * S::BK, m0, full_leader);
              } else {
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  tma_load_2d_pair(a_st + c * (64 * S::BK * 2), ma, m0 + c * 64, kb * S::BK,
                                   full_leader);
              }
              if (!args.b_mn) {
                tma_load_2d_pair(b_st, mb, kb * S::BK, n0, full_leader);
              } else {
                #pragma unroll
                for (int c = 0; 64 * c < kHalf; ++c)
                  tma_load_2d_pair(b_st + c * (64 * S::BK * 2), mb, n0 + c * 64, kb * S::BK,
                                   full_leader);
              }
            }
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader)
    if (leader && lane == 0) {
      const OperandDesc a_op = operand_desc(args.a_mn == 0);
      const OperandDesc b_op = operand_desc(args.b_mn == 0);
      bool ok = true;
      uint32_t it = 0, unit = 0;
      for (int i = cid; i < items && ok; i += ncl) {
        int t, split, kb0, kb1;
        work.get(i, t, split, kb0, kb1);
        const int step = kPromote ? kChunk : kb1 - kb0;
        for (int c0 = kb0; c0 < kb1; c0 += step, ++unit) {
          const int blocks = (min(c0 + step, kb1) - c0) * args.terms;
          const int b = unit & 1;
          const uint32_t aph = (unit >> 1) & 1;
          if (!mbar_wait_cluster(&sm.acc_empty[b], aph ^ 1, wc)) { ok = false; break; }
          tc_fence_after_sync();
          const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(b * S::BN);
          for (int k = 0; k < blocks; ++k, ++it) {
            const uint32_t s = it % S::STAGES, ph = (it / S::STAGES) & 1;
            if (!mbar_wait(&sm.full[s], ph, wc)) { ok = false; break; }
            tc_fence_after_sync();
            const uint32_t a_addr = smem_u32(tiles + s * S::STAGE_BYTES);
            const uint32_t b_addr = a_addr + S::A_BYTES;
#pragma unroll
            for (int kk = 0; kk < S::BK / 16; ++kk) {
              const uint64_t a_desc = smem_desc_sw128(a_addr + kk * a_op.step, a_op.lbo, 1024);
              const uint64_t b_desc = smem_desc_sw128(b_addr + kk * b_op.step, b_op.lbo, 1024);
              tc_mma_f16_pair(d_tmem, a_desc, b_desc, args.idesc, k != 0 || kk != 0);
            }
            mma_issued = true;
            tc_commit_pair_multicast(&sm.empty[s], 0x3);
          }
          if (!ok) break;
          tc_commit_pair_multicast(&sm.acc_full[b], 0x3);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;             // TMEM lane quarter this warp may access
    const int half = (warp - 2) >> 2;   // its 128 columns of the tile
    const uint32_t acc_empty0 = mapa_shared(smem_u32(&sm.acc_empty[0]), 0);
    const uint32_t acc_empty1 = mapa_shared(smem_u32(&sm.acc_empty[1]), 0);
    const uint32_t buf = smem_u32(out_stage + (warp - 2) * S::OUT_BUF_BYTES);
    uint32_t unit = 0;
    bool ok = true;
    for (int i = cid; i < items && ok; i += ncl) {
      int t, split, tm, tn, kb0, kb1;
      work.get(i, t, split, kb0, kb1);
      work.tile_at(t, tm, tn);
      const int64_t slot = kMode == kTrainSlots || t >= work.plan.direct
                               ? slot_of(work.plan, kMode == kTrainSlots, t, split) : -1;
      const int row0 = tm * S::BM + static_cast<int>(rank) * 128 + q * 32;
      Epilogue<kMode, kChunks> e{args, M, args.N, lane, row0, row0 + lane, half,
                                 static_cast<int>(rank), slot, tn * kWidth + half * kHalf, buf,
                                 {}, 1.0f};
      e.begin();
      const int step = kPromote ? kChunk : kb1 - kb0;
      float acc[kPromote ? 128 : 1];
      if (kPromote) {
#pragma unroll
        for (int j = 0; j < (kPromote ? 128 : 1); ++j) acc[j] = 0.0f;
      }
      for (int c0 = kb0; c0 < kb1; c0 += step, ++unit) {
        const int b = unit & 1;
        const uint32_t aph = (unit >> 1) & 1;
        int got = 1;
        if (lane == 0) got = mbar_wait(&sm.acc_full[b], aph, wc) ? 1 : 0;
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) { ok = false; break; }
        tc_fence_after_sync();
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                               static_cast<uint32_t>(b * S::BN + half * kHalf);
        if (kPromote) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(t_row + c * 32, r);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[kPromote ? 32 * c + j : 0] += __uint_as_float(r[j]);
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < kChunks; ++c) {
            uint32_t r[32];
            float x[32];
            tmem_ld_32x32b_x32(t_row + c * 32, r);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(r[j]);
            e.chunk(c, x);
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_peer(b ? acc_empty1 : acc_empty0);
      }
      if (!ok) break;
      if (kPromote) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          float x[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = acc[kPromote ? 32 * c + j : 0];
          e.chunk(c, x);
        }
      } else if (kb0 == kb1) {
        // no products at all (no rows in use): sums of zero
#pragma unroll 1
        for (int c = 0; c < kChunks; ++c) {
          float x[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = 0.0f;
          e.chunk(c, x);
        }
      }
      e.end(tn);
    }
  }

  // Teardown. On abort, the leader lets its issued MMAs and both CTAs' loads
  // (counted on its full barriers) finish, bounded, before the pair meets.
  __syncthreads();
  if (sm.abort_flag && leader) {
    if (warp == 1 && lane == 0 && mma_issued) {
      tc_commit_pair_multicast(&sm.drain, 0x1);
      mbar_wait_timed(&sm.drain, 0, 100000000ull);
    }
    if (warp == 0 && lane == 0) {
      const uint32_t first = prod_it > S::STAGES ? prod_it - S::STAGES : 0;
      for (uint32_t j = first; j < prod_it; ++j)
        if (!(args.fault == kFaultSkipFirstStage && j == 0))
          mbar_wait_timed(&sm.full[j % S::STAGES], (j / S::STAGES) & 1, 100000000ull);
    }
  }
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, S::TMEM_COLS);
  }
}

// The logits of few rows (up to 128): the call is one read of B, and the
// kernel's business is to keep it flowing. One SM a tile (M = 128, N = width): a
// k-block of 256 rows of B is 512 cycles of MMAs for 32 KB, 18 TB/s over 152 SMs,
// where the pair's M = 256 spends them on 16 KB an SM. The rows of A in use alone
// are loaded; the MMA reads 128 rows' bytes, the others being whatever the
// ring holds there, and the rows of D they make are not looked at. Tiles are as
// wide as spreads the columns evenly (32768 columns: 147 tiles of 224 on 152
// SMs, where 128 of 256 on 76 pairs are 1.7 waves). With B on the MMA's M side
// (N = 16 for one row) a k-block took 0.33 us whatever its height, N that small
// leaving the tensor cores waiting: 268 MB of weights took 62 us.
// Split operands: a stage holds a k-block of one part of B and of the parts of A
// that it meets (part p: the first 3 - p), so that B's parts are read once each.
struct FewSmem {
  uint64_t full[FewShape::MAX_STAGES];
  uint64_t empty[FewShape::MAX_STAGES];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(FewSmem) <= 512, "barrier block of the few-rows kernel");

struct FewTiles {
  int width, rows, stages, quarters;  // quarters: of the 128 rows that are looked at
};

template <int kMode, int kParts>
__global__ void __launch_bounds__(FewShape::THREADS, 1)
    train_few_kernel(const __grid_constant__ TrainMaps maps, const TrainArgs args,
                     const FewTiles few) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = align1024(smem_raw);
  uint8_t* out_stage = ring + FewShape::RING_BYTES;
  FewSmem& sm = *reinterpret_cast<FewSmem*>(out_stage + S::EPI_WARPS * S::OUT_BUF_BYTES);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t b_bytes = static_cast<uint32_t>(few.width) * 128u;
  const uint32_t a_bytes = static_cast<uint32_t>(few.rows) * 128u;
  const uint32_t stage_bytes = b_bytes + kParts * a_bytes;
  const uint32_t stages = static_cast<uint32_t>(few.stages);
  const int tiles = (args.N + few.width - 1) / few.width;
  const int kblocks = (args.K + S::BK - 1) / S::BK;
  const WaitCtx wc{args.err, &sm.abort_flag, args.wait_limit_ns, 0};
  uint32_t prod_it = 0;
  bool mma_issued = false;

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < stages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.acc_full[b], 1);
      mbar_init(&sm.acc_empty[b], 2 * few.quarters);
    }
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.a[0]);
    tma_prefetch_desc(&maps.b[0]);
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, S::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t tmem_base = sm.tmem_base;
  const int M = args.n ? min(*args.n, args.M) : args.M;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      bool ok = true;
      uint32_t s = 0, ph = 0;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        for (int k0 = 0; k0 < kblocks && ok; k0 += FewShape::CHUNK) {
          const int k1 = min(k0 + FewShape::CHUNK, kblocks);
          for (int p = kParts - 1; p >= 0 && ok; --p) {
            for (int kb = k0; kb < k1; ++kb, ++prod_it) {
              if (!mbar_wait(&sm.empty[s], ph ^ 1, wc)) { ok = false; break; }
              // Failure-detection tests: the first stage is never loaded.
              if (!(args.fault == kFaultSkipFirstStage && prod_it == 0)) {
                uint8_t* st = ring + s * stage_bytes;
                mbar_arrive_expect_tx(&sm.full[s], b_bytes + (kParts - p) * a_bytes);
                tma_load_2d(st, &maps.b[p], kb * S::BK, t * few.width, &sm.full[s]);
                for (int a = 0; a < kParts - p; ++a)
                  tma_load_2d(st + b_bytes + a * a_bytes, &maps.a[a], kb * S::BK, 0, &sm.full[s]);
              }
              if (++s == stages) {
                s = 0;
                ph ^= 1;
              }
            }
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      bool ok = true;
      uint32_t s = 0, ph = 0, unit = 0;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        for (int k0 = 0; k0 < kblocks; k0 += FewShape::CHUNK, ++unit) {
          const int k1 = min(k0 + FewShape::CHUNK, kblocks);
          const int b = unit & 1;
          if (!mbar_wait(&sm.acc_empty[b], ((unit >> 1) & 1) ^ 1, wc)) { ok = false; break; }
          tc_fence_after_sync();
          bool add = false;
          for (int p = kParts - 1; p >= 0 && ok; --p) {
            for (int kb = k0; kb < k1; ++kb) {
              if (!mbar_wait(&sm.full[s], ph, wc)) { ok = false; break; }
              tc_fence_after_sync();
              const uint32_t b_addr = smem_u32(ring + s * stage_bytes);
              for (int a = kParts - 1 - p; a >= 0; --a) {
#pragma unroll
                for (int kk = 0; kk < S::BK / 16; ++kk) {
                  tc_mma_f16(tmem_base + static_cast<uint32_t>(b * S::BN),
                             smem_desc_sw128(b_addr + b_bytes + a * a_bytes + kk * 32, 16, 1024),
                             smem_desc_sw128(b_addr + kk * 32, 16, 1024), args.idesc, add);
                  add = true;
                }
              }
              mma_issued = true;
              tc_commit(&sm.empty[s]);
              if (++s == stages) {
                s = 0;
                ph ^= 1;
              }
            }
          }
          if (!ok) break;
          tc_commit(&sm.acc_full[b]);
        }
      }
    }
  } else if ((warp & 3) < few.quarters) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int half = (warp - 2) >> 2;
    const uint32_t buf = smem_u32(out_stage + (warp - 2) * S::OUT_BUF_BYTES);
    uint32_t unit = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const int limit = min(args.N, (t + 1) * few.width);
      Epilogue<kMode, 4, kMode == kTrainGrad && kParts == 1 ? 2 : 1> e{
          args, M, limit, lane, q * 32, q * 32 + lane, half, 0, -1, t * few.width + half * 128,
          buf, {}, 1.0f};
      e.begin();
      float acc[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) acc[j] = 0.0f;
      for (int k0 = 0; k0 < kblocks; k0 += FewShape::CHUNK, ++unit) {
        const int b = unit & 1;
        int got = 1;
        if (lane == 0) got = mbar_wait(&sm.acc_full[b], (unit >> 1) & 1, wc) ? 1 : 0;
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) { ok = false; break; }
        tc_fence_after_sync();
        const uint32_t from = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                              static_cast<uint32_t>(b * S::BN + half * 128);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(from + c * 32, r);
          tc_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[32 * c + j] += __uint_as_float(r[j]);
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.acc_empty[b]);
      }
      if (!ok) break;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float x[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = acc[32 * c + j];
        e.chunk(c, x);
      }
      e.end(t);
    }
  }

  // Teardown: on abort, what was issued finishes (bounded) before TMEM is freed.
  __syncthreads();
  if (sm.abort_flag) {
    if (warp == 1 && lane == 0 && mma_issued) {
      tc_commit(&sm.drain);
      mbar_wait_timed(&sm.drain, 0, 100000000ull);
    }
    if (warp == 0 && lane == 0) {
      const uint32_t first = prod_it > stages ? prod_it - stages : 0;
      for (uint32_t j = first; j < prod_it; ++j)
        if (!(args.fault == kFaultSkipFirstStage && j == 0))
          mbar_wait_timed(&sm.full[j % stages], (j / stages) & 1, 100000000ull);
    }
    __syncthreads();
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, S::TMEM_COLS);
  }
}

// 32 rows x 32 columns of a tile at a time: slots are read along rows (512 bytes
// a warp), the output is written along columns, through shared memory. The
// blocks go round the tiles that have slots (few, or none, after a launch whose
// last wave was full: a block for each that might be took 13 us to find so).
__global__ void __launch_bounds__(256)
    slots_out_kernel(const TrainArgs args, const SlotsOut s, int clusters) {
  __shared__ float tile[32][36];
  grid_dependency_wait();
  grid_launch_dependents();
  const Work work(args, clusters);
  const int first = s.all ? 0 : work.plan.direct;
  const int64_t pieces = static_cast<int64_t>(work.plan.tiles - first) * 64;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = threadIdx.x >> 3, c4 = (threadIdx.x & 7) * 4;
  const float k = pieces ? s.alpha * (s.scale ? *s.scale : 1.0f) : 0.0f;
  for (int64_t i = blockIdx.x; i < pieces; i += gridDim.x) {
    const int t = first + static_cast<int>(i >> 6), part = static_cast<int>(i & 63);
    int tm, tn;
    work.tile_at(t, tm, tn);
    const int rank = part >> 5, q0 = ((part >> 3) & 3) * 32, half = (part >> 2) & 1, c = part & 3;
    const int row0 = tm * S::BM + rank * 128 + q0;
    const int col0 = tn * args.width + half * (args.width / 2) + c * 32;
    if (64 * c >= args.width || row0 >= work.M || col0 >= work.N) continue;
    const int ranges = t < work.plan.direct ? 1 : work.plan.splits;
    const float4* from = args.slots + slot_index(slot_of(work.plan, s.all, t, 0), rank, half, c,
                                                 warp, q0 + lane);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int side = 0; side <= s.fold; ++side, from += slot_index(0, 1, 0, 0, 0, 0)) {
#pragma unroll 8
      for (int p = 0; p < ranges; ++p) {
        const float4 o = __ldcg(from + p * (kSlotBytes / 16));
        v.x += o.x;
        v.y += o.y;
        v.z += o.z;
        v.w += o.w;
      }
    }
    __syncthreads();
    *reinterpret_cast<float4*>(&tile[lane][4 * warp]) = v;
    __syncthreads();
    if (row0 + r >= work.M) continue;
    const int64_t row = s.rows ? s.rows[row0 + r] : row0 + r;
    const int col = col0 + c4, cols = min(4, work.N - col);
    const int64_t at = row * s.ld + col;
    if (cols <= 0 ||
        !dev_check(c_span_ok(at, s.ld, s.out_rows, work.N, cols), args.err))
      continue;
    if (s.elem == kElemF32) {
      float* o = static_cast<float*>(s.out) + at;
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = s.beta != 0.0f && j < cols ? o[j] : 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < cols) o[j] = fmaf(s.beta, x[j], tile[r][c4 + j] * k);
    } else {
      uint16_t* o = static_cast<uint16_t*>(s.out) + at;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < cols) {
          const float x = tile[r][c4 + j] * k;
          o[j] = s.elem == kElemF16 ? __half_as_ushort(__float2half_rn(x))
                                    : __bfloat16_as_ushort(__float2bfloat16_rn(x));
        }
    }
  }
}

__global__ void __launch_bounds__(256) operand_copy_kernel(const OperandCopy job) {
  grid_dependency_wait();
  grid_launch_dependents();
  operand_copy(job, blockIdx.x, gridDim.x);
}

using TrainKernel = void (*)(const TrainMaps, const TrainArgs);

TrainKernel kernel_of(int mode, bool promote, int width) {
  switch (mode) {
    case kTrainStats:
      return promote ? train_tc_kernel<kTrainStats, true, 256>
                     : train_tc_kernel<kTrainStats, false, 256>;
    case kTrainGrad:
      return promote ? train_tc_kernel<kTrainGrad, true, 256>
                     : train_tc_kernel<kTrainGrad, false, 256>;
    case kTrainSlots:
      return promote ? train_tc_kernel<kTrainSlots, true, 256>
                     : train_tc_kernel<kTrainSlots, false, 256>;
    default:  // (sums short enough for half the width are never promoted)
      return width == 128 ? train_tc_kernel<kTrainOut, false, 128>
             : promote    ? train_tc_kernel<kTrainOut, true, 256>
                          : train_tc_kernel<kTrainOut, false, 256>;
  }
}

}  // namespace

int train_max_clusters() {
  static DeviceOnce cached;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= DeviceOnce::kDevices) return 0;
  const int n = cached.get(
      dev,
      [] {
        int least = INT_MAX;
        for (int i = 0; i < 9; ++i) {
            const TrainKernel k = i < 8 ? kernel_of(i / 2, i % 2 != 0, 256)
                                        : kernel_of(kTrainOut, false, 128);
            if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     S::SMEM_BYTES) != cudaSuccess)
              return -1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(2, 1, 1);
            cfg.blockDim = dim3(S::THREADS, 1, 1);
            cfg.dynamicSmemBytes = S::SMEM_BYTES;
            int c = 0;
            if (cudaOccupancyMaxActiveClusters(&c, k, &cfg) != cudaSuccess) c = 0;
            least = c < least ? c : least;
          }
        return least;
      },
      [](int v) { return v >= 0; });
  return n > 0 ? n : 0;
}

int train_operands(bool bf16, const TrainOperand& A, bool a_mn, const TrainOperand& B, bool b_mn,
                   TrainMaps* maps, TrainArgs* args, int a_rows, int b_rows) {
  const auto encode = [&](const TrainOperand& x, bool mn, int box_rows, CUtensorMap* m) {
    for (int p = 0; p < 3; ++p) {
      if (p >= x.parts) {
        m[p] = m[0];
        continue;
      }
      const void* base = static_cast<const char*>(x.base) + 2 * p * x.part_stride;
      const int st = map_16bit(&m[p], bf16, base, x.rows, x.cols, x.ld, mn ? 64 : box_rows);
      if (st != 0) return st;
    }
    return 0;
  };
  int st = encode(A, a_mn, a_rows ? a_rows : 128, maps->a);
  if (st == 0) st = encode(B, b_mn, b_rows ? b_rows : args->width / 2, maps->b);
  if (st != 0) return st;
  // Terms of split operands, small ones first: of 3 x 3 parts the six whose
  // product is above 2^-24 of the whole, or A's two or three parts against one B.
  args->terms = B.parts == 3 ? 6 : A.parts;
  args->term_code = B.parts == 3 ? 0x041582u : A.parts == 3 ? 0x012u : A.parts == 2 ? 0x01u : 0u;
  args->a_mn = a_mn;
  args->b_mn = b_mn;
  args->idesc = idesc_f16_f32acc(bf16, S::BM, args->width, a_mn, b_mn);
  return 0;
}

int few_width(int64_t N, int sms) {
  int best = 256;
  int64_t best_cols = INT64_MAX;  // of the SM with the most
  for (int w = 256; w >= 128; w -= 16) {
    const int64_t cols = ((N + w - 1) / w + sms - 1) / sms * w;
    if (cols < best_cols) {
      best_cols = cols;
      best = w;
    }
  }
  return best;
}

int few_rows(int64_t M) { return M <= 16 ? 16 : static_cast<int>((M + 31) / 32 * 32); }

cudaError_t launch_train_few(int mode, const TrainMaps& maps, TrainArgs args, bool bf16, int width,
                             int sm_count, cudaStream_t stream) {
  FewTiles few{};
  few.width = width;
  few.rows = few_rows(args.M);
  const int parts = args.terms == 6 ? 3 : 1;
  const int stage = (few.width + parts * few.rows) * 128;
  // the last stage's MMAs read 128 rows' bytes of A, however many were loaded
  few.stages = (FewShape::RING_BYTES - (FewShape::A_BYTES - few.rows * 128)) / stage;
  if (few.stages > FewShape::MAX_STAGES) few.stages = FewShape::MAX_STAGES;
  // dZ is read in k-blocks of 64 rows by the product over them
  few.quarters = mode == kTrainGrad ? (args.M + 63) / 64 * 2 : (args.M + 31) / 32;
  args.idesc = idesc_f16_f32acc(bf16, 128, width, false, false);
  const bool grad = mode == kTrainGrad;
  const auto kernel = parts == 3 ? (grad ? train_few_kernel<kTrainGrad, 3> : train_few_kernel<kTrainStats, 3>)
                                 : (grad ? train_few_kernel<kTrainGrad, 1> : train_few_kernel<kTrainStats, 1>);
  static DeviceOnce once[2][2];
  const cudaError_t e = set_smem_once(once[grad][parts == 3], kernel, FewShape::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const int tiles = (args.N + width - 1) / width;
  return launch_kernel(kernel, dim3(tiles < sm_count ? tiles : sm_count), dim3(FewShape::THREADS),
                       FewShape::SMEM_BYTES, stream, maps, args, few);
}

bool may_split(const TrainArgs& args, int clusters) {
  const int tiles = ((args.M + S::BM - 1) / S::BM) * ((args.N + args.width - 1) / args.width);
  const int blocks = (args.split_k + S::BK - 1) / S::BK;
  // with the rows in use known on the device only, any smaller plan may be the one
  return args.n ? blocks >= 8 && blocks * args.terms > 24
                : plan_tiles(tiles, blocks, blocks * args.terms, clusters).splits > 1;
}

cudaError_t launch_slots_out(const TrainArgs& args, const SlotsOut& s, int clusters,
                             cudaStream_t stream) {
  const int64_t tiles = static_cast<int64_t>((args.M + S::BM - 1) / S::BM) *
                        ((args.N + args.width - 1) / args.width);
  const int64_t most = 64 * (s.all || tiles < clusters ? tiles : clusters);  // a tail is under a wave
  const int64_t cap = 16 * clusters;  // 8 blocks an SM
  return launch_kernel(slots_out_kernel, dim3(static_cast<unsigned>(most < cap ? most : cap)),
                       dim3(256), 0, stream, args, s, clusters);
}

cudaError_t launch_operand_copy(const OperandCopy& job, int sm_count, cudaStream_t stream) {
  return launch_kernel(operand_copy_kernel, dim3(operand_copy_blocks(job, sm_count)), dim3(256), 0,
                       stream, job);
}

cudaError_t launch_train_tc(int mode, bool promote, const TrainMaps& maps, const TrainArgs& args,
                            int clusters, cudaStream_t stream) {
  return launch_kernel(kernel_of(mode, promote, args.width), dim3(2 * clusters), dim3(S::THREADS),
                       S::SMEM_BYTES, stream, maps, args);
}

}  // namespace gemm14
