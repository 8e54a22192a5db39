// train_tc.h -- the tensor-core kernel behind the training products
// (train_tc.cu): one mainloop on CTA pairs with the epilogues that the linear
// cross entropy and the weight gradient from 8-bit checkpoints need.
// Internal; nothing here crosses the library boundary.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace gemm14 {

// What becomes of a finished 256 x 256 tile of sums s (row i, column j):
//   kTrainStats  the tile's part of each row's sum of exponentials, and the
//                target's logit where the tile holds it (nothing else is kept);
//   kTrainGrad   (exp(s - lse[i]) - [j == target[i]]) coef[i], in 16 bits (or as
//                three bf16 parts of the fp32 value), rows from n on zero;
//   kTrainSlots  s into (or added to) the tile's slot of a private fp32 buffer;
//   kTrainOut    alpha s (+ beta out), row-major, in fp32, bf16 or fp16 (split
//                tiles: their sums into slots).
enum : int { kTrainStats = 0, kTrainGrad = 1, kTrainSlots = 2, kTrainOut = 3 };

// Element types of what an epilogue writes.
enum : int { kElemF32 = 0, kElemBf16 = 1, kElemF16 = 2, kElemBf16x3 = 3 };

// Largest size of a product: whole tiles of it are counted, and a tile's last
// column numbered, in 32 bits.
constexpr int64_t kTrainMaxSize = (int64_t(1) << 31) - 256;

struct TrainShape {
  static constexpr int BM = 256, BN = 256, BK = 64, STAGES = 6;
  static constexpr int EPI_WARPS = 8;                   // two for each TMEM lane quarter
  static constexpr int THREADS = (2 + EPI_WARPS) * 32;  // + producer, MMA
  static constexpr int A_BYTES = 128 * BK * 2, B_BYTES = 128 * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int OUT_BUF_BYTES = 32 * 128;  // per epilogue warp: 32 rows of 128 bytes
  static constexpr int TMEM_COLS = 512;
  static constexpr int SMEM_BYTES =
      STAGES * STAGE_BYTES + EPI_WARPS * OUT_BUF_BYTES + 256 + 1024;
  // k-blocks whose products one TMEM accumulator takes before the sum goes to
  // fp32 registers. The tensor cores add with truncation: measured on GB300,
  // n MMAs of K = 16 in a row leave a relative error of about 0.4 n 2^-24 (512
  // of them, K = 8192: 6.7e-6, against 6e-7 for an fp32 FMA sum). 64 MMAs, 16
  // k-blocks, leave 6e-7. Half as many leave 3e-7 and cost 1 to 5 % (wgrad 8192 x
  // 4096 x 11008: 535 -> 563 us): the drains then wait for each other.
  static constexpr int CHUNK = 16;
  // The same for logits, in both directions. Truncation moves them one way, a
  // learnt row's target the furthest, and adds up in lse - z_y, which is small
  // there: after 64 MMAs the losses of 600 such rows of fp16 over 1000 x 960 were
  // 1.2e-6 off (an fp32 product: 4e-7), after 32 they are 5e-7. dZ_y = exp(z_y -
  // lse) - 1 is such a difference too, and wants the very sums that lse came
  // from: with all of 4096 terms in one accumulator in the backward pass alone, dH of
  // rows of p_y = 0.99 .. 0.9995 was up to 11 % (bf16) and 19 % (fp16) off,
  // with 8192 terms 23 and 30 %; so it is 0.5 and 0.3 %, dZ's rounding or p_y's.
  // A step of 4096 x 65536 x 4096 bf16 takes 5533 -> 5679 us for it, 2047 x 50021 x
  // 1000 fp16 576 -> 591, 515 x 8191 x 769 fp32 256 -> 260.
  static constexpr int LOGITS_CHUNK = 8;
};

struct TrainArgs {
  // The product: M x N sums over K. n: the device's count of rows in use, in
  // place of M (or of K where n_is_k), or null.
  int M, N, K;
  const int* n;
  int n_is_k;
  int a_mn, b_mn;       // operand stored with its M (N) dimension contiguous
  // The sum over terms of products of operand parts (a value split in bf16
  // parts): nibble t of term_code is part(A) | part(B) << 2 of term t.
  int terms;
  uint32_t term_code;
  int width;            // columns of a tile: 256, or 128 (B stored K x N)
  int split_k;          // K that the split of tiles is planned for (0: none are split)
  uint32_t idesc;
  unsigned* err;
  unsigned long long wait_limit_ns;
  int fault;

  // kTrainStats, kTrainGrad: the vocabulary column of tile column 0 and
  // per-row data of the rows in use
  int v0;
  const int* target;            // column of the target, < 0: none
  const int64_t* target64;      // the same as the caller holds it (where target is null)
  const float* lse;
  const float* coef;
  float2* part;                 // [(tile column) * 2 + half][row], pitch part_ld
  int64_t part_ld;
  float* target_logit;          // [row]
  // kTrainGrad, kTrainOut: the output (part p of three at out + p * out_part)
  void* out;
  int64_t ld_out, out_part;
  int elem, out_vec;            // element type; rows start and end on 16 bytes
  float alpha, beta;
  const float* scale;           // device factor on alpha, or null
  // kTrainSlots
  float4* slots;
  int add;                      // add to what the slots hold
  // what the buffers hold, for the bounds checks of a checked build: rows and
  // columns of out, slots, entries of part
  int64_t out_rows, out_cols, slot_count, part_count;
};

// How a launch's tiles are worked on by `clusters` clusters: the first `direct`
// tiles whole, in full waves; each of the rest, which would leave clusters idle
// in a last partial wave, by `splits` ranges of its k-blocks whose sums go to
// slots and are added up by launch_slots_out (1: those tiles are whole too, and
// direct counts them). For each number of partial waves, 1 to 4, the most ranges
// that fit it are a candidate; the shortest wins (1 % of a tile's time is counted
// for each range's sums). A split has to save 24 k-blocks' time (about 8 us: the
// second launch takes 4 to 6), and a range has 4 k-blocks or more. Both launches
// work it out on the device, every thread from the rows in use: in whole
// numbers, a few instructions (trying every count took 5 us of each launch).
// `units`: k-blocks times terms.
struct TilePlan {
  int tiles, direct, splits;
};
constexpr int kTailWaves = 4;
__host__ __device__ inline TilePlan plan_tiles(int tiles, int kblocks, int units, int clusters) {
  const int tail = tiles % clusters;
  int best = 1, best_time = 1000;  // thousandths of a tile's time
  for (int waves = 1; waves <= kTailWaves && tail; ++waves) {
    int s = waves * clusters / tail;
    if (s > kblocks / 4) s = kblocks / 4;
    if (s > 64) s = 64;
    if (s < 2) continue;
    const int time = 1000 * waves / s + 10 * s;
    if (time < best_time - 30) {
      best_time = time;
      best = s;
    }
  }
  if ((1000 - best_time) * static_cast<int64_t>(units) < 24000) best = 1;
  return TilePlan{tiles, best > 1 ? tiles - tail : tiles, best};
}
// The slot of split s of a tile. all: every tile has slots (kTrainSlots).
__host__ __device__ inline int64_t slot_of(const TilePlan& p, bool all, int tile, int s) {
  if (tile < p.direct) return tile;
  return (all ? p.direct : 0) + static_cast<int64_t>(tile - p.direct) * p.splits + s;
}
// Slots that a launch of at most this many tiles of at most this many k-blocks
// can need.
inline int64_t slots_needed(int64_t tiles, int64_t kblocks, int clusters, bool all) {
  const int64_t ranges = kblocks / 4 < 64 ? kblocks / 4 : 64;
  const int64_t most = static_cast<int64_t>(kTailWaves) * clusters;
  const int64_t split = ranges < 2 ? 0 : tiles * ranges < most ? tiles * ranges : most;
  return (all ? tiles : 0) + split;
}
// float4 v (columns 4v ..) of chunk c (32 columns) of half h (128 columns) of row
// q of CTA r's 128 rows, in slot k: rows next to one another.
__host__ __device__ inline int64_t slot_index(int64_t k, int r, int h, int c, int v, int q) {
  return (((k * 2 + r) * 2 + h) * 4 + c) * 1024 + v * 128 + q;
}
constexpr int64_t kSlotBytes = 256 * 256 * 4;

// Columns of a tile of a kTrainOut product over `units` k-blocks times terms.
// Half the width halves the sums a tile writes (and reads, with beta) beside its
// products, and spreads short ones more evenly: dW of 4096 x 4096 from 16 rows 37
// -> 32 us, 4096 x 11008 from 256 rows 97 -> 92; from 1000 rows it loses (56 ->
// 58): A's k-blocks then feed half as many MMAs, and shared memory holds those to
// 58 % of their rate (2458 x 131072 x 2048: 785 us, 1359 on 128 columns, 945 on 192).
inline int tile_width(int64_t units) { return units <= 4 ? 128 : 256; }

// Clusters of two that fit at once on the current device (0: they cannot run).
int train_max_clusters();

// The parts' tensor maps (boxes of 64 k x 128 rows, K-major, or 64 x 64, with
// the 128-byte swizzle).
struct TrainMaps {
  CUtensorMap a[3], b[3];
};

// One operand of a launch: `parts` matrices of 16-bit elements, part p at
// base + p * part_stride (elements), rows x cols as stored, pitch ld.
struct TrainOperand {
  const void* base;
  int64_t rows, cols, ld;
  int parts;
  int64_t part_stride;
};
// The maps of A (M x K, or stored K x M when a_mn) and B (N x K, or K x N when
// b_mn), and the terms, instruction descriptor and a_mn / b_mn of *args, whose
// width is set.
// Returns a gemm14_status.
// a_rows, b_rows: of the K-major operands' boxes (0: a CTA's of a pair).
int train_operands(bool bf16, const TrainOperand& A, bool a_mn, const TrainOperand& B, bool b_mn,
                   TrainMaps* maps, TrainArgs* args, int a_rows = 0, int b_rows = 0);

// What follows a launch with slots: out[r] = alpha * *scale * (sum of row r's
// slots) + beta * out[r], for the rows in use (all: of every tile; otherwise of
// the split ones), row r going through `rows` where it is set. The other
// arguments are the launch's.
struct SlotsOut {
  bool all;
  const int* rows;
  float alpha, beta;
  const float* scale;
  void* out;
  int64_t ld;
  int elem;
  int64_t out_rows;
  int fold = 0;  // 1: row r's sums are those of rows r and r + 128 of its tile
};
// clusters: the launch's.
cudaError_t launch_slots_out(const TrainArgs& args, const SlotsOut& s, int clusters,
                             cudaStream_t stream);
// Whether a kTrainOut launch may split tiles (then launch_slots_out follows it).
bool may_split(const TrainArgs& args, int clusters);

// A rows x cols operand to copy (operand_copy.cuh): parts = 1, 16-bit elements
// at any address and pitch to rows that start on 16 bytes; parts = 3, fp32 values
// to three bf16 parts, part_stride elements apart. rows = 0: nothing.
struct OperandCopy {
  const void* src;
  int64_t ld_src, rows, cols;
  void* dst;
  int64_t ld_dst, part_stride;
  int parts;
};
// Blocks of 256 threads for it, at most 8 an SM.
inline int operand_copy_blocks(const OperandCopy& j, int sm_count) {
  const int64_t per_warp = j.parts == 3 ? 256 : 1024;  // columns of a row
  const int64_t blocks = (j.rows * ((j.cols + per_warp - 1) / per_warp) + 7) / 8;
  const int64_t cap = static_cast<int64_t>(sm_count) * 8;
  return static_cast<int>(blocks < cap ? blocks : cap);
}
cudaError_t launch_operand_copy(const OperandCopy& job, int sm_count, cudaStream_t stream);

// ---- few rows (train_tc.cu, train_few_kernel): kTrainStats or kTrainGrad with
// M <= 128 on one SM a tile of `width` columns; sums are always promoted.
struct FewShape {
  static constexpr int MAX_ROWS = 128;
  // As TrainShape::CHUNK; memory bounds this kernel, and one row's loss may be a
  // small difference of large numbers (1e-6 off with 16, 5e-7 with 4).
  static constexpr int CHUNK = 4;
  static constexpr int THREADS = TrainShape::THREADS;
  static constexpr int A_BYTES = 128 * 128;  // a k-block of 128 rows, as the MMA reads it
  static constexpr int MAX_STAGES = 12;
  static constexpr int RING_BYTES = 192 * 1024;
  static constexpr int SMEM_BYTES =
      RING_BYTES + TrainShape::EPI_WARPS * TrainShape::OUT_BUF_BYTES + 512 + 1024;
};
// Columns a tile, a multiple of 16 up to 256: the width at which the SM with
// the most tiles has the fewest columns.
int few_width(int64_t N, int sms);
// A's k-blocks are loaded with `rows` rows (16, or a multiple of 32 that holds M).
int few_rows(int64_t M);
// maps.a: boxes of 64 k x few_rows(M) rows; maps.b: 64 k x width rows, both K-major.
cudaError_t launch_train_few(int mode, const TrainMaps& maps, TrainArgs args, bool bf16, int width,
                             int sm_count, cudaStream_t stream);

// promote: sums leave the accumulators for fp32 registers every CHUNK k-blocks.
cudaError_t launch_train_tc(int mode, bool promote, const TrainMaps& maps, const TrainArgs& args,
                            int clusters, cudaStream_t stream);

}  // namespace gemm14
