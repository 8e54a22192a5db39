// Host check of the training kernel's tile plan (train_tc.h): over a sweep of
// tile counts, k-blocks and clusters, every k-block of every tile is worked on
// exactly once, whole tiles fill whole waves before the split ones, slots are
// distinct and within the count the workspace is sized for.
#include <cstdio>
#include <set>

#include <cuda_runtime.h>

#include "train_tc.h"

using namespace gemm14;

int main() {
  long plans = 0, splits = 0;
  for (int clusters : {1, 3, 38, 74, 76})
    for (int tiles = 0; tiles <= 400; tiles += tiles < 160 ? 1 : 7)
      for (int kblocks : {0, 1, 4, 7, 8, 9, 16, 39, 128, 513, 2049})
        for (int terms : {1, 3, 6})
          for (bool all : {false, true}) {
            const TilePlan p = plan_tiles(tiles, kblocks, kblocks * terms, clusters);
            ++plans;
            const int tail = p.tiles - p.direct;
            if (p.tiles != tiles || p.splits < 1 || p.direct < 0 || p.direct > tiles) return 1;
            if (p.splits == 1 && tail != 0) return 2;
            if (p.splits > 1) {
              ++splits;
              if (p.direct % clusters != 0 || tail <= 0 || tail >= clusters) return 3;
              if (kblocks / p.splits < 4) return 4;
            }
            const long most = slots_needed(tiles, kblocks, clusters, all);
            std::set<long> used;
            for (int t = 0; t < tiles; ++t) {
              const bool whole = t < p.direct;
              int next = 0;
              for (int s = 0; s < (whole ? 1 : p.splits); ++s) {
                if (!whole) {
                  const int k0 = static_cast<long>(kblocks) * s / p.splits;
                  const int k1 = static_cast<long>(kblocks) * (s + 1) / p.splits;
                  if (k0 != next) return 5;
                  next = k1;
                }
                if (whole && !all) continue;
                const long slot = slot_of(p, all, t, s);
                if (slot < 0 || slot >= most || !used.insert(slot).second) {
                  std::printf("tiles %d kblocks %d clusters %d all %d: slot %ld of %ld\n", tiles,
                              kblocks, clusters, all, slot, most);
                  return 6;
                }
              }
              if (!whole && next != kblocks) return 7;
            }
            // a plan of fewer tiles or k-blocks fits the slots of the larger one
            if (tiles > 0) {
              const TilePlan q = plan_tiles(tiles - 1, kblocks, kblocks * terms, clusters);
              const long last = q.tiles == 0 ? -1 : q.tiles == q.direct && !all
                                    ? -1 : slot_of(q, all, q.tiles - 1, q.tiles == q.direct ? 0 : q.splits - 1);
              if (last >= most) return 8;
            }
          }
  std::printf("%ld plans, %ld with split tiles\n", plans, splits);
  return splits > 0 ? 0 : 9;
}
