// serve.cpp - host model of the adapters' launch arithmetic: the kernels' own
// header, run on the CPU.
#include <cstdio>
#include <vector>

#include "serve_plan.hpp"

using namespace qmv;

static long bad = 0;
#define CHECK(c, ...) do { if (!(c)) { if (++bad < 20) { printf("FAIL %s: ", #c); printf(__VA_ARGS__); printf("\n"); } } } while (0)

int main() {
  const int64_t ns[] = {1, 2, 3, 15, 16, 17, 63, 64, 65, 128, 500, 512, 513, 1000, 1023, 1024, 2048, 2049, 4096, 100000, 1 << 20};
  const int64_t Ks[] = {8, 16, 248, 256, 264, 512, 1024, 4096, 4104, 14336, 1 << 20};
  const int64_t Ms[] = {1, 255, 256, 257, 1000, 4096, 14336, 128256, 1 << 24};
  const int ranks[] = {8, 16, 24, 64, 72, 128, 256};
  for (int64_t n : ns)
    for (int64_t K : Ks)
      for (int64_t M : Ms)
        for (int rank : ranks) {
          const LoraShape s = lora_shape(n, K, M, rank);
          // every row is looked at once, the last workgroup's rows end with the block
          CHECK(static_cast<int64_t>(s.blocks) * kLBlock >= n && static_cast<int64_t>(s.blocks - 1) * kLBlock < n, "n %ld blocks %d", (long)n, s.blocks);
          const int64_t rows = n < kLBlock ? n : kLBlock;
          CHECK(s.groups * s.leads >= rows && s.groups * s.leads <= kLBlock && (s.groups - 1) * s.leads < rows, "n %ld leads %d groups %d", (long)n, s.leads, s.groups);
          // ranges of K cover it once, none is empty
          const int64_t chunks = (K + kLoraChunk - 1) / kLoraChunk;
          CHECK(s.splits >= 1 && s.splits <= 16 && s.steps >= 1, "splits %d steps %d", s.splits, s.steps);
          CHECK(static_cast<int64_t>(s.splits) * s.steps >= chunks && static_cast<int64_t>(s.splits - 1) * s.steps < chunks, "K %ld splits %d steps %d", (long)K, s.splits, s.steps);
          CHECK(s.pieces >= 1 && static_cast<int64_t>(s.slices) * s.pieces * kLoraPiece >= M &&
                static_cast<int64_t>(s.slices - 1) * s.pieces * kLoraPiece < M, "M %ld slices %d pieces %d", (long)M, s.slices, s.pieces);
          CHECK(s.slices >= 1 && s.slices <= 64 && static_cast<int64_t>(s.slices - 1) * kLoraPiece < M, "M %ld slices %d", (long)M, s.slices);
          CHECK(s.ct == 1 || (s.ct == 2 && rank <= 64), "ct %d rank %d", s.ct, rank);
          CHECK(static_cast<int64_t>(s.blocks) * s.groups * (s.splits > s.slices ? s.splits : s.slices) < (int64_t(1) << 31), "grid");
        }
  printf("%ld failing check(s)\n", bad);
  return bad != 0;
}
