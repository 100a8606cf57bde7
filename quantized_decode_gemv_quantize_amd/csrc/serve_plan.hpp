// serve_plan.hpp - launch arithmetic of the operators of a step over many
// requests, shared by the launchers, the kernels and the host model of the tests.
#pragma once

#include "decode_plan.hpp"

namespace qmv {

constexpr int kLBlock = 64;                    // consecutive rows among which tiles are formed
constexpr int kLStep = 32;                     // of K, or ranks, a matrix product
constexpr int kLColumns = 16;                  // rows of x a matrix product
constexpr int kAWaves = 8, kBWaves = 4;        // of a workgroup of shrink and of expand
constexpr int kLoraChunk = kAWaves * kLStep;   // of K that a workgroup of shrink takes at a time
constexpr int kLoraPiece = kBWaves * 64;       // outputs that one of expand takes at a time

// Whether rows of floats are more than so many bytes, from which on they pass
// caches by: the L2 of all eight dies hold 32 MB, the last-level cache 256 MB,
// beside all else that the rows' reader needs.
inline bool past_caches(int64_t rows, int64_t length, int64_t bytes) { return rows * length * 4 > bytes; }
constexpr int64_t kL2 = int64_t(32) << 20;

// Embedding rows, stored as usual, through the L2 and past all caches: us alone
// and with the norm that makes q8_1 columns of them. Q4_K rows of 4096, 49 MB
// 15.1, 12.4, 11.2 and 41.8, 40.7, 44.1; 67 MB 17.4, 15.2, 13.2 and 52.4, 51.3,
// 56.1; 98 MB 24.9, 20.7, 18.6 and 75.0, 75.0, 79.3; 134 MB 31.4, 28.8, 24.9 and
// 118, 119, 104 (110, 120, 121 where the norm makes fp32 rows). BF16 rows of
// 2565, which end inside a line of 128 bytes, 62 MB 17.1, 17.4, 16.5 and, with
// fp32 rows of a norm, 55.6, 63.7, 62.2; 92 MB 24.4, 39.0, 23.8 and 90.0, 96.4,
// 92.8. So through the L2 from 32 MB on where rows are whole lines, and past
// the caches from here on. (8 MB past the caches 4.8 -> 5.0 alone.)
constexpr int64_t kEmbedPast = int64_t(104) << 20;

// Adapters' x, read past the caches from there on, and as usual before: us
// alone, and with the norm behind the projection and another reader of x. 34 MB
// (2100 rows of 4096) 49.8, 47.7 and 93.5, 91.7; 63 MB (1100 of 14336) 50.3, 45.4
// and 90.2, 88.6; 67 MB (4096 of 4096) 63.5, 65.9 and 155, 161; 86 MB (1500 of
// 14336) 77.6, 72 and 129, 132; 235 MB (4096 of 14336) 105, 127 and 252, 262.
constexpr int64_t kLoraPast = int64_t(63) << 20;

// Their out, stored as usual and past the caches: us alone, with the norm that
// adds it to the residual, with a norm of it. 52 MB (2100 rows of 4096 by 6144)
// 64.5, 56.5 and 106, 107 and 86.9, 88.0; 67 MB (4096 of 14336 by 4096) 115, 106
// and 166, 167 and 143, 149; 134 MB (8192 of 4096 by 4096) 126, 124 and 222, 225
// and 188, 189; 235 MB (4096 of 4096 by 14336) 171, 168 and 332, 342 and 250,
// 256. So past the caches from 32 MB up to there; in place it is all one.
constexpr int64_t kLoraOut = int64_t(104) << 20;

// Launch shape. How many tiles there are the host cannot see: it counts on
// rows of their own adapters in one block of rows, of one adapter beyond.
// K is cut towards a workgroup for every compute unit, in ranges of two chunks
// at least, or two of them in ranges of four (64 rows of their own, K = 4096:
// 4 ranges 34.6 us, 8 of two chunks 37.6; one row: 8.5 and 7.5; 4000 rows of
// 14336: 5 ranges 98, 3 108). M is cut towards two for every compute unit, in
// pieces of 256: 64 rows by 14336 in 8 slices 34.6 us, in 4 50, in 16 54; 4000 by
// 4096 in 5 115, in 3 129, in 10 126. Few rows do not fill the chip so: one of 4096
// by 4096 has 8 workgroups and then 16, which at high ranks stream its adapter
// at some 250 GB/s (rank 128 in fp32 27 us).
// From 1024 rows on tiles take 32, which halves the reads of the weights, but
// also the tiles to share them out by, and counts double where rows have adapters
// of their own. Tiles of 16 and of 32, 8 requests, us: 4096 by 4096, bf16 of rank
// 16, 1024 rows 26, 33, 2048 41, 45, 4096 73, 62, 8192 125, 131; fp32 of rank 64 88, 84
// and 104, 102 and 187, 142 and 327, 264; 4096 by 14336, bf16 of rank 16 62, 57 and
// 91, 87 and 185, 165 and 344, 340; 2048 rows of 1024 requests 86, 118.
// A workgroup looks for tiles at four rows of each block where there are several:
// most of one at each row would find none (512 rows of 8 adapters 46 -> 37 us,
// 512 of their own 53 -> 56).
struct LoraShape {
  int blocks, leads, groups, splits, steps, slices, pieces, ct;
};
inline LoraShape lora_shape(int64_t n, int64_t K, int64_t M, int max_rank) {
  LoraShape s;
  s.ct = n >= 1024 && max_rank <= 64 ? 2 : 1;
  s.blocks = static_cast<int>((n + kLBlock - 1) / kLBlock);
  s.leads = s.blocks == 1 ? 1 : s.blocks <= 32 ? 4 : kLColumns * s.ct;   // rows of a block that a workgroup looks for tiles at
  const int rows = n < kLBlock ? static_cast<int>(n) : kLBlock;
  s.groups = (rows + s.leads - 1) / s.leads;
  int64_t tiles = (n + kLColumns * s.ct - 1) / (kLColumns * s.ct);
  if (tiles < rows) tiles = rows;
  const auto fill = [&](int64_t groups) { return (groups + tiles - 1) / tiles; };
  const int64_t chunks = (K + kLoraChunk - 1) / kLoraChunk, one = fill(kCus), two = fill(2 * kCus);
  const int64_t few = (chunks + 1) / 2 < one ? (chunks + 1) / 2 : one, some = (chunks + 3) / 4;
  int64_t splits = few > some ? few : some;
  if (splits > two) splits = two;
  if (splits > 16) splits = 16;
  s.steps = static_cast<int>((chunks + splits - 1) / splits);
  s.splits = static_cast<int>((chunks + s.steps - 1) / s.steps);
  const int64_t pieces = (M + kLoraPiece - 1) / kLoraPiece;
  int64_t slices = two < pieces ? two : pieces;
  if (slices > 64) slices = 64;
  s.pieces = static_cast<int>((pieces + slices - 1) / slices);
  s.slices = static_cast<int>((pieces + s.pieces - 1) / s.pieces);
  return s;
}

}  // namespace qmv
