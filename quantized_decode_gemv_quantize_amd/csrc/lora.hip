// lora.hip - low-rank adapters of many requests beside a shared projection.
//
//   v = A_a x[t] (r numbers a row), out[t] = base[t] + scale_a * B_a v
//
// Two launches: shrink (v, in ranges of K) and expand (v of all ranges
// summed, B_a v, the addition). Up to 16 rows of one adapter (32 in large
// batches), out of 64 consecutive ones, share its weights: a side of 16x16x32
// bf16 matrix products, whose other side is 16 rows of A or B. Rows of one adapter are
// found in the ids of the 64 by a ballot, so that nothing has to be sorted
// or listed first; single tokens of as many adapters leave 15 of a tile's 16
// columns empty, but then the weights are all there is to read, and the
// products wait for them anyway.
//
// Bound by memory where there are many rows, by the chain of two launches, the
// ids, the ranks and the first loads where there are few: one row of 4096 by
// 4096 3.9 + 5.3 us. Adapters are rows of max_rank, of which a lower rank uses the
// front: B's lines are fetched whole, 64 rows of their own adapters of ranks 8
// to 64 read 77 MB for the 47 that count (expand 24 us, 3.3 TB/s). 4000 rows of
// 14336 by 4096, bf16 of rank 32: shrink 61 us (240 MB, 3.9 TB/s), expand 36
// (146 MB, 4.1).
//
// fp32 values enter a product as three bf16 parts by truncation, x = x1 + x2 +
// x3 exactly (8 bits each; what lies below 2^-133, bf16's last bit, is lost);
// weights as one (bf16), two (fp16: 11 bits) or three (fp32). All products of
// parts but that of the two last of three and three (2^-28 of the whole) are
// formed: fp32 products, for three, six or eight matrix instructions where one of
// fp32 takes the time of sixteen.
#include "launch.hpp"
#include "past.hpp"
#include "serve_args.hpp"

namespace qmv {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kPad = 4;                        // floats behind a row in LDS: rows a bank group apart

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// High halves of two words: two bf16 by truncation.
__device__ __forceinline__ uint32_t high_halves(float lo, float hi) {
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
__device__ __forceinline__ float truncated(float v) { return __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); }

// The first N bf16 parts of eight values.
template <int N>
__device__ __forceinline__ void split8(const float (&v)[8], u32x4 (&part)[N]) {
  float rest[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) rest[e] = v[e];
#pragma unroll
  for (int p = 0; p < N; ++p) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) part[p][e / 2] = high_halves(rest[e], rest[e + 1]);
    if (p + 1 < N) {
#pragma unroll
      for (int e = 0; e < 8; ++e) rest[e] -= truncated(rest[e]);
    }
  }
}

// Eight consecutive weights: as they are stored, and as bf16 parts.
template <int TYPE>
struct Weights {
  static constexpr int kParts = TYPE == MMVQ_BF16 ? 1 : TYPE == MMVQ_F16 ? 2 : 3;
  static constexpr int kBytes = TYPE == MMVQ_F32 ? 4 : 2;
  static constexpr int kQuads = TYPE == MMVQ_F32 ? 2 : 1;
  u32x4 raw[kQuads];
  __device__ __forceinline__ void load(const uint8_t* m, int64_t i) {
#pragma unroll
    for (int q = 0; q < kQuads; ++q) raw[q] = ld_a16_x4(m + i * kBytes + 16 * q);
  }
  // Those from `valid` on become 0 (8 and more: none).
  __device__ __forceinline__ void cut(int valid) {
#pragma unroll
    for (int q = 0; q < kQuads; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (TYPE == MMVQ_F32) raw[q][e] = 4 * q + e < valid ? raw[q][e] : 0u;
        else raw[q][e] &= (2 * e < valid ? 0x0000FFFFu : 0u) | (2 * e + 1 < valid ? 0xFFFF0000u : 0u);
      }
  }
  __device__ __forceinline__ void split(u32x4 (&part)[kParts]) const {
    if constexpr (TYPE == MMVQ_BF16) {
      part[0] = raw[0];
    } else {
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (TYPE == MMVQ_F32) {
          v[e] = __uint_as_float(raw[0][e]);
          v[e + 4] = __uint_as_float(raw[1][e]);
        } else {
          v[2 * e] = h2f(raw[0][e]);
          v[2 * e + 1] = h2f(raw[0][e] >> 16);
        }
      }
      split8<kParts>(v, part);
    }
  }
};

// c += weights x values over their parts, largest last.
template <int PARTS>
__device__ __forceinline__ f32x4 multiply(const u32x4 (&w)[PARTS], const u32x4 (&x)[3], f32x4 c) {
#pragma unroll
  for (int order = 3; order >= 0; --order)     // parts p and q are below 2^-7(p + q) of the product
#pragma unroll
    for (int p = PARTS - 1; p >= 0; --p)
      if (order - p >= 0 && order - p <= 2) c = mfma_bf16(w[p], x[order - p], c);
  return c;
}

// The tile that row `lead` of a block of 64 leads, the same in every wave.
struct Tile {
  int adapter;             // -1: none
  int rank;
  int count;               // rows; 0: none
  int row;                 // in lane i that of row i of the tile, the first one's behind count
  float scale;
};

__device__ __forceinline__ int adapter_of(const LoraArgs& a, int t) {
  const int s = a.row_seq ? a.row_seq[t] : t;
  if (s < 0 || s >= a.n_seqs) return -1;
  const int id = a.adapter[s];
  return id >= 0 && id < a.n_adapters ? id : -1;
}

// Adapters of the block's rows, one a lane; -2 behind the last row.
__device__ __forceinline__ int block_ids(const LoraArgs& a, int block) {
  const int t = block * kLBlock + lane_id();
  return t < a.n ? adapter_of(a, t) : -2;
}

template <int CT>
__device__ __forceinline__ Tile tile_of(const LoraArgs& a, int block, int ids, int lead) {
  constexpr int kRows = kLColumns * CT;
  Tile tile{__builtin_amdgcn_readlane(ids, lead), 0, 0, 0, 0.0f};
  const uint64_t same = __ballot(ids == tile.adapter);
  const int ahead = __builtin_popcountll(same & ((uint64_t(1) << lead) - 1));
  if (tile.adapter == -2 || ahead % kRows) return tile;
  const int left = __builtin_popcountll(same) - ahead;
  tile.count = left < kRows ? left : kRows;
  const int lane = lane_id(), mine = __builtin_popcountll(same & ((uint64_t(1) << lane) - 1)) - ahead;
  const bool member = ids == tile.adapter && mine >= 0 && mine < kRows;
  const int pushed = __builtin_amdgcn_ds_permute(4 * (member ? mine : kWave - 1), lane);
  tile.row = block * kLBlock + __shfl(pushed, lane < tile.count ? lane : 0);
  if (tile.adapter >= 0) {
    const int r = a.rank ? a.rank[tile.adapter] : a.max_rank;
    tile.rank = r < 0 ? 0 : r > a.max_rank ? a.max_rank : r;
    tile.scale = a.scale ? a.scale[tile.adapter] : 1.0f;
  }
  return tile;
}

__device__ __forceinline__ f32x4 ld_f4(const float* p) {   // 4-byte aligned
  return __builtin_bit_cast(f32x4, ld_x4(reinterpret_cast<const uint8_t*>(p)));
}
__device__ __forceinline__ void eight(f32x4 a, f32x4 b, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = a[e];
    v[e + 4] = b[e];
  }
}

// v of a tile over a range of K, 16 RT ranks at a time. The workgroup takes
// kLoraChunk of K after the other: rows of x go through LDS, as a row's values side
// by side are what memory reads best and 8 of each of 16 rows what the
// products take; each wave multiplies 32 of the chunk. The next chunk's loads
// are on their way meanwhile. Columns behind the tile's count and ranks
// behind the adapter's repeat real ones, so that no load waits for a condition;
// what comes of them is not stored, or not used.
// PAST: x passes the caches by (a branch about each load instead: 109 us for
// the prompts' 101).
template <int TYPE, int RT, int CT, bool PAST>
__global__ void __launch_bounds__(kAWaves * kWave) lora_shrink_kernel(LoraArgs a) {
  using W = Weights<TYPE>;
  constexpr int kRows = kLColumns * CT, kPer = kRows / kAWaves, kLine = kLoraChunk + kPad;
  __shared__ union {
    float x[2][kRows][kLine];
    f32x4 sums[kAWaves][RT][kWave];
  } lds;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane / 16;
  const int block = blockIdx.x, split = blockIdx.z;
  const int ids = block_ids(a, block);
  const int chunks = static_cast<int>((a.K + kLoraChunk - 1) / kLoraChunk);
  const int c0 = split * a.steps, c1 = c0 + a.steps < chunks ? c0 + a.steps : chunks;
  for (int lead = blockIdx.y * a.leads, end = lead + a.leads; lead < end; ++lead) {
    const Tile tile = tile_of<CT>(a, block, ids, lead);
    if (tile.count == 0 || tile.rank == 0) continue;       // uniform
    const float* x[kPer];                      // the wave's rows of the tile
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      x[i] = a.x + static_cast<int64_t>(__builtin_amdgcn_readlane(tile.row, wave + kAWaves * i)) * a.ldx + 4 * lane;
    const uint8_t* A = a.A + tile.adapter * a.stride_a * W::kBytes;
    for (int r0 = 0; r0 < tile.rank; r0 += 16 * RT) {
      f32x4 acc[RT][CT];
      int64_t w0[RT];                          // element of the lane's rank
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const int j = r0 + 16 * t + lane % 16;
        w0[t] = (j < tile.rank ? j : tile.rank - 1) * a.K;
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[t][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
      f32x4 next[kPer];
      W w[RT];
      const auto ld_row = [&](const float* p) QMV_INLINE { return PAST ? __builtin_bit_cast(f32x4, load_past(p)) : ld_f4(p); };
      const auto fetch = [&](int chunk) QMV_INLINE {       // values behind K are 0 and meet real weights
        const int64_t k = static_cast<int64_t>(chunk) * kLoraChunk, kw = k + kLStep * wave + 8 * g;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (wave + kAWaves * i < tile.count)             // uniform
            next[i] = k + 4 * lane < a.K ? ld_row(x[i] + k) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int t = 0; t < RT; ++t)
          if (RT == 1 || r0 + 16 * t < tile.rank) w[t].load(A, w0[t] + (kw < a.K ? kw : 0));
      };
      if (c0 < c1) fetch(c0);
      for (int c = c0; c < c1; ++c) {
        float(*at)[kLine] = lds.x[c & 1];
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (wave + kAWaves * i < tile.count) *reinterpret_cast<f32x4*>(&at[wave + kAWaves * i][4 * lane]) = next[i];
        u32x4 wp[RT][W::kParts];
#pragma unroll
        for (int t = 0; t < RT; ++t)
          if (RT == 1 || r0 + 16 * t < tile.rank) w[t].split(wp[t]);
        if (c + 1 < c1) fetch(c + 1);
        __syncthreads();                       // (the buffer was read two chunks ago, before the last barrier)
#pragma unroll
        for (int q = 0; q < CT; ++q) {
          const int column = lane % kLColumns + kLColumns * q;
          const float* from = &at[column < tile.count ? column : 0][kLStep * wave + 8 * g];
          float v[8];
          eight(*reinterpret_cast<const f32x4*>(from), *reinterpret_cast<const f32x4*>(from + 4), v);
          u32x4 xp[3];
          split8<3>(v, xp);
#pragma unroll
          for (int t = 0; t < RT; ++t)
            if (RT == 1 || r0 + 16 * t < tile.rank) acc[t][q] = multiply<W::kParts>(wp[t], xp, acc[t][q]);
        }
      }
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        __syncthreads();                       // LDS is read
#pragma unroll
        for (int t = 0; t < RT; ++t) lds.sums[wave][t][lane] = acc[t][c];
        __syncthreads();
        const int column = lane % kLColumns + kLColumns * c, row = __shfl(tile.row, column);
        for (int t = wave; t < RT; t += kAWaves) {
          const int j = r0 + 16 * t + 4 * g;
          f32x4 sum = lds.sums[0][t][lane];
#pragma unroll
          for (int w = 1; w < kAWaves; ++w) sum += lds.sums[w][t][lane];
          if (column < tile.count && j < a.max_rank)
            *reinterpret_cast<f32x4*>(a.part + (static_cast<int64_t>(split) * a.n + row) * a.max_rank + j) = sum;
        }
      }
      __syncthreads();                         // the sums are read
    }
  }
}

// base + scale * B v of a tile, for a slice of M; up to 32 RC ranks. The
// workgroup takes kLoraPiece outputs after the other; products go to LDS, and each
// wave adds whole rows of them to base: 1 KB side by side a load and a store,
// where the products' own layout has 64 bytes of each of 16 rows.
template <int TYPE, int RC, int CT>
__global__ void __launch_bounds__(kBWaves * kWave) lora_expand_kernel(LoraArgs a) {
  using W = Weights<TYPE>;
  constexpr int kRuns = kLoraPiece / (4 * kWave);   // of a row: four outputs a lane
  constexpr int kRows = kLColumns * CT, kPer = kRows * kRuns / kBWaves, kTiles = kLoraPiece / kBWaves / 16, kLine = kLoraPiece + kPad;
  __shared__ float lds[kRows][kLine], sums[kRows][kLStep * RC + kPad];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane / 16;
  const int block = blockIdx.x;
  const int ids = block_ids(a, block);
  // (pieces of a slice one after the other: 1% less than every gridDim.z-th)
  const int64_t slice = static_cast<int64_t>(a.pieces) * kLoraPiece, m_first = blockIdx.z * slice;
  const int64_t m_end = m_first + slice < a.M ? m_first + slice : a.M;
  for (int lead = blockIdx.y * a.leads, end = lead + a.leads; lead < end; ++lead) {
    const Tile tile = tile_of<CT>(a, block, ids, lead);
    if (tile.count == 0 || (tile.rank == 0 && a.base == a.out)) continue;   // uniform
    const uint8_t* B = a.B + (tile.adapter < 0 ? 0 : tile.adapter) * a.stride_b * W::kBytes;
    W w[kTiles][RC];
    const auto fetch = [&](int64_t m0) QMV_INLINE {
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        const int64_t m = m0 + 64 * wave + 16 * t + lane % 16, row = (m < a.M ? m : a.M - 1) * a.max_rank;
#pragma unroll
        for (int q = 0; q < RC; ++q) {
          const int j = kLStep * q + 8 * g;
          if (kLStep * q < tile.rank) w[t][q].load(B, row + (j < a.max_rank ? j : 0));   // uniform
        }
      }
    };
    if (m_first < m_end) fetch(m_first);       // on their way while v is summed
    // v: each four ranks of a row summed by one thread, 0 behind the adapter's rank (the sums there are others')
    constexpr int kRanks = kLStep * RC, kQuads = kRanks / 4;
    for (int i = static_cast<int>(threadIdx.x); i < kRows * kQuads; i += kBWaves * kWave) {
      const int c = i / kQuads, j = i % kQuads * 4;
      const float* part = a.part + static_cast<int64_t>(__shfl(tile.row, c)) * a.max_rank + j;
      const int64_t step = static_cast<int64_t>(a.n) * a.max_rank;
      f32x4 sum{0.0f, 0.0f, 0.0f, 0.0f};
      if (c < tile.count && j < tile.rank)
#pragma unroll 8
        for (int s = 0; s < a.splits; ++s) sum += ld_f4(part + s * step);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] = j + e < tile.rank ? sum[e] : 0.0f;
      *reinterpret_cast<f32x4*>(&sums[c][j]) = sum;
    }
    __syncthreads();
    u32x4 v[CT][RC][3];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int q = 0; q < RC; ++q) {
        const float* from = &sums[lane % kLColumns + kLColumns * c][kLStep * q + 8 * g];
        float one[8];
        eight(*reinterpret_cast<const f32x4*>(from), *reinterpret_cast<const f32x4*>(from + 4), one);
        split8<3>(one, v[c][q]);
      }
    __syncthreads();                           // (the next tile's sums)
    const bool cuts = tile.rank % kLStep != 0;   // uniform
    for (int64_t m0 = m_first; m0 < m_end; m0 += kLoraPiece) {
      f32x4 old[kPer];
      const float* base[kPer];
      float* out[kPer];
      int64_t o[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {         // the wave's runs of rows
        const int run = wave + kBWaves * i;
        const int64_t row = __builtin_amdgcn_readlane(tile.row, run / kRuns);
        o[i] = m0 + run % kRuns * 4 * kWave + 4 * lane;
        base[i] = a.base + row * a.ldb + o[i];
        out[i] = a.out + row * a.ldo + o[i];
        if (run / kRuns < tile.count && o[i] + 4 <= a.M) old[i] = ld_f4(base[i]);
      }
      if (tile.rank > 0) {                     // uniform
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          f32x4 acc[CT];
#pragma unroll
          for (int c = 0; c < CT; ++c) acc[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int q = 0; q < RC; ++q) {
            if (kLStep * q < tile.rank) {      // uniform
              if (cuts) w[t][q].cut(tile.rank - kLStep * q - 8 * g);
              u32x4 wp[W::kParts];
              w[t][q].split(wp);
#pragma unroll
              for (int c = 0; c < CT; ++c) acc[c] = multiply<W::kParts>(wp, v[c][q], acc[c]);
            }
          }
#pragma unroll
          for (int c = 0; c < CT; ++c)
            if (lane % kLColumns + kLColumns * c < tile.count)
              *reinterpret_cast<f32x4*>(&lds[lane % kLColumns + kLColumns * c][64 * wave + 16 * t + 4 * g]) = acc[c];
        }
        if (m0 + kLoraPiece < m_end) fetch(m0 + kLoraPiece);
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int run = wave + kBWaves * i;
        if (run / kRuns >= tile.count) continue;           // uniform
        f32x4 add{0.0f, 0.0f, 0.0f, 0.0f};
        if (tile.rank > 0) add = *reinterpret_cast<const f32x4*>(&lds[run / kRuns][run % kRuns * 4 * kWave + 4 * lane]);
        if (o[i] + 4 <= a.M) {
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = tile.rank > 0 ? old[i][e] + tile.scale * add[e] : old[i][e];
          store_four(out[i], y, CT == 2 && a.past);   // (single tokens: the branch alone 34.8 -> 35.3 us for 64 rows)
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (o[i] + e < a.M) out[i][e] = tile.rank > 0 ? base[i][e] + tile.scale * add[e] : base[i][e];
        }
      }
      if (tile.rank > 0) __syncthreads();      // LDS is read
    }
  }
}

int64_t lora_bytes(int64_t n, int64_t K, int64_t M, int max_rank) {
  if (n == 0) return 0;
  return lora_shape(n, K, M, max_rank).splits * n * max_rank * static_cast<int64_t>(sizeof(float));
}

template <int TYPE, int RT, int RC, int CT>
int launch_ranks(const LoraArgs& a, const LoraShape& s, hipStream_t st) {
  const dim3 grid(s.blocks, s.groups, s.splits), block(kAWaves * kWave);
  if (CT == 2 && past_caches(a.n, a.K, kLoraPast)) hipLaunchKernelGGL((lora_shrink_kernel<TYPE, RT, CT, CT == 2>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((lora_shrink_kernel<TYPE, RT, CT, false>), grid, block, 0, st, a);
  const int rc = check_launch();
  if (rc) return rc;
  hipLaunchKernelGGL((lora_expand_kernel<TYPE, RC, CT>), dim3(s.blocks, s.groups, s.slices), dim3(kBWaves * kWave), 0, st, a);
  return check_launch();
}

template <int TYPE>
int launch_type(const LoraArgs& given, hipStream_t st) {
  LoraArgs a = given;
  const LoraShape s = lora_shape(a.n, a.K, a.M, a.max_rank);
  a.splits = s.splits;
  a.steps = s.steps;
  a.leads = s.leads;
  a.pieces = s.pieces;
  a.past = past_caches(a.n, a.M, kL2) && !past_caches(a.n, a.M, kLoraOut);
  if (s.ct == 2) {
    if (a.max_rank <= 16) return launch_ranks<TYPE, 1, 1, 2>(a, s, st);
    if (a.max_rank <= 32) return launch_ranks<TYPE, 2, 1, 2>(a, s, st);
    return launch_ranks<TYPE, 4, 2, 2>(a, s, st);
  }
  if (a.max_rank <= 16) return launch_ranks<TYPE, 1, 1, 1>(a, s, st);
  if (a.max_rank <= 32) return launch_ranks<TYPE, 2, 1, 1>(a, s, st);
  if (a.max_rank <= 64) return launch_ranks<TYPE, 4, 2, 1>(a, s, st);
  if (a.max_rank <= 128) return launch_ranks<TYPE, 8, 4, 1>(a, s, st);
  return launch_ranks<TYPE, 8, 8, 1>(a, s, st);
}

int launch_lora(int type, const LoraArgs& a, hipStream_t st) {
  switch (type) {
    case MMVQ_F16: return launch_type<MMVQ_F16>(a, st);
    case MMVQ_BF16: return launch_type<MMVQ_BF16>(a, st);
    case MMVQ_F32: return launch_type<MMVQ_F32>(a, st);
    default: return MMVQ_ERR_TYPE;
  }
}

}  // namespace qmv
