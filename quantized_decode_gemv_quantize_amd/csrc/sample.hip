// sample.hip - the next tokens from rows of logits, by temperature, top-k,
// top-p and min-p.
//
//   w_i = exp((l_i - top) / T); in the order of falling logits, rising indices:
//   top-k keeps the first k, top-p those before which less than p * (sum of
//   these) has passed, min-p those with w_i >= m. All three keep a beginning
//   of the order, so what is kept is a border: the last kept logit and index.
//
// Nothing is sorted but the few tokens about that border. Launches:
//   stats   per row and chunk of kChunk logits: largest logit, sum of the
//           weights, and for filtered rows a histogram of their number and
//           sum over bins of a quarter octave of the weight, and the chunk's
//           tokens in its first bins (at most kTops);
//   pick    a workgroup a row: the chunks' histograms joined, and the bin in
//           which the border lies. Where no more than kArena tokens come up
//           to its end, they are cut and drawn from in LDS, sorted if they
//           are few; else the bin is narrowed until few are left of it;
//   probs   the distribution written out, if wanted, of rows that keep many;
//           of the others stats writes the zeros and pick what is kept.
// A chunk's bin is one 64-bit whole number: the count, and the sum in units of
// 2^-38 of 2^(-b/4) for bin b (adding in LDS in any order gives the same bits,
// and one addition a token is what the bins can bear).
// Cells of the search for a border hold such sums, too. Everything else is in 64
// bits or more: with 10^5 logits a running sum
// in 32 bits moves a border by more than many tokens' probability.
#include "draw.hpp"
#include "launch.hpp"
#include "past.hpp"
#include "serve_args.hpp"

namespace qmv {

constexpr int kSThreads = 256;
constexpr int kSPer = 16;                      // logits a lane
constexpr int kSWaves = kSThreads / kWave;
constexpr int kChunk = kSThreads * kSPer;
constexpr int kBins = 256;                     // the last one: everything below
constexpr int kDThreads = 512;
constexpr int kDWaves = kDThreads / kWave;
constexpr int kRank = 256;                     // tokens that are sorted, each by counting those before it
// Tokens that are cut and drawn from in LDS: what fits beside the descriptors of
// 2^24 logits' chunks. With 2560 256 rows of top-p (128256 logits) 113 -> 141 us
// and 128 with distributions 102 -> 185, the others 0.4 to 1 less.
constexpr int kArena = 5120;
// Tokens that a chunk lists. With 128 64 rows of top-p 56.7 -> 61.7 us, 256 of
// min-p 67.1 -> 63.8, one row 0.3 less; with 512 56.7 -> 52.5, 67.1 -> 71.7, one
// row 0.6 more.
constexpr int kTops = 256;
constexpr int kUnit = 38;                      // a bin's sum is in units of 2^-kUnit
constexpr int kSumBits = 51;                   // and behind them its count
constexpr uint64_t kSumMask = (uint64_t(1) << kSumBits) - 1;

struct ChunkStat {
  float top;                                   // largest logit of the chunk
  int at;                                      // its lowest index
  double sum;                                  // of the weights relative to top, in pick: of the kept ones to the row's
  int16_t listed;                              // tokens in its list: all those of its bins
  int16_t cut;                                 // up to this one
  int tokens;                                  // that have a weight
};
struct Pick {
  uint64_t border;                             // last kept place (below)
  double total;                                // sum of the kept weights; 0: none
  double rate;
  float top;
  int written;                                 // the distribution is there already
};

__device__ __forceinline__ ChunkStat* chunk_stats(const SampleArgs& a) { return reinterpret_cast<ChunkStat*>(a.ws); }
__device__ __forceinline__ Pick* picks(const SampleArgs& a) {
  return reinterpret_cast<Pick*>(chunk_stats(a) + static_cast<int64_t>(a.n_rows) * a.chunks);
}
__device__ __forceinline__ uint64_t* chunk_bins(const SampleArgs& a) { return reinterpret_cast<uint64_t*>(picks(a) + a.n_rows); }
__device__ __forceinline__ uint64_t* chunk_tops(const SampleArgs& a) {
  return chunk_bins(a) + static_cast<int64_t>(a.n_rows) * a.chunks * kBins;
}

int64_t sample_bytes(int n_rows, int vocab, int* chunks) {
  const int64_t c = (vocab + kChunk - 1) / kChunk;
  if (chunks) *chunks = static_cast<int>(c);
  return n_rows * (c * static_cast<int64_t>(sizeof(ChunkStat) + (kBins + kTops) * sizeof(uint64_t)) + static_cast<int64_t>(sizeof(Pick)));
}

// Settings of a row: log2(e) / T, and its filters (k = 0, p = 1, m = 0: off).
struct Settings {
  double rate, p, m;
  int k;
  bool none, greedy;                           // of no request; of temperature 0
  __device__ __forceinline__ bool filtered() const { return k > 0 || p < 1.0 || m > 0.0; }
  __device__ __forceinline__ bool plain() const { return !none && !greedy && !filtered(); }
};
__device__ __forceinline__ Settings settings_of(const SampleArgs& a, int r) {
  constexpr double kLog2e = 1.4426950408889634073599246810019;
  Settings s{kLog2e, 1.0, 0.0, 0, false, false};
  const int q = a.row_seq ? a.row_seq[r] : r;
  if (q < 0 || q >= a.n_seqs) {
    s.none = true;
    return s;
  }
  if (a.temperature) {
    const float t = a.temperature[q];
    s.greedy = !(t > 0.0f);
    s.rate = s.greedy ? 0.0 : kLog2e / static_cast<double>(t);
  }
  if (s.greedy) return s;
  if (a.top_k && a.top_k[q] > 0 && a.top_k[q] < a.vocab) s.k = a.top_k[q];
  if (a.top_p && a.top_p[q] < 1.0f) s.p = static_cast<double>(a.top_p[q]);
  if (a.min_p && a.min_p[q] > 0.0f) s.m = a.min_p[q] < 1.0f ? static_cast<double>(a.min_p[q]) : 1.0;
  return s;
}

// A logit as the operator takes it: no NaN, no negative zero.
__device__ __forceinline__ float taken(float v) { return v == v ? v + 0.0f : -INFINITY; }

// Whole numbers in the order of the logits.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return taken(__uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key));
}
// Places in the order of falling logits and rising indices.
constexpr int kIndexBits = 24;
constexpr uint64_t kLowIndex = (uint64_t(1) << kIndexBits) - 1;
__device__ __forceinline__ uint64_t place_of(float v, int i) {
  return static_cast<uint64_t>(~key_of(v)) << kIndexBits | static_cast<uint64_t>(i);
}
__device__ __forceinline__ uint64_t first_place(uint32_t key) { return static_cast<uint64_t>(~key) << kIndexBits; }
__device__ __forceinline__ uint64_t last_place(uint32_t key) { return first_place(key) | kLowIndex; }
__device__ __forceinline__ float value_at(uint64_t place) { return value_of(~static_cast<uint32_t>(place >> kIndexBits)); }

// Weight of a logit relative to `top`.
__device__ __forceinline__ double weight(const Exp2& exp2, float v, float top, double rate) {
  if (!(v > -INFINITY)) return 0.0;
  if (top == INFINITY) return v == top ? 1.0 : 0.0;
  return exp2((static_cast<double>(v) - static_cast<double>(top)) * rate);
}
// A quarter octave that a logit's weight lies in, on a grid that all chunks
// share: whole numbers that never fall with the logit. They and their
// differences are exact up to 2^53, and unlike logits that far up are more
// than kBins apart (2^-24 of their size).
__device__ __forceinline__ double quarter(float v, double rate4) { return floor(static_cast<double>(v) * rate4); }
// Bins between two quarters, the first one not below the other.
__device__ __forceinline__ int bins_between(double above, double below, int most) { return static_cast<int>(fmin(above - below, static_cast<double>(most))); }
// Bin of a logit below a largest one, kBins for none.
__device__ __forceinline__ int bin_of(float v, double rate4, float top, double top_quarter) {
  if (!(v > -INFINITY)) return kBins;
  if (top == INFINITY) return v == top ? 0 : kBins;
  return bins_between(top_quarter, quarter(v, rate4), kBins - 1);
}

// 2^(-b / 4), also for b below 0: what a bin's weights are relative to.
__device__ __forceinline__ double bin_scale(int b) {
  const double lower = b & 1 ? 0.84089641525371454303112547623321 : 1.0, half = b & 2 ? 0.70710678118654752440084436210485 : 1.0;
  return __builtin_ldexp(lower * half, -(b >> 2));
}
// A bin's sum in units: a whole number below 2^52 is the low bits of its sum with 2^52.
__device__ __forceinline__ double bin_units(uint64_t bin) {
  return __longlong_as_double(static_cast<long long>((bin & kSumMask) | 0x433ull << 52)) - 0x1p52;
}
__device__ __forceinline__ double bin_sum_of(uint64_t bin, int b) { return __builtin_ldexp(bin_units(bin), -kUnit) * bin_scale(b); }

// 2^(38 + x / 4) as a whole number, -1 <= x <= 1, in the low 52 bits of the
// result: the Taylor polynomial of degree 8 of exp(x ln 2 / 4), whose next
// term is below 4 10^-13 (a ninth of a unit), in units of 2^-kUnit, added to 2^52.
struct Units {
  static constexpr int kDegree = 8;
  double c[kDegree + 1];
  __device__ __forceinline__ Units() {
    double v = 0x1p38;
#pragma unroll
    for (int i = 0; i <= kDegree; ++i) {
      c[i] = v + (i == 0 ? 0x1p52 : 0.0);
      v = v * (0.69314718055994530941723212145818 / 4) / (i + 1);
    }
#pragma unroll
    for (int i = 0; i <= kDegree; ++i) asm("" : "+s"(c[i]));
  }
  __device__ __forceinline__ long long operator()(double x) const {
    double p = c[kDegree];
#pragma unroll
    for (int i = kDegree - 1; i >= 0; --i) p = fma(p, x, c[i]);
    return __double_as_longlong(p);
  }
};
static_assert(kUnit == 38);

// The row of a workgroup of a grid of chunks by rows. (Rows in a loop would
// have the compiler keep addresses and masks of every branch across it.)
constexpr int kGridRows = 1 << 15;
__device__ __forceinline__ int row_of_grid() { return static_cast<int>(blockIdx.z) * kGridRows + static_cast<int>(blockIdx.y); }

// Bound by vector instructions (44 to 56 a logit of filtered rows, of which 22,
// most of them 64-bit, form its bin and add to it, and most others list a
// chunk's tokens) and by the latencies of its steps; the LDS additions of lanes that meet in a bin
// are hidden behind them (four copies of the bins to keep them apart gained
// nothing: 57.3 and 58.6 us for 256 rows of 151669). 64 rows of 128256 take 18 us
// (33 MB, 1.8 TB/s), 256 of 151669 54 (155 MB, 2.9), 128 whose distributions' zeros
// it stores 33 (131 MB, 4.0).
__global__ void __launch_bounds__(kSThreads) sample_stats_kernel(SampleArgs a) {
  __shared__ float tops[kSWaves];
  __shared__ int ats[kSWaves], scans[kSWaves], next[kBins], ends[kBins], cut;
  __shared__ double sums[kSWaves];
  __shared__ unsigned long long bins[kBins];
  const int tid = threadIdx.x, wave = tid >> 6, c = blockIdx.x, i0 = c * kChunk + 4 * tid;
  const int r = row_of_grid();
  if (r >= a.n_rows) return;
  const Settings s = settings_of(a, r);
  const float* row = a.logits + r * a.ldl;
  float v[kSPer];                              // NaN as -inf
  if ((c + 1) * kChunk <= a.vocab) {           // uniform: all loads at once
#pragma unroll
    for (int k = 0; k < kSPer; k += 4) {
      const u32x4 x = ld_x4(reinterpret_cast<const uint8_t*>(row + i0 + k * kSThreads));
#pragma unroll
      for (int e = 0; e < 4; ++e) v[k + e] = fmaxf(__uint_as_float(x[e]), -INFINITY);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kSPer; ++k) {
      const int i = i0 + (k / 4) * 4 * kSThreads + k % 4;
      v[k] = row[i < a.vocab ? i : a.vocab - 1];
      v[k] = i < a.vocab ? fmaxf(v[k], -INFINITY) : -INFINITY;
    }
  }
  // (stores come last: a barrier would wait for those before it)
  const auto zeros = [&]() QMV_INLINE {
    if (!a.zeroed || s.plain()) return;        // the distribution's, while the chunk is here
    float* out = a.probs + r * a.ldp;
#pragma unroll
    for (int k = 0; k < kSPer; k += 4) {
      const int i = i0 + k * kSThreads;
      if (i + 4 <= a.vocab) {
        store_four(out + i, {0.0f, 0.0f, 0.0f, 0.0f}, a.past);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i + e < a.vocab) out[i + e] = 0.0f;
      }
    }
  };
  if (s.none) {                                // uniform
    zeros();
    return;
  }
  float top = -INFINITY;
  int at = 0x7fffffff;
#pragma unroll
  for (int k = 0; k < kSPer; ++k) top = fmaxf(top, v[k]);
  if (s.greedy) {                            // uniform; the others do without the index
#pragma unroll
    for (int k = kSPer - 1; k >= 0; --k)
      at = v[k] == top && top > -INFINITY ? i0 + (k / 4) * 4 * kSThreads + k % 4 : at;
  }
  wave_top(top, at);
  const bool filtered = s.filtered();
  if ((tid & 63) == 0) {
    tops[wave] = top;
    ats[wave] = at;
  }
  if (filtered) {
    bins[tid] = 0;
    if (tid == 0) cut = -1;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSWaves; ++w) take_top(top, at, tops[w], ats[w]);
  const bool any = !s.greedy && top > -INFINITY;
  double sum = 0.0;
  int bin[kSPer];
  float x[kSPer];
#pragma unroll
  for (int k = 0; k < kSPer; ++k) x[k] = v[k];
  if (top == INFINITY) {                     // uniform: the infinite ones share all
#pragma unroll
    for (int k = 0; k < kSPer; ++k) x[k] = v[k] == top ? 0.0f : -INFINITY;
  }
  const double dtop = top < INFINITY ? static_cast<double>(top) : 0.0, rate4 = 4.0 * s.rate, top_quarter = floor(dtop * rate4);
  if (any && !filtered) {
    const Exp2 exp2;                         // (in scalar registers that the other branch has no use for)
#pragma unroll
    for (int k = 0; k < kSPer; ++k) sum += exp2((static_cast<double>(x[k]) - dtop) * s.rate);
  } else if (any) {
    const Units units;
    constexpr long long kOne = (1ll << kSumBits) - (0x433ll << 52);   // a count, without the exponent of 2^52
#pragma unroll
    for (int k = 0; k < kSPer; ++k) {
      const double d = static_cast<double>(x[k]);
      const double down = fmin(top_quarter - floor(d * rate4), kBins - 1.0);
      const int b = static_cast<int>(down);
      // 4 log2(w) + b is within +-1 but for the last bin, whose tokens count
      // as 2^-64 of the largest at least: 2^-52 of the sum for all of them
      const double f = fmax(fma(d - dtop, rate4, down), -1.0);
      const unsigned long long add = static_cast<unsigned long long>(units(f) + kOne);
      if (x[k] > -INFINITY) atomicAdd(&bins[b], add);
      bin[k] = x[k] > -INFINITY ? b : kBins;
    }
  }
  __syncthreads();
  unsigned long long all = 0;
  if (filtered) {
    // the bins of at most kTops tokens together
    all = bins[tid];
    sum = bin_sum_of(all, tid);
    const int count = static_cast<int>(all >> kSumBits);
    int up = wave_scan(count);
    if (lane_id() == kWave - 1) scans[wave] = up;
    __syncthreads();
    for (int w = 0; w < wave; ++w) up += scans[w];
    next[tid] = up - count;
    ends[tid] = up;
    const uint64_t fits = __ballot(up <= kTops);
    if (lane_id() == 0 && fits) atomicMax(&cut, 64 * wave + 63 - __builtin_clzll(fits));
  }
  sum = wave_sum(sum);
  if ((tid & 63) == 0) sums[wave] = sum;
  __syncthreads();
  const int64_t place = static_cast<int64_t>(r) * a.chunks + c;
  if (tid == 0) {
    double whole = 0.0;
#pragma unroll
    for (int w = 0; w < kSWaves; ++w) whole += sums[w];
    const bool lists = filtered && cut >= 0;
    chunk_stats(a)[place] = ChunkStat{top, at, whole, static_cast<int16_t>(lists ? ends[cut] : 0), static_cast<int16_t>(lists ? cut : -1),
                                      filtered ? ends[kBins - 1] : 0};
  }
  if (filtered) {
    chunk_bins(a)[place * kBins + tid] = all;
    if (any) {                                 // their tokens, bin by bin
      uint64_t* list = chunk_tops(a) + place * kTops;
      // a lane's one after the other: few have more than four
      const int last = cut;
      uint32_t marks = 0;
#pragma unroll
      for (int k = 0; k < kSPer; ++k) marks |= bin[k] <= last ? 1u << k : 0u;
      while (marks) {
        const int k = __builtin_ctz(marks);
        marks &= marks - 1;
        const int i = i0 + (k / 4) * 4 * kSThreads + k % 4;
        const float mine = fmaxf(row[i], -INFINITY);       // (out of registers, it would be 16 selects)
        const int b = bin_of(mine, rate4, top, top_quarter);
        list[atomicAdd(&next[b], 1)] = place_of(taken(mine), i);
      }
    }
  }
  zeros();
}

// exp(chunk_top - top) in weights, the factor between the chunk's sums and the row's.
__device__ __forceinline__ double chunk_factor(const Exp2& exp2, float chunk_top, float top, double rate) {
  if (chunk_top == top) return 1.0;
  return weight(exp2, chunk_top, top, rate);
}

struct Running {                               // sums up to each bin's end
  double sum[kBins];
  int count[kBins];
};
struct PickLds {
  uint64_t arena[kArena];                      // places
  double weights[kArena];                      // of those, once they are asked for
  Running bins;
  uint64_t few[kRank], sorted[kRank];
  unsigned long long cell_sum[kBins], cell_rest[kBins];
  uint32_t cell_count[kBins];
  double waves[kDWaves];
  int found, n, first, last;
  uint32_t low;
  double kept;
};
struct ChunkShift {                            // of each chunk, in dynamic LDS
  union {
    double factor;                             // from units of its bins to weights of the row's bins; below 0: it has none
    unsigned long long kept;                   // at the end: of its kept tokens in the border's bin
  };
  int16_t shift;                               // from its bins to the row's
  int16_t cut, listed;                         // of its list
};
static_assert(sizeof(ChunkShift) == 16);

// A row at work.
struct Row {
  const float* logits;
  float top;
  double top_quarter, rate4;
  Settings s;
  ChunkStat* stats;
  const uint64_t* bins;
  const uint64_t* tops;
  ChunkShift* chunk;
  __device__ __forceinline__ int bin(float v) const { return bin_of(v, rate4, top, top_quarter); }
  __device__ __forceinline__ double weight_of(const Exp2& exp2, float v) const { return weight(exp2, v, top, s.rate); }
};

// Sum over the workgroup's lanes before this one, and of all.
__device__ __forceinline__ double block_scan_d(double v, double* lds, double& total) {
  const int wave = threadIdx.x >> 6;
  const double up = wave_scan(v);
  __syncthreads();
  if (lane_id() == kWave - 1) lds[wave] = up;
  __syncthreads();
  double before = 0.0;
  total = 0.0;
#pragma unroll
  for (int w = 0; w < kDWaves; ++w) {
    before += w < wave ? lds[w] : 0.0;
    total += lds[w];
  }
  return before + wave_before(up);
}

// First bin whose running count (k > 0) or sum reaches k or the goal; the
// last one that has tokens where rounding leaves it unreached.
__device__ __forceinline__ int crossing(const Running& up, int k, double goal, PickLds& l) {
  const int tid = threadIdx.x;
  __syncthreads();
  if (tid == 0) l.found = kBins - 1;
  __syncthreads();
  if (tid < kBins) {
    const int count = up.count[tid];
    const bool hit = count > 0 && ((k > 0 ? count >= k : up.sum[tid] >= goal) || count == up.count[kBins - 1]);
    const uint64_t hits = __ballot(hit);
    if (lane_id() == 0 && hits) atomicMin(&l.found, (tid & ~63) + __builtin_ctzll(hits));
  }
  __syncthreads();
  return l.found;
}

// Smallest key whose logit passes, of those up to `most`, which does; a wave
// for itself, 64 keys at a time.
template <class Fn>
__device__ __forceinline__ uint32_t first_key(uint32_t most, Fn passes) {
  uint64_t lo = 0, hi = most;                  // first in lo..hi
  while (lo < hi) {
    const uint64_t step = (hi - lo + kWave - 1) / kWave, at = lo + static_cast<uint64_t>(lane_id()) * step;
    const uint64_t hit = __ballot(at >= hi || passes(value_of(static_cast<uint32_t>(at < hi ? at : hi))));
    if (hit == 0) {
      lo += (kWave - 1) * step + 1;
      continue;
    }
    const int f = __builtin_ctzll(hit);
    const uint64_t up = lo + static_cast<uint64_t>(f) * step;
    if (f > 0) lo += static_cast<uint64_t>(f - 1) * step + 1;
    hi = up < hi ? up : hi;
  }
  return static_cast<uint32_t>(lo);
}

// Tokens between two places.
struct Span {
  uint64_t lo, hi;
};
__device__ __forceinline__ Span bin_span(const Row& row, int b) {
  const uint32_t most = key_of(row.top);
  const uint32_t low = first_key(most, [&](float v) QMV_INLINE { return row.bin(v) <= b; });
  const uint32_t high = b == 0 ? most : first_key(most, [&](float v) QMV_INLINE { return row.bin(v) < b; }) - 1;
  return Span{first_place(high), last_place(low)};
}

// Runs of four of the row's values, from i0 on and a step apart, -inf behind
// its end: all loads before the first use (a branch a run would wait for each).
template <int N>
__device__ __forceinline__ void load_runs(const float* row, int i0, int step, int n, float (&v)[N][4]) {
  const int first = __builtin_amdgcn_readfirstlane(i0);   // (a wave's lanes take 256 values in order)
  if (first + (N - 1) * step + 4 * kWave <= n) {
    u32x4 x[N];
#pragma unroll
    for (int q = 0; q < N; ++q) x[q] = ld_x4(reinterpret_cast<const uint8_t*>(row + i0 + q * step));
#pragma unroll
    for (int q = 0; q < N; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[q][e] = __uint_as_float(x[q][e]);
  } else {
#pragma unroll
    for (int q = 0; q < N; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + q * step + e;
        v[q][e] = row[i < n ? i : n - 1];
      }
#pragma unroll
    for (int q = 0; q < N; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[q][e] = i0 + q * step + e < n ? v[q][e] : -INFINITY;
  }
}

// f(place, value) for the row's tokens in a span, by all lanes, with eight
// loads on their way. Most are outside: their values alone tell.
template <class Fn>
__device__ __forceinline__ void each_of_row(const SampleArgs& a, const Row& row, Span g, Fn f) {
  constexpr int kAhead = 8;
  const float least = value_at(g.hi), most = value_at(g.lo);
  for (int i0 = 4 * static_cast<int>(threadIdx.x); i0 < a.vocab; i0 += 4 * kDThreads * kAhead) {
    float v[kAhead][4];
    load_runs(row.logits, i0, 4 * kDThreads, a.vocab, v);
#pragma unroll
    for (int q = 0; q < kAhead; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (v[q][e] >= least && v[q][e] <= most) {
          const float x = taken(v[q][e]);
          const uint64_t at = place_of(x, i0 + 4 * kDThreads * q + e);
          if (at >= g.lo && at <= g.hi) f(at, x);
        }
  }
}

// The row's tokens in a span (kArena at most), in the arena in any order;
// returns their number. A lane marks those of its 32 values first, so that the waves take
// their places once for all of them (one by one each token would wait for the
// one before: 47 us for 905 of 128256).
__device__ __forceinline__ int collect(const SampleArgs& a, const Row& row, Span g, PickLds& l) {
  constexpr int kAhead = 8;
  const float least = value_at(g.hi), greatest = value_at(g.lo);
  const bool inside = (g.lo & kLowIndex) != 0 || (g.hi & kLowIndex) != kLowIndex;   // an end among equal logits
  __syncthreads();
  if (threadIdx.x == 0) l.n = 0;
  __syncthreads();
  for (int i0 = 4 * static_cast<int>(threadIdx.x); i0 - 4 * static_cast<int>(threadIdx.x) < a.vocab; i0 += 4 * kDThreads * kAhead) {
    float v[kAhead][4];
    load_runs(row.logits, i0, 4 * kDThreads, a.vocab, v);
    uint32_t marks = 0;
#pragma unroll
    for (int q = 0; q < kAhead; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) marks |= v[q][e] >= least && v[q][e] <= greatest ? 1u << (4 * q + e) : 0u;
    if (inside) {                              // uniform
#pragma unroll
      for (int q = 0; q < kAhead; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t at = place_of(taken(v[q][e]), i0 + 4 * kDThreads * q + e);
          marks &= at < g.lo || at > g.hi ? ~(1u << (4 * q + e)) : ~0u;
        }
    }
    const int hits = __builtin_popcount(marks), up = wave_scan(hits), all = __builtin_amdgcn_readlane(up, kWave - 1);
    if (all == 0) continue;
    int first = 0;
    if (lane_id() == 0) first = atomicAdd(&l.n, all);
    int to = __builtin_amdgcn_readfirstlane(first) + up - hits;
#pragma unroll
    for (int q = 0; q < kAhead; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (marks >> (4 * q + e) & 1) {
          if (to < kArena) l.arena[to] = place_of(taken(v[q][e]), i0 + 4 * kDThreads * q + e);
          ++to;
        }
  }
  __syncthreads();
  return l.n < kArena ? l.n : kArena;
}

// Sorted into `to`, ascending: each goes to the number of those before it.
__device__ __forceinline__ void sort_few(const uint64_t* list, uint64_t* to, int n, PickLds& l) {
  const int tid = threadIdx.x;
  int wide = kWave;
  while (wide < n) wide <<= 1;
  const int parts = kDThreads / wide, part = tid / wide, i = tid & (wide - 1), per = (n + parts - 1) / parts;
  __syncthreads();
  if (tid < kRank) l.cell_count[tid] = 0;
  const uint64_t mine = i < n ? list[i] : 0;
  const int end = (part + 1) * per < n ? (part + 1) * per : n;
  int before = 0;
#pragma unroll 4
  for (int j = part * per; j < end; ++j) before += list[j] < mine;
  __syncthreads();
  if (i < n && before) atomicAdd(&l.cell_count[i], static_cast<uint32_t>(before));
  __syncthreads();
  if (part == 0 && i < n) to[l.cell_count[i]] = mine;
  __syncthreads();
}

// Running sums of kHalf of the row's bins from `first` on: of the chunks' bins,
// each moved to the row's grid. Most borders lie in the first half (32
// octaves), and the other is not read then. A wave takes every eighth chunk, a
// lane two bins. all, tokens: sum and number of all, where the last bin ends.
constexpr int kHalf = 2 * kWave;
__device__ __forceinline__ void join_half(const SampleArgs& a, const Row& row, int half, double all, int tokens, PickLds& l) {
  // chunks of a wave on their way: 40 of all eight, 163840 logits, in one round
  // (3 or 8: 64 rows of 128256 with all filters 34.7 -> 35.0 and 35.5 us; 1 row of
  // 200064, two rounds, 21.1, with 3 20.8)
  constexpr int kAhead = 5;
  const int wave = threadIdx.x >> 6, lane = lane_id();
  double sum[2] = {0.0, 0.0};
  int count[2] = {0, 0};
  for (int c0 = wave; c0 < a.chunks; c0 += kDWaves * kAhead) {
    uint64_t x[kAhead][2];
#pragma unroll
    for (int q = 0; q < kAhead; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = c0 + kDWaves * q < a.chunks ? c0 + kDWaves * q : c0, from = half * kHalf + e * kWave + lane - row.chunk[c].shift;
        x[q][e] = row.bins[static_cast<int64_t>(c) * kBins + (from > 0 ? from : 0)];
      }
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int c = c0 + kDWaves * q;
      if (c >= a.chunks) continue;             // uniform
      const ChunkShift h = row.chunk[c];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (h.factor >= 0.0 && half * kHalf + e * kWave + lane >= h.shift) {
          sum[e] = fma(bin_units(x[q][e]), h.factor, sum[e]);
          count[e] += static_cast<int>(x[q][e] >> kSumBits);
        }
    }
  }
  double* sums = reinterpret_cast<double*>(l.arena);
  int* counts = reinterpret_cast<int*>(l.arena + kDWaves * kHalf);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    sums[wave * kHalf + e * kWave + lane] = sum[e];
    counts[wave * kHalf + e * kWave + lane] = count[e];
  }
  __syncthreads();
  if (wave == 0) {
    double run = half ? l.bins.sum[kHalf - 1] : 0.0;
    int run_count = half ? l.bins.count[kHalf - 1] : 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = e * kWave + lane, bin = half * kHalf + i;
      double one = 0.0;
      int n = 0;
#pragma unroll
      for (int w = 0; w < kDWaves; ++w) {
        one += sums[w * kHalf + i];
        n += counts[w * kHalf + i];
      }
      one = wave_scan(one * bin_scale(bin)) + run;
      n = wave_scan(n) + run_count;
      l.bins.sum[bin] = bin == kBins - 1 ? all : one;
      l.bins.count[bin] = bin == kBins - 1 ? tokens : n;
      run = __shfl(one, kWave - 1);
      run_count = __builtin_amdgcn_readlane(n, kWave - 1);
    }
  }
  __syncthreads();
}

// First bin of the first half whose running count (k > 0) or sum reaches k or
// the goal, kHalf where none does; every wave for itself.
__device__ __forceinline__ int crossing_near(const Running& up, int k, double goal) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = e * kWave + lane_id(), count = up.count[i];
    const uint64_t hits = __ballot(count > 0 && (k > 0 ? count >= k : up.sum[i] >= goal));
    if (hits) return e * kWave + __builtin_ctzll(hits);
  }
  return kHalf;
}

// The tokens of bins from..b (kArena at most) from the chunks' lists, in the
// arena. Returns their number, -1 where a chunk lists fewer.
__device__ __forceinline__ int gather(const SampleArgs& a, const Row& row, int from, int b, PickLds& l) {
  constexpr int kAhead = 5;                    // lists on their way, as in join_half
  const int tid = threadIdx.x, wave = tid >> 6;
  bool covered = true;
  for (int c = tid; c < a.chunks; c += kDThreads) {
    const ChunkShift h = row.chunk[c];
    if (h.factor >= 0.0 && h.cut < kBins - 1 && (b == kBins - 1 || h.cut + h.shift < b)) covered = false;
  }
  __syncthreads();
  if (tid == 0) l.n = 0;
  if (!__syncthreads_and(covered)) return -1;
  for (int c0 = wave; c0 < a.chunks; c0 += kDWaves * kAhead) {
    uint64_t x[kAhead];
    const auto entry = [&](int c, int i) QMV_INLINE { return row.tops[static_cast<int64_t>(c) * kTops + i]; };
#pragma unroll
    for (int q = 0; q < kAhead; ++q) x[q] = entry(c0 + kDWaves * q < a.chunks ? c0 + kDWaves * q : c0, lane_id());
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int c = c0 + kDWaves * q;
      if (c >= a.chunks) continue;             // uniform
      const ChunkShift h = row.chunk[c];
      // (a chunk from kBins on has all its tokens in the row's last bin)
      const int listed = h.factor >= 0.0 && (h.shift <= b || b == kBins - 1) ? h.listed : 0;
      for (int i = lane_id(), more = listed; more > 0; more -= kWave, i += kWave) {
        if (i != lane_id()) x[q] = i < listed ? entry(c, i) : 0;
        const int its = i < listed ? row.bin(value_at(x[q])) : kBins;
        const bool in = its >= from && its <= b;
        const uint64_t ins = __ballot(in);
        if (ins) {
          int first = 0;
          if (lane_id() == 0) first = atomicAdd(&l.n, __builtin_popcountll(ins));
          const int at = __builtin_amdgcn_readfirstlane(first) + __builtin_popcountll(ins & ((uint64_t(1) << lane_id()) - 1));
          if (in && at < kArena) l.arena[at] = x[q];
        }
        if (__ballot(its > b)) break;          // the list goes bin by bin
      }
    }
  }
  __syncthreads();
  return l.n < kArena ? l.n : kArena;
}

// Whole units of a weight up to 1, as the low bits of a sum with 2^52.
__device__ __forceinline__ unsigned long long units_of(double w, int unit) {
  return static_cast<unsigned long long>(__double_as_longlong(__builtin_ldexp(w, unit) + 0x1p52)) & ((1ull << 52) - 1);
}

// The weights of the arena's n tokens, and the key of the lowest.
__device__ __forceinline__ void weigh(const Exp2& exp2, const Row& row, int n, PickLds& l) {
  constexpr int kAhead = 4;
  uint32_t low = 0xFFFFFFFFu;
  __syncthreads();
  if (threadIdx.x == 0) l.low = 0xFFFFFFFFu;
  __syncthreads();
  for (int i0 = threadIdx.x; i0 < n; i0 += kDThreads * kAhead) {
    double w[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int i = i0 + kDThreads * q;
      const float v = value_at(l.arena[i < n ? i : i0]);
      w[q] = row.weight_of(exp2, v);
      low = key_of(v) < low ? key_of(v) : low;
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q)
      if (i0 + kDThreads * q < n) l.weights[i0 + kDThreads * q] = w[q];
  }
  for (int mask = kWave / 2; mask > 0; mask >>= 1) {
    const uint32_t other = static_cast<uint32_t>(__shfl_xor(static_cast<int>(low), mask));
    low = other < low ? other : low;
  }
  if (lane_id() == 0) atomicMin(&l.low, low);
  __syncthreads();
}

// Cells of tokens: their sums in units, and their number.
__device__ __forceinline__ void clear_cells(PickLds& l) {
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kDThreads) {
    l.cell_sum[i] = 0;
    l.cell_rest[i] = 0;
    l.cell_count[i] = 0;
  }
  __syncthreads();
}
__device__ __forceinline__ void add_to_cell(PickLds& l, int cell, unsigned long long units) {
  atomicAdd(&l.cell_sum[cell], units);
  atomicAdd(&l.cell_count[cell], 1u);
}
// For the draw: weights up to 2^scale (larger ones count as that) in whole
// units of 2^(scale - kFine) and what is left in units of 2^(scale - 2 kFine),
// so that sums in any order are those of 64 bits. The arena's 2^13 tokens at
// most stay below 2^62 of either.
constexpr int kFine = 49;
__device__ __forceinline__ void add_weight(PickLds& l, int cell, double w, int scale) {
  const double x = fmin(__builtin_ldexp(w, kFine - scale), 0x1p49), whole = floor(x);
  add_to_cell(l, cell, units_of(whole, 0));
  atomicAdd(&l.cell_rest[cell], units_of(x - whole, kFine));
}
static_assert(kFine == 49 && kArena <= 1 << 13);
struct CellFound {
  int cell, count, ahead;                      // tokens in it and before it
  double passed, total;                        // weight before it, and of all
};
// The first cell that hit(running sum, running count) holds for, the last one
// that has a weight (by_weight, of add_weight) or tokens where it holds for
// none. Every wave for itself, so that nothing has to be handed on.
template <class Hit>
__device__ __forceinline__ CellFound find_cell(const PickLds& l, int unit, bool by_weight, Hit hit) {
  constexpr int kPer = kBins / kWave;
  double sum[kPer], own = 0.0;
  int count[kPer], own_count = 0;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    sum[e] = __builtin_ldexp(static_cast<double>(l.cell_sum[kPer * lane_id() + e]), -unit);
    if (by_weight) sum[e] += __builtin_ldexp(static_cast<double>(l.cell_rest[kPer * lane_id() + e]), -unit - kFine);
    count[e] = static_cast<int>(l.cell_count[kPer * lane_id() + e]);
    own += sum[e];
    own_count += count[e];
  }
  const double up = wave_scan(own), start = wave_before(up);
  const int up_count = wave_scan(own_count), start_count = up_count - own_count;
  double run = start;
  int run_count = start_count, first = kPer, last = -1;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    run += sum[e];
    run_count += count[e];
    const bool some = by_weight ? sum[e] > 0.0 : count[e] > 0;
    first = first == kPer && some && hit(run, run_count) ? e : first;
    last = some ? e : last;
  }
  const uint64_t hits = __ballot(first < kPer), somes = __ballot(last >= 0);
  const int lane = hits ? __builtin_ctzll(hits) : somes ? 63 - __builtin_clzll(somes) : 0;
  const int e = __builtin_amdgcn_readlane(hits ? first : last < 0 ? 0 : last, lane);
  CellFound f;
  f.cell = kPer * lane + e;
  double passed = start;
  int ahead = start_count, mine = count[0];
#pragma unroll
  for (int i = 0; i < kPer - 1; ++i) {
    passed += i < e ? sum[i] : 0.0;
    ahead += i < e ? count[i] : 0;
    mine = i + 1 == e ? count[i + 1] : mine;
  }
  f.passed = __shfl(passed, lane);
  f.ahead = __builtin_amdgcn_readlane(ahead, lane);
  f.count = __builtin_amdgcn_readlane(mine, lane);
  f.total = __shfl(up, kWave - 1);
  return f;
}

// Where the border of a filter is looked for: `count` tokens, behind `ahead`
// others of the weight `passed`; n of them, all, are in the arena (-1: not yet).
struct Search {
  Span g;
  int count, ahead, n;
  double passed;
  bool weighed;
};

// The last place kept by top-k (k > 0: the k-th token) or by top-p (the last
// before which less than `goal` has passed); kept: the weight up to it. The
// span is cut into cells of equal width until few tokens are left in one. On
// return s.n tells whether all its tokens are in the arena.
__device__ __forceinline__ uint64_t find_border(const SampleArgs& a, const Exp2& exp2, const Row& row, Search& s, int k, double goal, PickLds& l,
                                                double& kept) {
  const int tid = threadIdx.x, whole = s.count;
  Span g = s.g;
  int count = s.count, ahead = s.ahead, n = s.n;
  double passed = s.passed;
  bool weighed = s.weighed;
#pragma unroll 1
  while (true) {
    if (n < 0 && count <= kArena) n = collect(a, row, g, l);
    if (count <= kRank) break;
    if (n >= 0 && !weighed) {
      weigh(exp2, row, n, l);
      weighed = true;
    }
    const uint64_t wide = g.hi - g.lo;
    const int bits = 64 - __builtin_clzll(wide | 1), shift = bits > 8 ? bits - 8 : 0;   // at most kBins cells
    // 2^24 tokens at most, none above the weight of the first place
    int most;
    (void)__builtin_frexp(row.weight_of(exp2, value_at(g.lo)), &most);
    const int unit = kUnit - most;
    clear_cells(l);
    if (n >= 0) {
      for (int i = tid; i < n; i += kDThreads) {
        const uint64_t at = l.arena[i];
        if (at >= g.lo && at <= g.hi) add_to_cell(l, static_cast<int>((at - g.lo) >> shift), units_of(l.weights[i], unit));
      }
    } else {
      each_of_row(a, row, g, [&](uint64_t at, float v) QMV_INLINE {
        add_to_cell(l, static_cast<int>((at - g.lo) >> shift), units_of(row.weight_of(exp2, v), unit));
      });
    }
    __syncthreads();
    const CellFound f = find_cell(l, unit, false, [&](double sum, int tokens) QMV_INLINE {
      return k > 0 ? ahead + tokens >= k : passed + sum >= goal;
    });
    g.lo += static_cast<uint64_t>(f.cell) << shift;
    const uint64_t end = g.lo + ((uint64_t(1) << shift) - 1);
    g.hi = end < g.hi ? end : g.hi;
    passed += f.passed;
    ahead += f.ahead;
    count = f.count;
  }
  s.n = n == whole ? n : -1;
  s.weighed = weighed;
  // the few, sorted
  __syncthreads();
  if (tid == 0) l.n = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kDThreads) {
    const uint64_t at = l.arena[i];
    if (at >= g.lo && at <= g.hi) {
      const int to = atomicAdd(&l.n, 1);
      if (to < kRank) l.few[to] = at;
    }
  }
  __syncthreads();
  const int m = l.n < kRank ? l.n : kRank;
  sort_few(l.few, l.sorted, m, l);
  const uint64_t mine = tid < m ? l.sorted[tid] : 0;
  const double w = tid < m ? row.weight_of(exp2, value_at(mine)) : 0.0;
  double total;
  const double before = passed + block_scan_d(w, l.waves, total);
  if (tid == 0) l.last = 0;
  __syncthreads();
  const uint64_t ins = __ballot(tid < m && (k > 0 ? ahead + tid < k : before < goal));
  if (lane_id() == 0 && ins) atomicMax(&l.last, (tid & ~63) + 63 - __builtin_clzll(ins));
  __syncthreads();
  const int last = l.last;                     // the first one in any case
  if (tid == last) l.kept = before + w;
  __syncthreads();
  kept = l.kept;
  return l.sorted[last];
}

// Where a row's draw stands.
struct Drawn {
  uint64_t border;
  double total, chosen;
  int token;
};

// All `count` tokens (kRank at most) up to the border's bin, in the arena:
// sorted, cut by all filters, and drawn from. all: the sum of the row's weights;
// probs: where the kept ones' probabilities go, if anywhere.
__device__ __forceinline__ Drawn draw_short(const Exp2& exp2, const Row& row, int count, double all, float u, float* probs, PickLds& l) {
  const int tid = threadIdx.x;
  const Settings& s = row.s;
  uint64_t* sorted = l.sorted;
  double* weights = l.weights;
  sort_few(l.arena, sorted, count, l);
  const int k = s.k > 0 && s.k < count ? s.k : count;
  const uint64_t at = tid < k ? sorted[tid] : 0;
  double w = tid < k ? row.weight_of(exp2, value_at(at)) : 0.0, total;
  const double before = block_scan_d(w, l.waves, total), goal = s.p * (s.k > 0 ? total : all);
  if (tid == 0) {
    l.last = 0;
    l.first = 0x7fffffff;
    l.found = -1;
  }
  __syncthreads();
  const uint64_t ins = __ballot(tid < k && (s.p >= 1.0 || before < goal) && w >= s.m);
  if (ins && lane_id() == 0) atomicMax(&l.last, (tid & ~63) + 63 - __builtin_clzll(ins));
  __syncthreads();
  const int last = l.last;                     // the first token is kept in any case
  Drawn d;
  d.border = sorted[last];
  // the kept ones by their indices
  if (tid <= last) {
    weights[tid] = w;
    l.arena[tid] = (at & kLowIndex) << 12 | static_cast<uint64_t>(tid);
  }
  __syncthreads();                             // (the border is read)
  sort_few(l.arena, sorted, last + 1, l);
  const uint64_t x = tid <= last ? sorted[tid] : 0;
  w = tid <= last ? weights[x & 4095] : 0.0;
  const double up = block_scan_d(w, l.waves, d.total) + w;
  if (probs && tid <= last) probs[x >> 12] = static_cast<float>(w / d.total);
  const uint64_t hits = __ballot(w > 0.0 && up > static_cast<double>(u) * d.total), some = __ballot(w > 0.0);
  if (hits && lane_id() == 0) atomicMin(&l.first, (tid & ~63) + __builtin_ctzll(hits));
  if (some && lane_id() == 0) atomicMax(&l.found, (tid & ~63) + 63 - __builtin_clzll(some));
  __syncthreads();
  const uint64_t take = sorted[l.first != 0x7fffffff ? l.first : l.found];
  d.token = static_cast<int>(take >> 12);
  d.chosen = weights[take & 4095] / d.total;
  return d;
}

// The same of at most 64 tokens, by one wave: each lane has a token.
__device__ __forceinline__ Drawn draw_wave(const Exp2& exp2, const Row& row, int count, double all, float u, float* probs, uint64_t* list) {
  const Settings& s = row.s;
  const int lane = lane_id();
  const auto sorted = [&](uint64_t mine, int n) QMV_INLINE {   // the lane's of n in list
    int before = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) before += list[j] < mine;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (lane < n) list[before] = mine;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    return lane < n ? list[lane] : 0;
  };
  const uint64_t at = sorted(lane < count ? list[lane] : 0, count);
  const int k = s.k > 0 && s.k < count ? s.k : count;
  double w = lane < k ? row.weight_of(exp2, value_at(at)) : 0.0;
  double up = wave_scan(w);
  const double goal = s.p * (s.k > 0 ? __shfl(up, kWave - 1) : all);
  const uint64_t ins = __ballot(lane < k && (s.p >= 1.0 || up - w < goal) && w >= s.m) | 1;   // the first in any case
  const int last = 63 - __builtin_clzll(ins);
  Drawn d;
  d.border = __shfl(at, last);
  // the kept ones by their indices
  const uint64_t mine = lane <= last ? (at & kLowIndex) << 6 | static_cast<uint64_t>(lane) : 0;
  if (lane <= last) list[lane] = mine;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  const uint64_t x = sorted(mine, last + 1);
  w = __shfl(w, static_cast<int>(x & 63));
  w = lane <= last ? w : 0.0;
  up = wave_scan(w);
  d.total = __shfl(up, kWave - 1);
  const uint64_t hits = __ballot(w > 0.0 && up > static_cast<double>(u) * d.total), some = __ballot(w > 0.0);
  const int take = hits ? __builtin_ctzll(hits) : 63 - __builtin_clzll(some);
  const double p = w / d.total;
  if (probs && lane <= last) probs[x >> 6] = static_cast<float>(p);
  d.token = static_cast<int>(__shfl(x, take) >> 6);
  d.chosen = __shfl(p, take);
  return d;
}

// The border by all filters. listed: tokens in the arena, all up to the border
// (0: none there); else of: the bin whose tokens are there in the end, -1 for none.
__device__ __forceinline__ uint64_t far_border(const SampleArgs& a, const Exp2& exp2, const Row& row, double all, int tokens, int listed, int& of,
                                               int& of_listed, PickLds& l) {
  const Settings& s = row.s;
  uint64_t border = ~uint64_t(0);
  of = -1;
  of_listed = 0;
  double total = all;
#pragma unroll 1
  for (int turn = 0; turn < 2; ++turn) {       // top-k, then top-p
    if (turn == 0 ? s.k == 0 || s.k >= tokens : s.p >= 1.0) continue;   // uniform
    const int k = turn == 0 ? s.k : 0;
    const double goal = s.p * total;
    Search search{Span{first_place(key_of(row.top)), last_place(l.low)}, listed, 0, listed, 0.0, listed > 0};
    if (listed == 0) {
      of = crossing(l.bins, k, goal, l);
      const int ahead = of > 0 ? l.bins.count[of - 1] : 0, count = l.bins.count[of] - ahead;
      const double passed = of > 0 ? l.bins.sum[of - 1] : 0.0;
      search = Search{bin_span(row, of), count, ahead, count <= kArena ? gather(a, row, of, of, l) : -1, passed, false};
    }
    double kept;
    const uint64_t found = find_border(a, exp2, row, search, k, goal, l, kept);
    of_listed = search.n;
    if (turn == 0) total = kept;
    border = found < border ? found : border;
    __syncthreads();
  }
  if (s.m > 0.0) {                             // every wave for itself
    const uint64_t least =
        last_place(first_key(key_of(row.top), [&](float v) QMV_INLINE { return row.weight_of(exp2, v) >= s.m; }));
    border = least < border ? least : border;
  }
  return border;
}

// A draw from the arena's n tokens up to the border: their weights summed over
// cells of indices, until few are left in the one in which the running sum
// passes the goal. Against a goal far below the largest weight (u = 0, above
// all) they are summed again, in units of the goal's size: a token that weighs
// more passes it, however much more.
__device__ __forceinline__ Drawn draw_list(const Exp2& exp2, const Row& row, int n, uint64_t border, int vocab, float u, float* probs, PickLds& l) {
  constexpr int kLeast = -1000;                // 2^-1074, the smallest weight, is a number of its units
  const int tid = threadIdx.x;
  Drawn d{border, 0.0, 0.0, -1};
  int lo = 0, shift = 32 - __builtin_clz(static_cast<uint32_t>(vocab)) - 8;
  shift = shift > 0 ? shift : 0;
  double passed = 0.0, drawn = 0.0;
  int scale = 0;
  bool known = false;
#pragma unroll 1
  while (true) {
    clear_cells(l);
    for (int i = tid; i < n; i += kDThreads) {
      const uint64_t at = l.arena[i];
      const int index = static_cast<int>(at & kLowIndex) - lo;
      if (at <= border && index >= 0 && index >> shift < kBins) add_weight(l, index >> shift, l.weights[i], scale);
    }
    __syncthreads();
    const auto passes = [&](double sum, int) QMV_INLINE { return known && passed + sum > drawn; };
    CellFound f = find_cell(l, kFine - scale, true, passes);
    if (!known) {                              // the first time: the number goes by the sum
      known = true;
      d.total = f.total;
      drawn = static_cast<double>(u) * d.total;
      if (drawn < 0x1p-32) {
        scale = kLeast;
        if (drawn > 0x1p-999) (void)__builtin_frexp(drawn, &scale);
        continue;
      }
      f = find_cell(l, kFine, true, passes);
    }
    lo += f.cell << shift;
    passed += f.passed;
    if (f.count <= kRank) break;               // (a cell of one index has one)
    shift = shift > 8 ? shift - 8 : 0;
  }
  // the few by their indices
  __syncthreads();
  if (tid == 0) {
    l.n = 0;
    l.first = kRank;
    l.last = 0;
  }
  __syncthreads();
  const double share = 1.0 / d.total;
  for (int i = tid; i < n; i += kDThreads) {
    const uint64_t at = l.arena[i];
    const int index = static_cast<int>(at & kLowIndex) - lo;
    if (at <= border) {
      if (probs) probs[at & kLowIndex] = static_cast<float>(l.weights[i] * share);
      if (index >= 0 && index >> shift == 0) {
        const int to = atomicAdd(&l.n, 1);
        if (to < kRank) l.few[to] = (at & kLowIndex) << 32 | static_cast<uint64_t>(i);
      }
    }
  }
  __syncthreads();
  const int m = l.n < kRank ? l.n : kRank;
  sort_few(l.few, l.sorted, m, l);
  const uint64_t x = tid < m ? l.sorted[tid] : 0;
  const double w = tid < m ? l.weights[x & 0xFFFFFFFFu] : 0.0;
  double all;
  const double up = passed + block_scan_d(w, l.waves, all) + w;
  const uint64_t hits = __ballot(w > 0.0 && up > drawn), some = __ballot(w > 0.0);
  if (hits && lane_id() == 0) atomicMin(&l.first, (tid & ~63) + __builtin_ctzll(hits));
  if (some && lane_id() == 0) atomicMax(&l.last, (tid & ~63) + 63 - __builtin_clzll(some));
  __syncthreads();
  const uint64_t take = l.sorted[l.first < kRank ? l.first : l.last];
  d.token = static_cast<int>(take >> 32);
  d.chosen = l.weights[take & 0xFFFFFFFFu] / d.total;
  return d;
}

// The kept weights of each chunk, in its stats. From the bins they are good to
// 2^-38 of each weight. (Always from the row itself, in 64 bits: 64 rows of top-p
// 57 -> 84 us, 128 with distributions 102 -> 142.)
__device__ __forceinline__ void kept_sums(const SampleArgs& a, const Exp2& exp2, const Row& row, uint64_t border, int listed, int of, PickLds& l) {
  const int tid = threadIdx.x, wave = tid >> 6;
  if (border == ~uint64_t(0)) {
    for (int c = tid; c < a.chunks; c += kDThreads) row.stats[c].sum *= chunk_factor(exp2, row.stats[c].top, row.top, row.s.rate);
    __syncthreads();
    return;
  }
  const int b = row.bin(value_at(border)), count = l.bins.count[b] - (b > 0 ? l.bins.count[b - 1] : 0);
  // no list of that bin: the row again; also for the last bin, whose weights are
  // too unlike for its units (a chunk that has no others would count as without weight)
  if (of != b || listed != count || b == kBins - 1) {
    for (int c = wave; c < a.chunks; c += kDWaves) {
      double sum = 0.0;
#pragma unroll 1
      for (int j = 0; j < kChunk / (4 * kWave); j += 4) {
        const int i0 = c * kChunk + 4 * (j * kWave + lane_id());
        float v[4][4];
        load_runs(row.logits, i0, 4 * kWave, a.vocab, v);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = taken(v[q][e]);
            if (place_of(x, i0 + 4 * kWave * q + e) <= border) sum += row.weight_of(exp2, x);
          }
      }
      sum = wave_sum(sum);
      if (lane_id() == 0) row.stats[c].sum = sum;
    }
    __syncthreads();
    return;
  }
  // the bins before the border's, and the tokens in that
  for (int c = wave; c < a.chunks; c += kDWaves) {
    const ChunkShift h = row.chunk[c];
    double sum = 0.0;
    if (h.factor >= 0.0) {
#pragma unroll
      for (int j = 0; j < kBins / kWave; ++j) {
        const int at = j * kWave + lane_id();
        const uint64_t x = row.bins[static_cast<int64_t>(c) * kBins + at];
        sum += at + h.shift < b ? bin_units(x) * bin_scale(at + h.shift) : 0.0;
      }
      sum = wave_sum(sum) * h.factor;
    }
    if (lane_id() == 0) row.stats[c].sum = sum;
  }
  __syncthreads();
  for (int c = tid; c < a.chunks; c += kDThreads) row.chunk[c].kept = 0;
  __syncthreads();
  for (int i = tid; i < listed; i += kDThreads) {
    const uint64_t at = l.arena[i];
    if (at <= border) {
      const double w = __builtin_ldexp(row.weight_of(exp2, value_at(at)), kUnit + (b >> 2)) + 0x1p52;
      atomicAdd(&row.chunk[(at & kLowIndex) / kChunk].kept, static_cast<unsigned long long>(__double_as_longlong(w) & ((1ll << 52) - 1)));
    }
  }
  __syncthreads();
  for (int c = tid; c < a.chunks; c += kDThreads)
    row.stats[c].sum += __builtin_ldexp(static_cast<double>(row.chunk[c].kept), -(kUnit + (b >> 2)));
  __syncthreads();
}

// A draw by the chunks' kept weights: the chunk in which the running sum
// passes the goal, then its element.
__device__ __forceinline__ Drawn draw_long(const SampleArgs& a, const Exp2& exp2, const Row& row, uint64_t border, float u, PickLds& l) {
  constexpr int kPer = kChunk / kDThreads;
  const int tid = threadIdx.x;
  const ChunkStat* st = row.stats;
  Drawn d{border, 0.0, 0.0, -1};
  double sum = 0.0;
  for (int c = lane_id(); c < a.chunks; c += kWave) sum += st[c].sum;
  d.total = wave_sum(sum);
  if (!a.tokens && !a.chosen) return d;
  const double goal = static_cast<double>(u) * d.total;
  double run = 0.0, before = 0.0, last_before = 0.0;
  int found = -1, last = 0;
  for (int c0 = 0; c0 < a.chunks && found < 0; c0 += kWave) {
    const int c = c0 + lane_id();
    const double w = c < a.chunks ? st[c].sum : 0.0, sums = wave_scan(w), up = sums + run, ahead = wave_before(sums) + run;
    // (a chunk without weight may have the larger sum by rounding alone: the scan adds in another order at each lane)
    const uint64_t hit = __ballot(w > 0.0 && up > goal), some = __ballot(w > 0.0);
    if (some) {
      const int i = 63 - __builtin_clzll(some);
      last = c0 + i;
      last_before = __shfl(ahead, i);
    }
    if (hit) {
      const int i = __builtin_ctzll(hit);
      found = c0 + i;
      before = __shfl(ahead, i);
    }
    run = __shfl(up, kWave - 1);
  }
  const int c = found >= 0 ? found : last;
  if (found < 0) before = last_before;
  // its elements, a run of eight a lane
  const int i0 = c * kChunk + kPer * tid;
  float v[kPer];
  double w[kPer], own = 0.0, all;
#pragma unroll
  for (int q = 0; q < kPer; q += 4) {
    float four[4];
    load_quad(row.logits, i0 + q, a.vocab, -INFINITY, four);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[q + e] = taken(four[e]);
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    w[e] = place_of(v[e], i0 + e) <= border ? row.weight_of(exp2, v[e]) : 0.0;
    own += w[e];
  }
  double up = before + block_scan_d(own, l.waves, all);
  if (tid == 0) {
    l.first = 0x7fffffff;
    l.found = -1;
  }
  __syncthreads();
  int hit = 0x7fffffff, some = -1;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    up += w[e];
    if (w[e] > 0.0) {
      some = i0 + e;
      if (up > goal && hit == 0x7fffffff) hit = i0 + e;
    }
  }
  if (hit != 0x7fffffff) atomicMin(&l.first, hit);
  if (some >= 0) atomicMax(&l.found, some);
  __syncthreads();
  d.token = l.first != 0x7fffffff ? l.first : l.found;
  if (d.token >= 0) d.chosen = row.weight_of(exp2, taken(row.logits[d.token])) / d.total;
  return d;
}

// A chain of latencies: the chunks' tops, their bins, the crossing, the lists,
// ranks, a scan. Over 128256 logits: 10 us for a row with few tokens up to its
// border's bin, 17 for 64 rows of mixed filters, 36 for 128 rows of top-p where the
// slowest has thousands (weights, cells and barriers in LDS), 60 where it has to be
// read again, which one workgroup does in 23 us (22 GB/s); 160 where the border's
// bin alone has more than kArena (temperature 2, top-p 0.95) and it is read more than
// once. A wave has the registers of two a SIMD: with 1024 threads a call of 128 rows
// takes 76 us for 63.
__global__ void __launch_bounds__(kDThreads) sample_pick_kernel(SampleArgs a) {
  __shared__ PickLds l;
  extern __shared__ __align__(16) uint8_t dynamic[];
  const Exp2 exp2;
  const int tid = threadIdx.x, r = blockIdx.x;
  Row row;
  row.s = settings_of(a, r);
  row.logits = a.logits + r * a.ldl;
  row.stats = chunk_stats(a) + static_cast<int64_t>(r) * a.chunks;
  row.bins = chunk_bins(a) + static_cast<int64_t>(r) * a.chunks * kBins;
  row.tops = chunk_tops(a) + static_cast<int64_t>(r) * a.chunks * kTops;
  row.chunk = reinterpret_cast<ChunkShift*>(dynamic);
  row.rate4 = 4.0 * row.s.rate;
  const float u = a.u ? a.u[r] : 0.0f;
  float top = -INFINITY;
  int at = 0x7fffffff;
  if (!row.s.none) {
    for (int c = lane_id(); c < a.chunks; c += kWave) take_top(top, at, row.stats[c].top, row.stats[c].at);
    wave_top(top, at);
    top = taken(top);
  }
  row.top = top;
  row.top_quarter = quarter(top, row.rate4);
  Drawn d{0, 0.0, 0.0, -1};
  float* probs = a.zeroed ? a.probs + r * a.ldp : nullptr;
  bool written = a.zeroed && !row.s.plain();   // else the last launch writes the distribution
  if (top == -INFINITY) {                      // uniform
  } else if (row.s.greedy) {
    d = Drawn{place_of(top, at), 1.0, 1.0, at};
    if (probs && tid == 0) probs[at] = 1.0f;
  } else if (!row.s.filtered()) {
    kept_sums(a, exp2, row, ~uint64_t(0), 0, -1, l);
    d = draw_long(a, exp2, row, ~uint64_t(0), u, l);
  } else {
    double all = 0.0;                          // of the weights, in every wave
    int tokens = 0;
    for (int c = lane_id(); c < a.chunks; c += kWave) {
      const ChunkStat st = row.stats[c];
      const bool has = st.top > -INFINITY && (top < INFINITY || st.top == top);
      const double factor = has ? chunk_factor(exp2, st.top, top, row.s.rate) : 0.0;
      all += st.sum * factor;
      tokens += has ? st.tokens : 0;
      if (tid < kWave) {
        ChunkShift h;
        const int shift = has && top < INFINITY ? bins_between(row.top_quarter, quarter(st.top, row.rate4), kBins) : 0;
        h.factor = has ? __builtin_ldexp(factor, -kUnit) * bin_scale(-shift) : -1.0;
        h.shift = static_cast<int16_t>(shift);
        h.cut = st.cut;
        h.listed = st.listed;
        row.chunk[c] = h;
      }
    }
    all = wave_sum(all);
    tokens = __builtin_amdgcn_readlane(wave_scan(tokens), kWave - 1);
    __syncthreads();
    // the last bin that can hold the border
    const bool by_weight = row.s.m > 0.0 && (row.s.k == 0 || row.s.p >= 1.0);   // (top-p needs the sum of all k)
    // w >= m ends in the bin of 4 log2(m), to one by rounding, behind the top's
    const int end = by_weight ? static_cast<int>(fmin(4.0 * -log2(row.s.m) + 2.0, kBins - 1.0)) : kBins - 1;
    const bool by_place = row.s.k > 0 || row.s.p < 1.0;
    int b = end, n = -1;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      join_half(a, row, half, all, tokens, l);
      if (half) b = by_place ? crossing(l.bins, row.s.k, row.s.p * all, l) : kBins - 1;
      else b = by_place ? crossing_near(l.bins, row.s.k, row.s.p * all) : kHalf;
      b = b < end ? b : end;
      if (b < kHalf * (half + 1) && l.bins.count[b] <= kArena) {
        n = gather(a, row, 0, b, l);
        if (n >= 0) break;
      }
    }
    if (n >= 0 && n <= kWave) {                // uniform
      if (tid < kWave) d = draw_wave(exp2, row, n, all, u, probs, l.arena);
    } else if (n >= 0 && n <= kRank) {
      d = draw_short(exp2, row, n, all, u, probs, l);
    } else {
      int of, of_listed;
      if (n > 0) weigh(exp2, row, n, l);
      const uint64_t border = far_border(a, exp2, row, all, tokens, n > 0 ? n : 0, of, of_listed, l);
      if (n > 0) {
        d = draw_list(exp2, row, n, border, a.vocab, u, probs, l);
      } else {
        written = false;
        kept_sums(a, exp2, row, border, of_listed, of, l);
        d = draw_long(a, exp2, row, border, u, l);
      }
    }
  }
  if (tid == 0) {
    if (a.tokens) a.tokens[r] = d.token;
    if (a.chosen) a.chosen[r] = static_cast<float>(d.chosen);
    if (a.probs) picks(a)[r] = Pick{d.border, d.total, row.s.rate, top, written};
  }
}

// Reads and writes every logit's place: 64 plain rows of 128256 take 16 us more
// with their distributions than without (66 MB, 4.1 TB/s).
__global__ void __launch_bounds__(kSThreads) sample_probs_kernel(SampleArgs a) {
  const Exp2 exp2;
  const int r = row_of_grid();
  if (r >= a.n_rows) return;
  const Pick pick = picks(a)[r];
  if (pick.written) return;                    // uniform
  const float* row = a.logits + r * a.ldl;
  float* out = a.probs + r * a.ldp;
  float v[kSPer / 4][4];
  const int i0 = blockIdx.x * kChunk + 4 * static_cast<int>(threadIdx.x);
  load_runs(row, i0, 4 * kSThreads, a.vocab, v);
  // (a product with the rounded 1 / total, 2^-53 off: a quotient each is most of the kernel's instructions)
  const double share = pick.total > 0.0 ? 1.0 / pick.total : 0.0;
#pragma unroll
  for (int k = 0; k < kSPer / 4; ++k) {
    const int i = i0 + 4 * k * kSThreads;
    float p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = taken(v[k][e]);
      p[e] = place_of(x, i + e) <= pick.border ? static_cast<float>(weight(exp2, x, pick.top, pick.rate) * share) : 0.0f;
    }
    if (i + 4 <= a.vocab) {
      store_four(out + i, p, a.past);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < a.vocab) out[i + e] = p[e];
    }
  }
}

int launch_sample(const SampleArgs& given, hipStream_t st) {
  SampleArgs a = given;
  // (Distributions of top-p rows stored as usual and past the caches, us alone and
  // with mmvq_verify_draft behind: 49 MB 53.5, 53.0 and 73.1, 73.5; 66 MB 66.7, 60.0
  // and 88.0, 87.6; 99 MB 84.0, 80.8 and 112, 113; 131 MB 107, 98 and 135, 132.)
  a.past = past_caches(a.n_rows, a.vocab, kL2);
  const unsigned chunks = static_cast<unsigned>(a.chunks), rows = static_cast<unsigned>(a.n_rows);
  const dim3 grid(chunks, rows < kGridRows ? rows : kGridRows, (rows + kGridRows - 1) / kGridRows);
  hipLaunchKernelGGL(sample_stats_kernel, grid, dim3(kSThreads), 0, st, a);
  int rc = check_launch();
  if (rc) return rc;
  hipLaunchKernelGGL(sample_pick_kernel, dim3(rows), dim3(kDThreads), chunks * sizeof(ChunkShift), st, a);
  rc = check_launch();
  if (rc || !a.probs) return rc;
  hipLaunchKernelGGL(sample_probs_kernel, grid, dim3(kSThreads), 0, st, a);
  return check_launch();
}

}  // namespace qmv
