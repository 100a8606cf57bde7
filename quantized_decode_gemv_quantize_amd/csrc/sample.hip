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
//           which the border lies. Where no more than kList tokens come up to
//           its end, they are sorted, cut and drawn from in LDS; else the
//           bin is narrowed until as few are left of it, and the row is
//           summed again;
//   probs   the distribution written out, if wanted.
// A chunk's bin is one 64-bit whole number: the count, and the sum in units of
// 2^-38 of its weights (adding in LDS in any order gives the same bits).
// Everything else is in 64-bit floating point: with 10^5 logits a running sum
// in 32 bits moves a border by more than many tokens' probability.
#include "draw.hpp"
#include "launch.hpp"
#include "serve_args.hpp"

namespace qmv {

constexpr int kSThreads = 256;
constexpr int kSPer = 16;                      // logits a lane
constexpr int kSWaves = kSThreads / kWave;
constexpr int kChunk = kSThreads * kSPer;
constexpr int kBins = 256;                     // the last one: everything below
constexpr int kDThreads = 1024;
constexpr int kDWaves = kDThreads / kWave;
constexpr int kList = 2048;                    // tokens that are sorted in LDS
constexpr int kTops = 256;                     // tokens that a chunk lists
constexpr int kUnit = 38;                      // a bin's sum is in units of 2^-kUnit
constexpr int kSumBits = 51;                   // and behind them its count
constexpr uint64_t kSumMask = (uint64_t(1) << kSumBits) - 1;

struct ChunkStat {
  float top;                                   // largest logit of the chunk
  int at;                                      // its lowest index
  double sum;                                  // of the weights relative to top, in pick: of the kept ones to the row's
  int listed;                                  // tokens in its list: all those of its bins
  int cut;                                     // up to this one
};
struct Pick {
  uint64_t border;                             // last kept place (below)
  double total;                                // sum of the kept weights; 0: none
  double rate;
  float top;
  int pad;
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

// 2^(-b / 4): what a bin's weights are relative to.
__device__ __forceinline__ double bin_scale(int b) {
  const double lower = b & 1 ? 0.84089641525371454303112547623321 : 1.0, half = b & 2 ? 0.70710678118654752440084436210485 : 1.0;
  return __builtin_ldexp(lower * half, -(b >> 2));
}
// A bin's sum, from its units.
__device__ __forceinline__ double bin_sum_of(uint64_t bin, int b) {
  return __builtin_ldexp(static_cast<double>(bin & kSumMask), -kUnit) * bin_scale(b);
}

// 2^(38 + x / 4) as a whole number, -1 <= x <= 1, in the low 52 bits of the
// result: the Taylor polynomial of degree 10 of exp(x ln 2 / 4), whose next
// term is below 2 10^-16, in units of 2^-kUnit, added to 2^52.
struct Units {
  double c[11];
  __device__ __forceinline__ Units() {
    double v = 0x1p38;
#pragma unroll
    for (int i = 0; i <= 10; ++i) {
      c[i] = v + (i == 0 ? 0x1p52 : 0.0);
      v = v * (0.69314718055994530941723212145818 / 4) / (i + 1);
    }
#pragma unroll
    for (int i = 0; i <= 10; ++i) asm("" : "+s"(c[i]));
  }
  __device__ __forceinline__ long long operator()(double x) const {
    double p = c[10];
#pragma unroll
    for (int i = 9; i >= 0; --i) p = fma(p, x, c[i]);
    return __double_as_longlong(p);
  }
};
static_assert(kUnit == 38);

// The row of a workgroup of a grid of chunks by rows. (Rows in a loop would
// have the compiler keep addresses and masks of every branch across it.)
constexpr int kGridRows = 1 << 15;
__device__ __forceinline__ int row_of_grid() { return static_cast<int>(blockIdx.z) * kGridRows + static_cast<int>(blockIdx.y); }

// Histogram of a chunk. Lanes add to one of kCopies copies, so that those of
// one bin meet less often (one copy 106 us, NN for four, for 256 rows of 151669).
constexpr int kCopies = 4;

__global__ void __launch_bounds__(kSThreads) sample_stats_kernel(SampleArgs a) {
  __shared__ float tops[kSWaves];
  __shared__ int ats[kSWaves], scans[kSWaves], listed, cut;
  __shared__ double sums[kSWaves];
  __shared__ unsigned long long bins[kBins * kCopies];
  const int tid = threadIdx.x, wave = tid >> 6, c = blockIdx.x, i0 = c * kChunk + 4 * tid;
  const int r = row_of_grid();
  if (r >= a.n_rows) return;
  const Settings s = settings_of(a, r);
  if (s.none) return;                          // uniform
  const float* row = a.logits + r * a.ldl;
  float v[kSPer];
  if ((c + 1) * kChunk <= a.vocab) {         // uniform: all loads at once
#pragma unroll
    for (int k = 0; k < kSPer; k += 4) {
      const u32x4 x = ld_x4(reinterpret_cast<const uint8_t*>(row + i0 + k * kSThreads));
#pragma unroll
      for (int e = 0; e < 4; ++e) v[k + e] = taken(__uint_as_float(x[e]));
    }
  } else {
#pragma unroll
    for (int k = 0; k < kSPer; ++k) {
      const int i = i0 + (k / 4) * 4 * kSThreads + k % 4;
      v[k] = row[i < a.vocab ? i : a.vocab - 1];
      v[k] = i < a.vocab ? taken(v[k]) : -INFINITY;
    }
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
#pragma unroll
    for (int k = 0; k < kCopies; ++k) bins[k * kSThreads + tid] = 0;
    if (tid == 0) {
      listed = 0;
      cut = -1;
    }
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
  const double dtop = top < INFINITY ? static_cast<double>(top) : 0.0;
  if (any && !filtered) {
    const Exp2 exp2;                         // (in scalar registers that the other branch has no use for)
#pragma unroll
    for (int k = 0; k < kSPer; ++k) sum += exp2((static_cast<double>(x[k]) - dtop) * s.rate);
  } else if (any) {
    const Units units;
    unsigned long long* mine = bins + (tid & (kCopies - 1));
    constexpr long long kOne = (1ll << kSumBits) - (0x433ll << 52);   // a count, without the exponent of 2^52
    const double rate4 = 4.0 * s.rate, top_quarter = floor(dtop * rate4);
#pragma unroll
    for (int k = 0; k < kSPer; ++k) {
      const double d = static_cast<double>(x[k]);
      const int b = bins_between(top_quarter, floor(d * rate4), kBins - 1);
      // 4 log2(w) + b is within +-1 but for the last bin, whose tokens count
      // as 2^-64 of the largest at least: 2^-52 of the sum for all of them
      const double f = fmax(fma(d - dtop, rate4, static_cast<double>(b)), -1.0);
      const unsigned long long add = static_cast<unsigned long long>(units(f) + kOne);
      if (x[k] > -INFINITY) atomicAdd(mine + b * kCopies, add);
      bin[k] = x[k] > -INFINITY ? b : kBins;
    }
  }
  const int64_t place = static_cast<int64_t>(r) * a.chunks + c;
  __syncthreads();
  if (filtered) {
    // the bins of at most kTops tokens together, and these tokens
    unsigned long long all = 0;
#pragma unroll
    for (int k = 0; k < kCopies; ++k) all += bins[tid * kCopies + k];
    chunk_bins(a)[place * kBins + tid] = all;
    sum = bin_sum_of(all, tid);
    int up = wave_scan(static_cast<int>(all >> kSumBits));
    if (lane_id() == kWave - 1) scans[wave] = up;
    __syncthreads();
    for (int w = 0; w < wave; ++w) up += scans[w];
    const uint64_t fits = __ballot(up <= kTops);
    if (lane_id() == 0 && fits) atomicMax(&cut, 64 * wave + 63 - __builtin_clzll(fits));
    __syncthreads();
    int hits = 0;
#pragma unroll
    for (int k = 0; k < kSPer; ++k) hits += any && bin[k] <= cut;
    int to = wave_scan(hits);
    int first = 0;
    if (lane_id() == kWave - 1 && to) first = atomicAdd(&listed, to);
    to += __builtin_amdgcn_readlane(first, kWave - 1) - hits;
    if (hits) {
      uint64_t* list = chunk_tops(a) + place * kTops;
#pragma unroll
      for (int k = 0; k < kSPer; ++k)
        if (bin[k] <= cut) list[to++] = place_of(v[k], i0 + (k / 4) * 4 * kSThreads + k % 4);
    }
  }
  sum = wave_sum(sum);
  if ((tid & 63) == 0) sums[wave] = sum;
  __syncthreads();
  if (tid == 0) {
    double all = 0.0;
#pragma unroll
    for (int w = 0; w < kSWaves; ++w) all += sums[w];
    chunk_stats(a)[place] = ChunkStat{top, at, all, filtered ? listed : 0, filtered ? cut : -1};
  }
}

// exp(chunk_top - top) in weights, the factor between the chunk's sums and the row's.
__device__ __forceinline__ double chunk_factor(const Exp2& exp2, float chunk_top, float top, double rate) {
  if (chunk_top == top) return 1.0;
  return weight(exp2, chunk_top, top, rate);
}

struct PickLds {
  double part_sum[4][kBins];                   // of bins, by quarter of the chunks
  int part_count[4][kBins];
  double bin_sum[kBins];                       // of the row's bins, then running sums up to their ends
  int bin_count[kBins];
  uint64_t list[kList];
  double weights[kList];
  double waves[kDWaves];
  unsigned long long cell_sum[kBins];
  uint32_t cell_count[kBins];
  int64_t ahead;
  double d0, d1, d2;
  int i0, i1, i2;
};
struct ChunkShift {                            // of each chunk, in dynamic LDS
  double factor;                               // from its weights to the row's; below 0: it has none
  int shift;                                   // from its bins to the row's
  int pad;
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
  return before + (up - v);
}

// Elements of the row whose place is in lo..hi: f(place, value), by all lanes,
// with eight loads on their way.
template <class Fn>
__device__ __forceinline__ void each_between(const SampleArgs& a, const float* row, uint64_t lo, uint64_t hi, Fn f) {
  constexpr int kAhead = 8;
  for (int i0 = 4 * static_cast<int>(threadIdx.x); i0 < a.vocab; i0 += 4 * kDThreads * kAhead) {
    float v[kAhead][4];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) load_quad(row, i0 + 4 * kDThreads * q, a.vocab, -INFINITY, v[q]);
#pragma unroll
    for (int q = 0; q < kAhead; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = taken(v[q][e]);
        const uint64_t at = place_of(x, i0 + 4 * kDThreads * q + e);
        if (x > -INFINITY && at >= lo && at <= hi) f(at, x);
      }
  }
}

// Ascending, n a power of two; the workgroup.
__device__ __forceinline__ void sort_list(uint64_t* list, int n) {
  for (int k = 2; k <= n; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      __syncthreads();
      for (int t = threadIdx.x; t < n / 2; t += kDThreads) {
        const int i = 2 * t - (t & (j - 1));   // pairs i, i + j
        const uint64_t x = list[i], y = list[i + j];
        if ((x > y) == ((i & k) == 0)) {
          list[i] = y;
          list[i + j] = x;
        }
      }
    }
  __syncthreads();
}

// The border of a filter among the `count` elements with places lo..hi, before
// which `ahead` elements of the weight `passed` come: the last place kept by
// top-k (k > 0: the k-th element) or by top-p (the last before which less than
// `goal` has passed); `kept`: the weight up to it.
__device__ uint64_t find_border(const SampleArgs& a, const Exp2& exp2, const float* row, float top, double rate, uint64_t lo, uint64_t hi,
                                int64_t count, int64_t ahead, double passed, int k, double goal, PickLds& l, double& kept) {
  const int tid = threadIdx.x;
  while (count > kList) {
    // cells of equal width; at the end a cell is one place
    int shift = 0;
    while (((hi - lo) >> shift) >= kBins) ++shift;
    __syncthreads();
    if (tid < kBins) {
      l.cell_sum[tid] = 0;
      l.cell_count[tid] = 0;
    }
    __syncthreads();
    // weights of a row's 2^24 elements at most, in units that their sum stays below 2^63 in
    int most;
    (void)__builtin_frexp(weight(exp2, value_at(lo), top, rate), &most);
    const int unit = 38 - most;
    each_between(a, row, lo, hi, [&](uint64_t at, float v) QMV_INLINE {
      const int cell = static_cast<int>((at - lo) >> shift);
      atomicAdd(&l.cell_sum[cell], static_cast<unsigned long long>(__builtin_ldexp(weight(exp2, v, top, rate), unit) + 0.5));
      atomicAdd(&l.cell_count[cell], 1u);
    });
    __syncthreads();
    if (tid == 0) {
      int cell = 0;
      // where rounding leaves the goal unreached: the last cell that has elements
      int last = kBins - 1;
      while (last > 0 && l.cell_count[last] == 0) --last;
      for (; cell < last; ++cell) {
        const double sum = __builtin_ldexp(static_cast<double>(l.cell_sum[cell]), -unit);
        if (l.cell_count[cell] && (k > 0 ? ahead + l.cell_count[cell] >= k : passed + sum >= goal)) break;
        ahead += l.cell_count[cell];
        passed += sum;
      }
      l.i0 = cell;
      l.d0 = passed;
      l.ahead = ahead;
    }
    __syncthreads();
    const uint64_t from = lo + (static_cast<uint64_t>(l.i0) << shift), to = from + ((uint64_t(1) << shift) - 1);
    lo = from;
    hi = to < hi ? to : hi;
    count = l.cell_count[l.i0];
    ahead = l.ahead;
    passed = l.d0;
    __syncthreads();
  }
  __syncthreads();
  if (tid == 0) l.i0 = 0;
  __syncthreads();
  each_between(a, row, lo, hi, [&](uint64_t at, float) QMV_INLINE {
    const int to = atomicAdd(&l.i0, 1);
    if (to < kList) l.list[to] = at;
  });
  __syncthreads();
  int n = 2;
  while (n < count) n <<= 1;
  for (int i = static_cast<int>(count) + tid; i < n; i += kDThreads) l.list[i] = ~uint64_t(0);
  sort_list(l.list, n);
  // two neighbours a lane
  double w[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) w[e] = 2 * tid + e < count ? weight(exp2, value_at(l.list[2 * tid + e]), top, rate) : 0.0;
  double total;
  const double before = passed + block_scan_d(w[0] + w[1], l.waves, total);
  if (tid == 0) l.i1 = 0;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = 2 * tid + e;
    const bool in = i < count && (k > 0 ? ahead + i < k : before + (e ? w[0] : 0.0) < goal);
    if (in) atomicMax(&l.i1, i);
  }
  __syncthreads();
  const int last = l.i1;
  if (last / 2 == tid) l.d1 = before + w[0] + (last & 1 ? w[1] : 0.0);
  __syncthreads();
  kept = l.d1;
  return l.list[last];
}

// Smallest key whose logit passes, of those up to `most`, which does; one
// wave, 64 keys at a time.
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

// Running sums of the row's bins: of the chunks', each moved to the row's
// grid. A fourth of the threads takes a fourth of the chunks; chunk bins that
// the row's last bin takes in are summed by the threads they belong to.
__device__ __forceinline__ void join_bins(const SampleArgs& a, int r, const ChunkShift* chunk, PickLds& l) {
  const int tid = threadIdx.x, part = tid / kBins, bin = tid % kBins;
  const uint64_t* bins = chunk_bins(a) + static_cast<int64_t>(r) * a.chunks * kBins;
  double sum = 0.0, far_sum = 0.0;
  int count = 0, far_count = 0;
#pragma unroll 4
  for (int c = part; c < a.chunks; c += kDThreads / kBins) {
    const ChunkShift h = chunk[c];
    if (h.factor < 0.0) continue;              // uniform in a wave
    const int from = bin - h.shift;
    const bool near = from >= 0 && bin < kBins - 1, far = bin + h.shift >= kBins - 1;
    const uint64_t x = near ? bins[static_cast<int64_t>(c) * kBins + from] : 0, y = far ? bins[static_cast<int64_t>(c) * kBins + bin] : 0;
    sum += bin_sum_of(x, near ? from : 0) * h.factor;
    count += static_cast<int>(x >> kSumBits);
    far_sum += bin_sum_of(y, bin) * h.factor;
    far_count += static_cast<int>(y >> kSumBits);
  }
  // the last bin
  const double far_wave = wave_sum(far_sum);
  const int far_wave_count = __builtin_amdgcn_readlane(wave_scan(far_count), kWave - 1);
  __syncthreads();                             // the row before is done with LDS
  l.part_sum[part][bin] = sum;
  l.part_count[part][bin] = count;
  if (tid < kDWaves) l.cell_count[tid] = 0;
  __syncthreads();
  if (lane_id() == 0) {
    l.waves[tid >> 6] = far_wave;
    l.cell_count[tid >> 6] = far_wave_count;
  }
  __syncthreads();
  double own = 0.0;
  int own_count = 0;
  if (tid < kBins) {
    own = (l.part_sum[0][tid] + l.part_sum[1][tid]) + (l.part_sum[2][tid] + l.part_sum[3][tid]);
    own_count = l.part_count[0][tid] + l.part_count[1][tid] + l.part_count[2][tid] + l.part_count[3][tid];
    if (tid == kBins - 1)
      for (int w = 0; w < kDWaves; ++w) {
        own += l.waves[w];
        own_count += static_cast<int>(l.cell_count[w]);
      }
  }
  double up = wave_scan(own);
  int up_count = wave_scan(own_count);
  __syncthreads();
  if (lane_id() == kWave - 1) {
    l.waves[tid >> 6] = up;
    l.cell_count[tid >> 6] = up_count;
  }
  __syncthreads();
  if (tid < kBins) {
    for (int w = 0; w < (tid >> 6); ++w) {
      up += l.waves[w];
      up_count += static_cast<int>(l.cell_count[w]);
    }
    l.bin_sum[tid] = up;
    l.bin_count[tid] = up_count;
  }
  __syncthreads();
}

// First bin whose running count (k > 0) or sum reaches k or the goal; the
// last one that has tokens where none does.
__device__ __forceinline__ int crossing(const PickLds& l, int k, double goal, int* slot) {
  const int tid = threadIdx.x;
  if (tid == 0) *slot = kBins;
  __syncthreads();
  if (tid < kBins) {
    const int count = l.bin_count[tid], all = l.bin_count[kBins - 1];
    const bool hit = (k > 0 ? count >= k : l.bin_sum[tid] >= goal) || count == all;
    const uint64_t hits = __ballot(hit && count > 0);
    if (lane_id() == 0 && hits) atomicMin(slot, (tid & ~63) + __builtin_ctzll(hits));
  }
  __syncthreads();
  return *slot;
}

// Where a row's draw stands.
struct Drawn {
  uint64_t border;
  double total, chosen;
  int token;
};

// All `count` tokens up to the border's bin, in LDS: sorted, cut by all
// filters, and drawn from. all: the sum of the row's weights.
__device__ __forceinline__ Drawn draw_short(const Exp2& exp2, const Settings& s, float top, int count, double all, float u, PickLds& l) {
  const int tid = threadIdx.x;
  int n = 2;
  while (n < count) n <<= 1;
  for (int i = count + tid; i < n; i += kDThreads) l.list[i] = ~uint64_t(0);
  sort_list(l.list, n);
  double w[2], total;
#pragma unroll
  for (int e = 0; e < 2; ++e) w[e] = 2 * tid + e < count ? weight(exp2, value_at(l.list[2 * tid + e]), top, s.rate) : 0.0;
  const int k = s.k > 0 && s.k < count ? s.k : count;
#pragma unroll
  for (int e = 0; e < 2; ++e) w[e] = 2 * tid + e < k ? w[e] : 0.0;
  const double before = block_scan_d(w[0] + w[1], l.waves, total);
  const double goal = s.p * (s.k > 0 ? total : all);
  if (tid == 0) l.i0 = 0;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = 2 * tid + e;
    const bool in = i < k && (s.p >= 1.0 || before + (e ? w[0] : 0.0) < goal) && w[e] >= s.m;
    const uint64_t ins = __ballot(in);
    if (ins && lane_id() == 63 - __builtin_clzll(ins)) atomicMax(&l.i0, i);
  }
  __syncthreads();
  const int last = l.i0;                       // the first token is kept in any case
  Drawn d;
  d.border = l.list[last];
  // the kept ones by their indices
  n = 2;
  while (n < last + 1) n <<= 1;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = 2 * tid + e;
    if (i < n) {
      l.weights[i] = w[e];
      l.list[i] = i <= last ? (l.list[i] & kLowIndex) << 12 | static_cast<uint64_t>(i) : ~uint64_t(0);
    }
  }
  sort_list(l.list, n);
  int index[2] = {-1, -1};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = 2 * tid + e;
    w[e] = 0.0;
    if (i <= last) {
      const uint64_t x = l.list[i];
      w[e] = l.weights[x & 4095];
      index[e] = static_cast<int>(x >> 12);
    }
  }
  const double up = block_scan_d(w[0] + w[1], l.waves, d.total);
  if (tid == 0) {
    l.i0 = 0x7fffffff;
    l.i1 = -1;
  }
  __syncthreads();
  const double drawn = static_cast<double>(u) * d.total;
  const bool hit0 = w[0] > 0.0 && up + w[0] > drawn, hit1 = w[1] > 0.0 && up + w[0] + w[1] > drawn;
  const uint64_t hits = __ballot(hit0 || hit1), some = __ballot(w[0] > 0.0 || w[1] > 0.0);
  if (hits && lane_id() == __builtin_ctzll(hits)) atomicMin(&l.i0, 2 * tid + (hit0 ? 0 : 1));
  if (some && lane_id() == 63 - __builtin_clzll(some)) atomicMax(&l.i1, 2 * tid + (w[1] > 0.0 ? 1 : 0));
  __syncthreads();
  const int take = l.i0 != 0x7fffffff ? l.i0 : l.i1;
  const uint64_t x = l.list[take];
  d.token = static_cast<int>(x >> 12);
  d.chosen = l.weights[x & 4095] / d.total;
  return d;
}

// The border by all filters, of a row with more tokens up to it than fit LDS.
__device__ uint64_t far_border(const SampleArgs& a, const Exp2& exp2, const float* row, const Settings& s, float top, PickLds& l) {
  const int tid = threadIdx.x;
  const double top_quarter = quarter(top, 4.0 * s.rate);
  const uint32_t most = key_of(top);
  uint64_t border = ~uint64_t(0);
  if (s.m > 0.0)                               // every wave for itself
    border = last_place(first_key(most, [&](float v) QMV_INLINE { return weight(exp2, v, top, s.rate) >= s.m; }));
  double total = l.bin_sum[kBins - 1];
  for (int turn = 0; turn < 2; ++turn) {       // top-k, then top-p
    if (turn == 0 ? s.k == 0 || s.k >= l.bin_count[kBins - 1] : s.p >= 1.0) continue;   // uniform
    const int k = turn == 0 ? s.k : 0;
    const double goal = s.p * total;
    const int b = crossing(l, k, goal, &l.i2);
    const int ahead = b > 0 ? l.bin_count[b - 1] : 0, count = l.bin_count[b] - ahead;
    const double passed = b > 0 ? l.bin_sum[b - 1] : 0.0;
    const uint32_t low = first_key(most, [&](float v) QMV_INLINE { return bin_of(v, 4.0 * s.rate, top, top_quarter) <= b; });
    const uint32_t high = b == 0 ? most : first_key(most, [&](float v) QMV_INLINE { return bin_of(v, 4.0 * s.rate, top, top_quarter) < b; }) - 1;
    double kept;
    const uint64_t found = find_border(a, exp2, row, top, s.rate, first_place(high), last_place(low), count, ahead, passed, k, goal, l, kept);
    if (turn == 0) total = kept;
    border = found < border ? found : border;
    __syncthreads();
  }
  (void)tid;
  return border;
}

// The kept weights of each chunk, and a draw by them: the chunk in which the
// running sum passes the goal, then its element.
__device__ __forceinline__ Drawn draw_long(const SampleArgs& a, const Exp2& exp2, const float* row, ChunkStat* st, const Settings& s, float top,
                                           uint64_t border, float u, PickLds& l) {
  const int tid = threadIdx.x, wave = tid >> 6;
  Drawn d{border, 0.0, 0.0, -1};
  __syncthreads();
  if (border != ~uint64_t(0)) {
    for (int c = wave; c < a.chunks; c += kDWaves) {
      double sum = 0.0;
#pragma unroll 4
      for (int j = 0; j < kChunk / (4 * kWave); ++j) {
        const int i = c * kChunk + 4 * (j * kWave + lane_id());
        float v[4];
        load_quad(row, i, a.vocab, -INFINITY, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = taken(v[e]);
          if (place_of(x, i + e) <= border) sum += weight(exp2, x, top, s.rate);
        }
      }
      sum = wave_sum(sum);
      if (lane_id() == 0) st[c].sum = sum;
    }
  } else {
    for (int c = tid; c < a.chunks; c += kDThreads) st[c].sum *= chunk_factor(exp2, st[c].top, top, s.rate);
  }
  __syncthreads();
  double sum = 0.0;
  for (int c = lane_id(); c < a.chunks; c += kWave) sum += st[c].sum;
  d.total = wave_sum(sum);
  if (!a.tokens && !a.chosen) return d;
  const double goal = static_cast<double>(u) * d.total;
  double run = 0.0, before = 0.0, last_before = 0.0;
  int found = -1, last = 0;
  for (int c0 = 0; c0 < a.chunks && found < 0; c0 += kWave) {
    const int c = c0 + lane_id();
    const double w = c < a.chunks ? st[c].sum : 0.0, up = wave_scan(w) + run;
    const uint64_t hit = __ballot(up > goal), some = __ballot(w > 0.0);
    if (some) {
      const int i = 63 - __builtin_clzll(some);
      last = c0 + i;
      last_before = __shfl(up - w, i);
    }
    if (hit) {
      const int i = __builtin_ctzll(hit);
      found = c0 + i;
      before = __shfl(up - w, i);
    }
    run = __shfl(up, kWave - 1);
  }
  const int c = found >= 0 ? found : last;
  if (found < 0) before = last_before;
  // its elements, a run of four a lane
  const int i0 = c * kChunk + 4 * tid;
  float v[4];
  double w[4], own = 0.0;
  load_quad(row, i0, a.vocab, -INFINITY, v);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float x = taken(v[e]);
    w[e] = place_of(x, i0 + e) <= border ? weight(exp2, x, top, s.rate) : 0.0;
    own += w[e];
  }
  double all;
  double up = before + block_scan_d(own, l.waves, all);
  if (tid == 0) {
    l.i0 = 0x7fffffff;
    l.i1 = -1;
  }
  __syncthreads();
  int hit = 0x7fffffff, last_hit = -1;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    up += w[e];
    if (w[e] > 0.0) {
      last_hit = i0 + e;
      if (up > goal && hit == 0x7fffffff) hit = i0 + e;
    }
  }
  if (hit != 0x7fffffff) atomicMin(&l.i0, hit);
  if (last_hit >= 0) atomicMax(&l.i1, last_hit);
  __syncthreads();
  d.token = l.i0 != 0x7fffffff ? l.i0 : l.i1;
  if (d.token >= 0) d.chosen = weight(exp2, taken(row[d.token]), top, s.rate) / d.total;
  return d;
}

// The tokens of bins 0..b in l.list: from the chunks' lists, or from the row
// where a chunk lists fewer. Returns their number.
__device__ __forceinline__ int gather(const SampleArgs& a, const float* row, int r, const Settings& s, float top, int b, const ChunkShift* chunk,
                                      PickLds& l) {
  const int tid = threadIdx.x, wave = tid >> 6;
  const ChunkStat* st = chunk_stats(a) + static_cast<int64_t>(r) * a.chunks;
  const double top_quarter = quarter(top, 4.0 * s.rate);
  bool covered = true;
  for (int c = tid; c < a.chunks; c += kDThreads)
    if (chunk[c].factor >= 0.0 && st[c].cut < kBins - 1 && (b == kBins - 1 || st[c].cut + chunk[c].shift < b)) covered = false;
  if (tid == 0) l.i0 = 0;
  if (__syncthreads_and(covered)) {
    for (int c = wave; c < a.chunks; c += kDWaves) {
      if (chunk[c].factor < 0.0 || chunk[c].shift > b) continue;
      const uint64_t* list = chunk_tops(a) + (static_cast<int64_t>(r) * a.chunks + c) * kTops;
      const int listed = st[c].listed;
#pragma unroll
      for (int j = 0; j < kTops / kWave; ++j) {
        const int i = j * kWave + lane_id();
        const uint64_t x = i < listed ? list[i] : 0;
        const bool in = i < listed && bin_of(value_at(x), 4.0 * s.rate, top, top_quarter) <= b;
        const uint64_t ins = __ballot(in);
        if (ins == 0) continue;
        int first = 0;
        if (lane_id() == 0) first = atomicAdd(&l.i0, __builtin_popcountll(ins));
        first = __builtin_amdgcn_readfirstlane(first);
        const int at = first + __builtin_popcountll(ins & ((uint64_t(1) << lane_id()) - 1));
        if (in && at < kList) l.list[at] = x;
      }
    }
  } else {
    const uint32_t low = first_key(key_of(top), [&](float v) QMV_INLINE { return bin_of(v, 4.0 * s.rate, top, top_quarter) <= b; });
    each_between(a, row, 0, last_place(low), [&](uint64_t at, float) QMV_INLINE {
      const int to = atomicAdd(&l.i0, 1);
      if (to < kList) l.list[to] = at;
    });
  }
  __syncthreads();
  const int n = l.i0 < kList ? l.i0 : kList;
  __syncthreads();
  return n;
}

__global__ void __launch_bounds__(kDThreads) sample_pick_kernel(SampleArgs a) {
  __shared__ PickLds l;
  extern __shared__ __align__(16) uint8_t dynamic[];
  ChunkShift* chunk = reinterpret_cast<ChunkShift*>(dynamic);
  const Exp2 exp2;
  const int tid = threadIdx.x;
  const int r = blockIdx.x;
  const Settings s = settings_of(a, r);
  const float* row = a.logits + r * a.ldl;
  const float u = a.u ? a.u[r] : 0.0f;
  ChunkStat* st = chunk_stats(a) + static_cast<int64_t>(r) * a.chunks;
  float top = -INFINITY;
  int at = 0x7fffffff;
  if (!s.none) {
    for (int c = lane_id(); c < a.chunks; c += kWave) take_top(top, at, st[c].top, st[c].at);
    wave_top(top, at);
  }
  Drawn d{0, 0.0, 0.0, -1};
  if (top == -INFINITY) {                    // uniform
  } else if (s.greedy) {
    d = Drawn{place_of(top, at), 1.0, 1.0, at};
  } else if (!s.filtered()) {
    d = draw_long(a, exp2, row, st, s, top, ~uint64_t(0), u, l);
  } else {
    const double top_quarter = quarter(top, 4.0 * s.rate);
    for (int c = tid; c < a.chunks; c += kDThreads) {
      const float ct = st[c].top;
      const bool has = ct > -INFINITY && (top < INFINITY || ct == top);
      const int shift = has && top < INFINITY ? bins_between(top_quarter, quarter(ct, 4.0 * s.rate), kBins) : 0;
      chunk[c] = ChunkShift{has ? chunk_factor(exp2, ct, top, s.rate) : -1.0, shift, 0};
    }
    __syncthreads();
    join_bins(a, r, chunk, l);
    // the last bin that can hold the border
    const double all = l.bin_sum[kBins - 1];
    int b = kBins - 1;
    if (s.k > 0) b = crossing(l, s.k, 0.0, &l.i2);
    else if (s.p < 1.0) b = crossing(l, 0, s.p * all, &l.i2);
    if (s.m > 0.0 && (s.k == 0 || s.p >= 1.0)) {   // (top-p needs the sum of all k)
      // w >= m ends in the bin of 4 log2(m), to one by rounding, behind the top's
      const double end = 4.0 * -log2(s.m) + 2.0;
      if (end < b) b = static_cast<int>(end);
    }
    __syncthreads();
    if (l.bin_count[b] <= kList) {
      const int n = gather(a, row, r, s, top, b, chunk, l);
      d = draw_short(exp2, s, top, n, all, u, l);
    } else {
      const uint64_t border = far_border(a, exp2, row, s, top, l);
      d = draw_long(a, exp2, row, st, s, top, border, u, l);
    }
  }
  if (tid == 0) {
    if (a.tokens) a.tokens[r] = d.token;
    if (a.chosen) a.chosen[r] = static_cast<float>(d.chosen);
    if (a.probs) picks(a)[r] = Pick{d.border, d.total, s.rate, top, 0};
  }
}

__global__ void __launch_bounds__(kSThreads) sample_probs_kernel(SampleArgs a) {
  const Exp2 exp2;
  const int r = row_of_grid();
  if (r >= a.n_rows) return;
  const Pick pick = picks(a)[r];
  const float* row = a.logits + r * a.ldl;
  float* out = a.probs + r * a.ldp;
  float v[kSPer];
  const int i0 = blockIdx.x * kChunk + 4 * static_cast<int>(threadIdx.x);
#pragma unroll
  for (int k = 0; k < kSPer; k += 4) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + k * kSThreads + e;
      v[k + e] = i < a.vocab ? taken(row[i]) : -INFINITY;
    }
  }
#pragma unroll
  for (int k = 0; k < kSPer; k += 4) {
    const int i = i0 + k * kSThreads;
    float p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool in = pick.total > 0.0 && place_of(v[k + e], i + e) <= pick.border;
      p[e] = in ? static_cast<float>(weight(exp2, v[k + e], pick.top, pick.rate) / pick.total) : 0.0f;
    }
    if (i + 4 <= a.vocab) {
      __builtin_memcpy(__builtin_assume_aligned(out + i, 4), p, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < a.vocab) out[i + e] = p[e];
    }
  }
}

int launch_sample(const SampleArgs& a, hipStream_t st) {
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
