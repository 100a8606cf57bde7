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
//           sum over bins of a quarter octave of the weight;
//   pick    a workgroup a row: the chunks joined, the bin in which the border
//           lies, its tokens sorted, the kept weights summed, the token drawn;
//   probs   the distribution written out, if wanted.
// A bin's sums are 64-bit whole numbers in units of 2^-51 of its weights (sums
// in LDS in any order give the same bits), everything else is in 64-bit
// floating point: with 10^5 logits a running sum in 32 bits moves a border by
// more than many tokens' probability.
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

struct ChunkStat {
  float top;                                   // largest logit of the chunk
  int at;                                      // its lowest index
  double sum;                                  // of the weights relative to top, in pick: of the kept ones to the row's
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
__device__ __forceinline__ uint64_t* bin_sums(const SampleArgs& a) { return reinterpret_cast<uint64_t*>(picks(a) + a.n_rows); }
__device__ __forceinline__ uint32_t* bin_counts(const SampleArgs& a) {
  return reinterpret_cast<uint32_t*>(bin_sums(a) + static_cast<int64_t>(a.n_rows) * a.chunks * kBins);
}

int64_t sample_bytes(int n_rows, int vocab, int* chunks) {
  const int64_t c = (vocab + kChunk - 1) / kChunk;
  if (chunks) *chunks = static_cast<int>(c);
  return n_rows * (c * (static_cast<int64_t>(sizeof(ChunkStat)) + kBins * 12) + static_cast<int64_t>(sizeof(Pick)));
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
// share: whole numbers that never fall with the logit.
__device__ __forceinline__ double quarter(float v, double rate) {
  constexpr double kMost = 1125899906842624.0;   // 2^50: differences stay exact
  if (!(v < INFINITY)) return kMost;
  return fmin(fmax(floor(static_cast<double>(v) * (4.0 * rate)), -kMost), kMost);
}
// Bin of a logit below a largest one, kBins for none.
__device__ __forceinline__ int bin_of(float v, double rate, float top, double top_quarter) {
  if (!(v > -INFINITY)) return kBins;
  if (top == INFINITY) return v == top ? 0 : kBins;
  return static_cast<int>(fmin(top_quarter - quarter(v, rate), kBins - 1.0));
}

template <int WAVES>
__device__ __forceinline__ double join_waves(const double* lds) {
  double sum = 0.0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) sum += lds[w];
  return sum;
}

__global__ void __launch_bounds__(kSThreads) sample_stats_kernel(SampleArgs a) {
  __shared__ float tops[kSWaves];
  __shared__ int ats[kSWaves];
  __shared__ double sums[kSWaves];
  __shared__ uint64_t bin_sum[kBins];
  __shared__ uint32_t bin_count[kBins];
  const Exp2 exp2;
  const int tid = threadIdx.x, wave = tid >> 6, c = blockIdx.x, i0 = c * kChunk + 4 * tid;
  for (int r = blockIdx.y; r < a.n_rows; r += gridDim.y) {
    const Settings s = settings_of(a, r);
    if (s.none) continue;                      // uniform
    const float* row = a.logits + r * a.ldl;
    float v[kSPer];
#pragma unroll
    for (int k = 0; k < kSPer; k += 4) {
      float four[4];
      load_quad(row, i0 + k * kSThreads, a.vocab, -INFINITY, four);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[k + e] = taken(four[e]);
    }
    float top = -INFINITY;
    int at = 0x7fffffff;
#pragma unroll
    for (int k = 0; k < kSPer; ++k) top = fmaxf(top, v[k]);
#pragma unroll
    for (int k = kSPer - 1; k >= 0; --k)
      at = v[k] == top && top > -INFINITY ? i0 + (k / 4) * 4 * kSThreads + k % 4 : at;
    wave_top(top, at);
    const bool bins = s.filtered();
    __syncthreads();                           // the row before is done with LDS
    if ((tid & 63) == 0) {
      tops[wave] = top;
      ats[wave] = at;
    }
    if (bins) {
      bin_sum[tid] = 0;
      bin_count[tid] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSWaves; ++w) take_top(top, at, tops[w], ats[w]);
    double sum = 0.0;
    if (!s.greedy && top > -INFINITY) {
      const double top_quarter = quarter(top, s.rate);
#pragma unroll
      for (int k = 0; k < kSPer; ++k) {
        const double w = weight(exp2, v[k], top, s.rate);
        sum += w;
        if (bins) {
          const int b = bin_of(v[k], s.rate, top, top_quarter);
          if (b < kBins) {
            // w 2^(b / 4) is below 2^1.25: 4096 of them in units of 2^-50 stay below 2^64
            atomicAdd(reinterpret_cast<unsigned long long*>(&bin_sum[b]),
                      static_cast<unsigned long long>(__builtin_ldexp(w, 50 + b / 4) + 0.5));
            atomicAdd(&bin_count[b], 1u);
          }
        }
      }
    }
    sum = wave_sum(sum);
    if ((tid & 63) == 0) sums[wave] = sum;
    __syncthreads();
    const int64_t place = static_cast<int64_t>(r) * a.chunks + c;
    if (tid == 0) chunk_stats(a)[place] = ChunkStat{top, at, join_waves<kSWaves>(sums)};
    if (bins) {
      bin_sums(a)[place * kBins + tid] = bin_sum[tid];
      bin_counts(a)[place * kBins + tid] = bin_count[tid];
    }
  }
}

// exp(chunk_top - top) in weights, the factor between the chunk's sums and the row's.
__device__ __forceinline__ double chunk_factor(const Exp2& exp2, float chunk_top, float top, double rate) {
  if (chunk_top == top) return 1.0;
  return weight(exp2, chunk_top, top, rate);
}

struct PickLds {
  double sum[4][kBins];                        // of bins, by quarter of the chunks
  int count[4][kBins];
  double bin_sum[kBins];
  int bin_count[kBins];
  uint64_t list[kList];
  double waves[kDWaves];
  int iwaves[kDWaves];
  unsigned long long cell_sum[kBins];
  uint32_t cell_count[kBins];
  uint64_t border;
  double d0, d1;
  int i0, i1, i2;
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

// Elements of the row whose place is in lo..hi: f(place, value), by all lanes.
template <class Fn>
__device__ __forceinline__ void each_between(const SampleArgs& a, const float* row, uint64_t lo, uint64_t hi, Fn f) {
  for (int i0 = 4 * static_cast<int>(threadIdx.x); i0 < a.vocab; i0 += 4 * kDThreads) {
    float v[4];
    load_quad(row, i0, a.vocab, -INFINITY, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = taken(v[e]);
      const uint64_t at = place_of(x, i0 + e);
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
      l.list[0] = static_cast<uint64_t>(ahead);
    }
    __syncthreads();
    const uint64_t from = lo + (static_cast<uint64_t>(l.i0) << shift), to = from + ((uint64_t(1) << shift) - 1);
    lo = from;
    hi = to < hi ? to : hi;
    count = l.cell_count[l.i0];
    ahead = static_cast<int64_t>(l.list[0]);
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

// The row's border by all filters.
__device__ uint64_t border_of(const SampleArgs& a, const Exp2& exp2, const float* row, int r, const Settings& s, float top, PickLds& l) {
  const int tid = threadIdx.x;
  const ChunkStat* st = chunk_stats(a) + static_cast<int64_t>(r) * a.chunks;
  const uint64_t* hs = bin_sums(a) + static_cast<int64_t>(r) * a.chunks * kBins;
  const uint32_t* hc = bin_counts(a) + static_cast<int64_t>(r) * a.chunks * kBins;
  const double top_quarter = quarter(top, s.rate);
  // a fourth of the threads takes a fourth of the chunks
  const int part = tid / kBins, bin = tid % kBins;
  double bin_sum = 0.0;
  int bin_count = 0;
  for (int c = part; c < a.chunks; c += kDThreads / kBins) {
    const float ct = st[c].top;
    if (!(ct > -INFINITY) || (top == INFINITY && ct != top)) continue;
    const double shift = top == INFINITY ? 0.0 : top_quarter - quarter(ct, s.rate);
    const double factor = chunk_factor(exp2, ct, top, s.rate);
    // bins of the chunk that fall into this one: the last takes all behind it
    int from = static_cast<int>(fmax(bin - shift, -1.0)), to = from;
    if (bin == kBins - 1) {
      from = from < 0 ? 0 : from;
      to = kBins - 1;
    }
    for (int b = from; b <= to; ++b) {
      if (b < 0) continue;
      bin_sum += __builtin_ldexp(static_cast<double>(hs[c * kBins + b]), -(50 + b / 4)) * factor;
      bin_count += static_cast<int>(hc[c * kBins + b]);
    }
  }
  __syncthreads();                             // the row before is done with LDS
  l.sum[part][bin] = bin_sum;
  l.count[part][bin] = bin_count;
  __syncthreads();
  if (tid < kBins) {
    l.bin_sum[tid] = (l.sum[0][tid] + l.sum[1][tid]) + (l.sum[2][tid] + l.sum[3][tid]);
    l.bin_count[tid] = l.count[0][tid] + l.count[1][tid] + l.count[2][tid] + l.count[3][tid];
  }
  // min-p: the smallest logit that is kept
  __syncthreads();
  if (tid < kWave && s.m > 0.0) {
    const uint32_t least = first_key(key_of(top), [&](float v) QMV_INLINE { return weight(exp2, v, top, s.rate) >= s.m; });
    if (tid == 0) l.border = last_place(least);
  }
  __syncthreads();
  uint64_t border = s.m > 0.0 ? l.border : ~uint64_t(0);
  double total = 0.0;
  for (int turn = 0; turn < 2; ++turn) {       // top-k, then top-p
    if (turn == 0 ? s.k == 0 : s.p >= 1.0) continue;
    const double goal = s.p * total;
    __syncthreads();
    if (tid == 0) {
      int b = 0, last = -1;
      int64_t ahead = 0, ahead_last = 0;
      double passed = 0.0, passed_last = 0.0, all = 0.0;
      if (turn == 1 && s.k == 0)
        for (int i = 0; i < kBins; ++i) all += l.bin_sum[i];
      l.d1 = all;
      const double want = s.k == 0 ? s.p * all : goal;
      for (; b < kBins; ++b) {
        if (l.bin_count[b] == 0) continue;
        last = b;
        ahead_last = ahead;
        passed_last = passed;
        if (turn == 0 ? ahead + l.bin_count[b] >= s.k : passed + l.bin_sum[b] >= want) break;
        ahead += l.bin_count[b];
        passed += l.bin_sum[b];
      }
      l.i0 = last;
      l.i1 = static_cast<int>(ahead_last);
      l.i2 = b == kBins;                       // nothing is cut off
      l.d0 = passed_last;
    }
    __syncthreads();
    const int b = l.i0, ahead = l.i1, open = l.i2;
    const double passed = l.d0, all = l.d1;
    if (turn == 1 && s.k == 0) total = all;
    __syncthreads();
    if (turn == 0 && open) {                   // fewer than k tokens have a weight
      if (tid == 0) {
        double sum = 0.0;
        for (int i = 0; i < kBins; ++i) sum += l.bin_sum[i];
        l.d0 = sum;
      }
      __syncthreads();
      total = l.d0;
      continue;
    }
    // keys of the bin
    if (tid < kWave) {
      const uint32_t most = key_of(top);
      const uint32_t low = first_key(most, [&](float v) QMV_INLINE { return bin_of(v, s.rate, top, top_quarter) <= b; });
      const uint32_t high = b == 0 ? most : first_key(most, [&](float v) QMV_INLINE { return bin_of(v, s.rate, top, top_quarter) < b; }) - 1;
      if (tid == 0) {
        l.list[0] = first_place(high);
        l.list[1] = last_place(low);
      }
    }
    __syncthreads();
    const uint64_t lo = l.list[0], hi = l.list[1];
    __syncthreads();
    double kept;
    const uint64_t found = find_border(a, exp2, row, top, s.rate, lo, hi, l.bin_count[b], ahead, passed, turn == 0 ? s.k : 0,
                                       s.p * total, l, kept);
    if (turn == 0) total = kept;
    border = found < border ? found : border;
    __syncthreads();
  }
  return border;
}

__global__ void __launch_bounds__(kDThreads) sample_pick_kernel(SampleArgs a) {
  __shared__ PickLds l;
  const Exp2 exp2;
  const int tid = threadIdx.x, wave = tid >> 6;
  for (int r = blockIdx.x; r < a.n_rows; r += gridDim.x) {
    const Settings s = settings_of(a, r);
    const float* row = a.logits + r * a.ldl;
    ChunkStat* st = chunk_stats(a) + static_cast<int64_t>(r) * a.chunks;
    float top = -INFINITY;
    int at = 0x7fffffff;
    if (!s.none) {
      for (int c = lane_id(); c < a.chunks; c += kWave) take_top(top, at, st[c].top, st[c].at);
      wave_top(top, at);
    }
    Pick pick{0, 0.0, s.rate, top, 0};
    int token = -1;
    double chosen = 0.0;
    if (top == -INFINITY) {                    // uniform
    } else if (s.greedy) {
      pick.border = place_of(top, at);
      pick.total = chosen = 1.0;
      token = at;
    } else {
      pick.border = s.filtered() ? border_of(a, exp2, row, r, s, top, l) : ~uint64_t(0);
      // the chunks' kept weights, relative to the row's top
      __syncthreads();
      if (s.filtered()) {
        for (int c = wave; c < a.chunks; c += kDWaves) {
          double sum = 0.0;
          for (int i = c * kChunk + 4 * lane_id(); i < (c + 1) * kChunk && i < a.vocab; i += 4 * kWave) {
            float v[4];
            load_quad(row, i, a.vocab, -INFINITY, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = taken(v[e]);
              if (place_of(x, i + e) <= pick.border) sum += weight(exp2, x, top, s.rate);
            }
          }
          sum = wave_sum(sum);
          if (lane_id() == 0) st[c].sum = sum;
        }
      } else {
        for (int c = tid; c < a.chunks; c += kDThreads) st[c].sum *= chunk_factor(exp2, st[c].top, top, s.rate);
      }
      __syncthreads();
      // the chunk in which the running sum passes the goal
      double sum = 0.0;
      for (int c = lane_id(); c < a.chunks; c += kWave) sum += st[c].sum;
      pick.total = wave_sum(sum);
      if (a.tokens || a.chosen) {
        const double goal = static_cast<double>(a.u[r]) * pick.total;
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
          w[e] = place_of(x, i0 + e) <= pick.border ? weight(exp2, x, top, s.rate) : 0.0;
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
        token = l.i0 != 0x7fffffff ? l.i0 : l.i1;
        if (token >= 0) chosen = weight(exp2, taken(row[token]), top, s.rate) / pick.total;
      }
    }
    if (tid == 0) {
      if (a.tokens) a.tokens[r] = token;
      if (a.chosen) a.chosen[r] = static_cast<float>(chosen);
      if (a.probs) picks(a)[r] = pick;
    }
    __syncthreads();                           // the row is done with LDS
  }
}

__global__ void __launch_bounds__(kSThreads) sample_probs_kernel(SampleArgs a) {
  const Exp2 exp2;
  for (int r = blockIdx.y; r < a.n_rows; r += gridDim.y) {
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
}

int launch_sample(const SampleArgs& a, hipStream_t st) {
  const unsigned chunks = static_cast<unsigned>(a.chunks), rows = a.n_rows < 65535 ? a.n_rows : 65535;
  hipLaunchKernelGGL(sample_stats_kernel, dim3(chunks, rows), dim3(kSThreads), 0, st, a);
  int rc = check_launch();
  if (rc) return rc;
  hipLaunchKernelGGL(sample_pick_kernel, dim3(rows), dim3(kDThreads), 0, st, a);
  rc = check_launch();
  if (rc || !a.probs) return rc;
  hipLaunchKernelGGL(sample_probs_kernel, dim3(chunks, rows), dim3(kSThreads), 0, st, a);
  return check_launch();
}

}  // namespace qmv
