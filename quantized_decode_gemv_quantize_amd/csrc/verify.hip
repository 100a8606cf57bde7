// verify.hip - verification of drafted tokens (speculative sampling).
//
// Launches over the target's rows, cut into chunks of kChunk logits:
//   stats    per row and chunk: largest logit, its lowest index, and the sum
//            of e_i = exp((l_i - largest) / T) (or of the weights);
//   decide   per sequence: the rows' sums joined over the chunks, and the
//            drafts accepted one after the other;
//   draw     per sequence: the chunk and then the index in which the running
//            sum of the weights passes u * total.
// Without draft probabilities decide and draw are one launch of a workgroup a
// sequence: the weights to draw from are e_i but for the refused token, so
// the chunks' sums are known but for one. With them, max(e_i - q_i Z, 0) has
// to be summed over the row first: the decide launch has a workgroup a chunk,
// each of which joins the sums for itself, and draw follows.
//
// Everything that a token depends on is in 64 bits: with 10^5 logits a
// running sum in 32 bits moves a border by more than the probability of many
// tokens. The stats launch reads every row once and is bound by that read
// with the exponentials beside it (21 64-bit operations each, 2^f by its
// Taylor polynomial): 141 rows of 128256 take 23 us, 3.1 TB/s, of which 16 are
// vector issue. The others are short chains of latencies (finish 12.3 us for
// 32 sequences, decide and draw 7.1 and 6.2 for one).
#include "decode_args.hpp"
#include "draw.hpp"
#include "launch.hpp"

namespace qmv {

constexpr int kVThreads = 512;
constexpr int kVWaves = kVThreads / kWave;
constexpr int kVPer = 8;                       // elements a lane
constexpr int kChunk = kVThreads * kVPer;
constexpr int kSThreads = 256;                 // the stats launch: fewer lanes with more elements each, as
constexpr int kSPer = kChunk / kSThreads;      // its reductions cost a wave what 7 elements a lane do
constexpr int kSWaves = kSThreads / kWave;

struct RowStat {
  float top;                                   // largest logit of the chunk
  int at;                                      // its lowest index
  double sum;                                  // sum of the weights relative to top
};
struct SeqSum {
  double rest, all;                            // of max(e - q Z, 0) and of e
};
struct Decision {
  int row, taken, last, best;                  // row drawn from (-1: none)
  float top;
  int token;                                   // refused there, -1 in a sequence's last row
  double z, refused;                           // sum of the row's weights, weight of the refused token
};

__device__ __forceinline__ RowStat* row_stats(const VerifyArgs& a) { return reinterpret_cast<RowStat*>(a.ws); }
__device__ __forceinline__ SeqSum* seq_sums(const VerifyArgs& a) {
  return reinterpret_cast<SeqSum*>(row_stats(a) + static_cast<int64_t>(a.n_rows) * a.chunks);
}
__device__ __forceinline__ Decision* decisions(const VerifyArgs& a) {
  return reinterpret_cast<Decision*>(seq_sums(a) + static_cast<int64_t>(a.n_seqs) * a.chunks);
}

int64_t verify_bytes(int n_seqs, int n_rows, int vocab, int* chunks) {
  const int64_t c = (vocab + kChunk - 1) / kChunk;
  if (chunks) *chunks = static_cast<int>(c);
  return n_rows * c * static_cast<int64_t>(sizeof(RowStat)) + n_seqs * c * static_cast<int64_t>(sizeof(SeqSum)) +
         n_seqs * static_cast<int64_t>(sizeof(Decision));
}

// A sequence's temperature: log2(e) / T, and whether it is greedy (T = +inf
// gives a rate of 0, too: a softmax of equal weights, not a greedy row).
struct Heat {
  double rate;
  bool greedy;
};
__device__ __forceinline__ Heat heat_of(const VerifyArgs& a, int s) {
  constexpr double kLog2e = 1.4426950408889634073599246810019;
  if (!a.temperature) return Heat{kLog2e, false};
  const float t = a.temperature[s];
  return Heat{t > 0.0f ? kLog2e / static_cast<double>(t) : 0.0, !(t > 0.0f)};
}

// Unnormalised weight of element i of a row whose largest logit is `top` (at
// its lowest index `best`).
__device__ __forceinline__ double weight(const VerifyArgs& a, const Exp2& exp2, float v, int i, float top, int best, Heat h) {
  if (a.kind == MMVQ_TARGET_WEIGHTS) return v > 0.0f && v < INFINITY ? static_cast<double>(v) : 0.0;
  if (h.greedy) return i == best ? 1.0 : 0.0;
  if (top == -INFINITY) return 0.0;            // nothing but -inf and NaN
  if (top == INFINITY) return v == top ? 1.0 : 0.0;
  return exp2((static_cast<double>(v) - static_cast<double>(top)) * h.rate);
}

// A probability of the draft; what is not positive counts as 0.
__device__ __forceinline__ double draft_weight(float q) { return q > 0.0f ? static_cast<double>(q) : 0.0; }

// The sequence that row r belongs to, -1 for none: the last one that starts
// at or before it. The 64 lanes probe 64 starts at a time.
__device__ __forceinline__ int sequence_of(const VerifyArgs& a, int r) {
  int lo = 0, hi = a.n_seqs;
  while (true) {
    const int step = (hi - lo + 63) / 64, i = lo + lane_id() * step;
    const uint64_t hit = __ballot(i < hi && a.row_start[i < hi ? i : lo] <= r);
    if (hit == 0) return -1;
    lo += (63 - __builtin_clzll(hit)) * step;
    if (step == 1) break;
    hi = lo + step < hi ? lo + step : hi;
  }
  return r < a.row_start[lo + 1] ? lo : -1;
}

// Rows of a sequence, inside the buffers.
__device__ __forceinline__ void seq_rows(const VerifyArgs& a, int s, int& first, int& count) {
  const int b = a.row_start[s], e = a.row_start[s + 1];
  first = b < 0 ? 0 : b > a.n_rows ? a.n_rows : b;
  const int end = e > a.n_rows ? a.n_rows : e;
  count = end > first ? end - first : 0;
}

// exp(chunk_top - top) of two largest logits, the factor between their sums.
__device__ __forceinline__ double chunk_scale(const VerifyArgs& a, const Exp2& exp2, float chunk_top, float top, Heat h) {
  if (a.kind == MMVQ_TARGET_WEIGHTS || chunk_top == top) return 1.0;
  if (!(chunk_top > -INFINITY) || top == INFINITY) return 0.0;
  return exp2((static_cast<double>(chunk_top) - static_cast<double>(top)) * h.rate);
}

// Each wave sums relative to its own largest logit; one wave joins the four.
template <bool LOGITS>
__global__ void __launch_bounds__(kSThreads) verify_stats_kernel(VerifyArgs a) {
  __shared__ RowStat st[kSWaves];
  const Exp2 exp2;
  const int tid = threadIdx.x, wave = tid >> 6, c = blockIdx.x, i0 = c * kChunk + 4 * tid;
  for (int r = blockIdx.y; r < a.n_rows; r += gridDim.y) {
    const float* row = a.target + r * a.ldt;
    float v[kSPer];
    if ((c + 1) * kChunk <= a.vocab) {         // uniform: all loads at once
#pragma unroll
      for (int k = 0; k < kSPer; k += 4) {
        const u32x4 x = ld_x4(reinterpret_cast<const uint8_t*>(row + i0 + k * kSThreads));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k + e] = __uint_as_float(x[e]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kSPer; ++k) {
        const int i = i0 + (k / 4) * 4 * kSThreads + k % 4;
        v[k] = row[i < a.vocab ? i : a.vocab - 1];
        v[k] = i < a.vocab ? v[k] : -INFINITY;
      }
    }
    const int s = sequence_of(a, r);
    if (s < 0) continue;                       // uniform: every wave finds the same
    RowStat own{-INFINITY, 0x7fffffff, 0.0};
    bool greedy = false;
    Heat h{0.0, false};
    if constexpr (LOGITS) {
      h = heat_of(a, s);
      greedy = h.greedy;
#pragma unroll
      for (int k = 0; k < kSPer; ++k) own.top = fmaxf(own.top, v[k]);
#pragma unroll
      for (int k = kSPer - 1; k >= 0; --k)
        own.at = v[k] == own.top && own.top > -INFINITY ? i0 + (k / 4) * 4 * kSThreads + k % 4 : own.at;
      wave_top(own.top, own.at);
      if (!greedy && own.top > -INFINITY) {
        if (own.top < INFINITY) {
          const double top = static_cast<double>(own.top);
#pragma unroll
          for (int k = 0; k < kSPer; ++k) own.sum += exp2((static_cast<double>(v[k]) - top) * h.rate);
        } else {
#pragma unroll
          for (int k = 0; k < kSPer; ++k) own.sum += v[k] == own.top ? 1.0 : 0.0;
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < kSPer; ++k) own.sum += v[k] > 0.0f && v[k] < INFINITY ? static_cast<double>(v[k]) : 0.0;
    }
    if (!greedy) own.sum = wave_sum(own.sum);
    __syncthreads();                           // the row before is joined
    if ((tid & 63) == 0) st[wave] = own;
    __syncthreads();
    if (wave == 0) {
      const RowStat o = st[tid & (kSWaves - 1)];
      RowStat all{o.top, o.at, 0.0};
      if constexpr (LOGITS) wave_top(all.top, all.at);
      all.sum = wave_sum(tid < kSWaves ? o.sum * chunk_scale(a, exp2, o.top, all.top, h) : 0.0);
      if (tid == 0) row_stats(a)[static_cast<int64_t>(r) * a.chunks + c] = all;
    }
  }
}

// A row's chunks joined, by one wave: the same in all lanes; `mine` is the
// lane's chunk's part of z (not for a greedy row).
__device__ __forceinline__ void join_row(const VerifyArgs& a, const Exp2& exp2, int r, Heat h, float& top, int& at, double& z,
                                         double& mine) {
  const RowStat* st = row_stats(a) + static_cast<int64_t>(r) * a.chunks;
  top = -INFINITY;
  at = 0x7fffffff;
  z = 0.0;
  const RowStat none{-INFINITY, 0x7fffffff, 0.0}, own = lane_id() < a.chunks ? st[lane_id()] : none;
  if (a.kind == MMVQ_TARGET_LOGITS) {
    take_top(top, at, own.top, own.at);
    for (int c = lane_id() + kWave; c < a.chunks; c += kWave) take_top(top, at, st[c].top, st[c].at);
    wave_top(top, at);
  }
  mine = 0.0;
  if (h.greedy) {
    z = top > -INFINITY ? 1.0 : 0.0;
    return;
  }
  z = mine = own.sum * chunk_scale(a, exp2, own.top, top, h);
  for (int c = lane_id() + kWave; c < a.chunks; c += kWave) z += st[c].sum * chunk_scale(a, exp2, st[c].top, top, h);
  z = wave_sum(z);
}

// The weight to draw from and the plain one, of element i of the decided row.
__device__ __forceinline__ void draw_weights(const VerifyArgs& a, const Exp2& exp2, const Decision& d, Heat h, int x, float v,
                                             float q, int i, double& rest, double& all) {
  all = weight(a, exp2, v, i, d.top, d.best, h);
  if (a.draft_probs) rest = fmax(all - draft_weight(q) * d.z, 0.0);
  else rest = i == x ? 0.0 : all;              // q is 1 there, and e_i <= Z
}

// Accepts the drafts of sequence s in order; the whole workgroup. Rows eight
// at a time, one a wave.
struct DecideLds {
  Decision dec;
  int ok[kVWaves], ats[kVWaves], tokens[kVWaves], slot;   // slot: wave that had the decided row
  float tops[kVWaves];
  double zs[kVWaves], es[kVWaves];
  double sums[kVWaves][kWave];                 // parts of z of each wave's row, of its first 64 chunks
};
__device__ __forceinline__ void decide(const VerifyArgs& a, const Exp2& exp2, int first, int count, Heat h, DecideLds& l) {
  const int tid = threadIdx.x, wave = tid >> 6;
  __syncthreads();                             // the sequence before is done with LDS
  if (tid == 0) {
    l.dec.row = -1;
    l.dec.taken = 0;
    l.dec.last = 0;
  }
  bool open = true;                            // uniform: every draft so far accepted
  for (int i0 = 0; i0 < count && open; i0 += kVWaves) {
    const int i = i0 + wave, r = first + i;
    if (i < count) {
      // the draft's own values are on their way while the sums are joined
      const bool drafted = i + 1 < count;
      const int x = drafted ? a.draft_tokens[r] : -1;
      const bool real = x >= 0 && x < a.vocab;
      const float v = a.target[r * a.ldt + (real ? x : 0)];
      const float q = a.draft_probs && real ? a.draft_probs[r * a.ldd + x] : 1.0f, u = drafted ? a.u_accept[r] : 0.0f;
      float top;
      int at;
      double z, mine;
      join_row(a, exp2, r, h, top, at, z, mine);
      l.sums[wave][tid & 63] = mine;
      const double e = real ? weight(a, exp2, v, x, top, at, h) : 0.0;
      const bool yes = real && static_cast<double>(u) * draft_weight(q) * z < e;
      if ((tid & 63) == 0) {
        l.ok[wave] = yes && z > 0.0 && z < INFINITY;
        l.tops[wave] = top;
        l.ats[wave] = at;
        l.tokens[wave] = x;
        l.zs[wave] = z;
        l.es[wave] = e;
      }
    }
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < kVWaves && i0 + w < count; ++w) {
        if (l.ok[w]) {
          ++l.dec.taken;
          continue;
        }
        const bool valid = l.zs[w] > 0.0 && l.zs[w] < INFINITY;
        l.dec.row = valid ? first + i0 + w : -2;
        l.dec.last = i0 + w + 1 == count;
        l.dec.top = l.tops[w];
        l.dec.best = l.ats[w];
        l.dec.token = l.tokens[w];
        l.slot = w;
        l.dec.z = l.zs[w];
        l.dec.refused = l.es[w];
        break;
      }
    }
    __syncthreads();
    open = l.dec.row == -1;
  }
  __syncthreads();
}

// Sums of a chunk's weights over the workgroup.
__device__ __forceinline__ SeqSum chunk_sums(const VerifyArgs& a, const Exp2& exp2, const Decision& d, Heat h, int x, int c,
                                             double* lds) {
  const int tid = threadIdx.x, wave = tid >> 6;
  double rest = 0.0, all = 0.0;
#pragma unroll
  for (int k = 0; k < kVPer / 4; ++k) {
    const int i = c * kChunk + 4 * (k * kVThreads + tid);
    float v[4], q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    load_quad(a.target + d.row * a.ldt, i, a.vocab, -INFINITY, v);
    if (a.draft_probs && !d.last) load_quad(a.draft_probs + d.row * a.ldd, i, a.vocab, 0.0f, q);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      double re, al;
      draw_weights(a, exp2, d, h, x, v[e], q[e], i + e, re, al);
      rest += re;
      all += al;
    }
  }
  rest = wave_sum(rest);
  all = wave_sum(all);
  if ((tid & 63) == 0) {
    lds[2 * wave] = rest;
    lds[2 * wave + 1] = all;
  }
  __syncthreads();
  SeqSum sum{0.0, 0.0};
#pragma unroll
  for (int w = 0; w < kVWaves; ++w) {
    sum.rest += lds[2 * w];
    sum.all += lds[2 * w + 1];
  }
  return sum;
}

struct DrawLds {
  double wsum[kVWaves], before, goal;
  int chunk, rest, hit, last;
};
// Draws from the decided row with the number u; sums(c): the chunks' sums.
// The whole workgroup.
template <class S>
__device__ __forceinline__ int draw(const VerifyArgs& a, const Exp2& exp2, const Decision& d, Heat h, float u, int x, S sums,
                                    DrawLds& l) {
  const int tid = threadIdx.x, wave = tid >> 6;
  if (wave == 0) {
    const SeqSum none{0.0, 0.0}, own = lane_id() < a.chunks ? sums(lane_id()) : none;
    double rest = own.rest, all = own.all;
    for (int c = lane_id() + kWave; c < a.chunks; c += kWave) {
      const SeqSum o = sums(c);
      rest += o.rest;
      all += o.all;
    }
    rest = wave_sum(rest);
    all = wave_sum(all);
    const bool use = !d.last && rest > 0.0;
    const double goal = static_cast<double>(u) * (use ? rest : all);
    // first chunk in which the running sum passes the goal; behind the last
    // border, the last chunk that has a weight
    double run = 0.0, before = 0.0, last_before = 0.0;
    int found = -1, last = 0;
    for (int c0 = 0; c0 < a.chunks && found < 0; c0 += kWave) {
      const int c = c0 + lane_id();
      const SeqSum o = c0 == 0 ? own : c < a.chunks ? sums(c) : none;
      const double w = use ? o.rest : o.all;
      const double row_up = wave_scan(w), up = row_up + run, ahead = wave_before(row_up) + run;
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
    if (lane_id() == 0) {
      l.chunk = found >= 0 ? found : last;
      l.before = found >= 0 ? before : last_before;
      l.goal = goal;
      l.rest = use;
      l.hit = 0x7fffffff;
      l.last = -1;
    }
  }
  __syncthreads();
  // the chunk again, a run of consecutive elements a lane
  const int base = l.chunk * kChunk + kVPer * tid;
  double w[kVPer], own = 0.0;
#pragma unroll
  for (int k = 0; k < kVPer; k += 4) {
    float v[4], q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    load_quad(a.target + d.row * a.ldt, base + k, a.vocab, -INFINITY, v);
    if (a.draft_probs && !d.last) load_quad(a.draft_probs + d.row * a.ldd, base + k, a.vocab, 0.0f, q);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      double re, al;
      draw_weights(a, exp2, d, h, x, v[e], q[e], base + k + e, re, al);
      w[k + e] = l.rest ? re : al;
      own += w[k + e];
    }
  }
  const double up = wave_scan(own);
  if ((tid & 63) == 63) l.wsum[wave] = up;
  __syncthreads();
  double run = l.before + wave_before(up);
  for (int v = 0; v < wave; ++v) run += l.wsum[v];
  int hit = 0x7fffffff, last = -1;
#pragma unroll
  for (int k = 0; k < kVPer; ++k) {
    run += w[k];
    if (w[k] > 0.0) {
      last = base + k;
      if (run > l.goal && hit == 0x7fffffff) hit = base + k;
    }
  }
  if (hit != 0x7fffffff) atomicMin(&l.hit, hit);
  if (last >= 0) atomicMax(&l.last, last);
  __syncthreads();
  return l.hit != 0x7fffffff ? l.hit : l.last;
}

// The drafted token that this lane will put out, if it is accepted.
__device__ __forceinline__ int own_draft(const VerifyArgs& a, int first, int count) {
  const int tid = threadIdx.x;
  return tid + 1 < count ? a.draft_tokens[first + tid] : -1;   // (the last row has none)
}
__device__ __forceinline__ void put_tokens(const VerifyArgs& a, int s, int first, int taken, int token, int own) {
  for (int i = threadIdx.x; i < a.max_out; i += kVThreads)
    a.tokens[static_cast<int64_t>(s) * a.max_out + i] =
        i < taken ? (i < kVThreads ? own : a.draft_tokens[first + i]) : i == taken ? token : -1;
  if (threadIdx.x == 0) a.n_accepted[s] = taken;
}

// With draft probabilities: the decision, and the sums to draw from.
__global__ void __launch_bounds__(kVThreads) verify_decide_kernel(VerifyArgs a) {
  const Exp2 exp2;
  __shared__ DecideLds l;
  __shared__ double lds[2 * kVWaves];
  const int tid = threadIdx.x, c = blockIdx.x;
  for (int s = blockIdx.y; s < a.n_seqs; s += gridDim.y) {
    int first, count;
    seq_rows(a, s, first, count);
    const Heat h = heat_of(a, s);
    decide(a, exp2, first, count, h, l);
    const Decision d = l.dec;
    if (c == 0 && tid == 0) decisions(a)[s] = d;
    if (d.row < 0) continue;                   // uniform; (decide waits for the sequence before)
    const SeqSum sum = chunk_sums(a, exp2, d, h, d.token, c, lds);
    if (tid == 0) seq_sums(a)[static_cast<int64_t>(s) * a.chunks + c] = sum;
  }
}

__global__ void __launch_bounds__(kVThreads) verify_draw_kernel(VerifyArgs a) {
  const Exp2 exp2;
  __shared__ DrawLds l;
  for (int s = blockIdx.x; s < a.n_seqs; s += gridDim.x) {
    const Decision d = decisions(a)[s];
    int first, count, token = -1;
    seq_rows(a, s, first, count);
    const SeqSum* cs = seq_sums(a) + static_cast<int64_t>(s) * a.chunks;
    const Heat h = heat_of(a, s);
    const float u = a.u_sample[s];
    const int own = own_draft(a, first, count);
    __syncthreads();                           // the sequence before is done with LDS
    if (d.row >= 0)                            // uniform
      token = draw(a, exp2, d, h, u, d.token, [&](int c) QMV_INLINE { return cs[c]; }, l);
    put_tokens(a, s, first, d.taken, token, own);
  }
}

// Without draft probabilities: decision and draw. Of the chunks' sums only
// that of the refused token's changes. Its difference is off by 2^-53 of the
// sum: where less than 2^-10 of the chunk is left, that is summed again.
__global__ void __launch_bounds__(kVThreads) verify_finish_kernel(VerifyArgs a) {
  const Exp2 exp2;
  __shared__ DecideLds l;
  __shared__ DrawLds dl;
  __shared__ double lds[2 * kVWaves];
  for (int s = blockIdx.x; s < a.n_seqs; s += gridDim.x) {
    int first, count, token = -1;
    seq_rows(a, s, first, count);
    const Heat h = heat_of(a, s);
    const float u = a.u_sample[s];
    const int own = own_draft(a, first, count);
    decide(a, exp2, first, count, h, l);
    const Decision d = l.dec;
    if (d.row >= 0) {                          // uniform
      const int x = d.token, cx = x >= 0 && x < a.vocab ? x / kChunk : -1;
      const double* parts = l.sums[l.slot];
      const RowStat* st = row_stats(a) + static_cast<int64_t>(d.row) * a.chunks;
      const auto sum_of = [&](int c) QMV_INLINE {
        if (h.greedy) return d.best / kChunk == c ? 1.0 : 0.0;
        if (a.chunks <= kWave) return parts[c];
        return st[c].sum * chunk_scale(a, exp2, st[c].top, d.top, h);
      };
      double left = 0.0;
      if (cx >= 0) {
        const double all = sum_of(cx);
        left = all - d.refused;
        if (left < 0x1p-10 * all) left = chunk_sums(a, exp2, d, h, x, cx, lds).rest;
      }
      token = draw(a, exp2, d, h, u, x, [&](int c) QMV_INLINE {
        const double all = sum_of(c);
        return SeqSum{c == cx ? left : all, all};
      }, dl);
    }
    put_tokens(a, s, first, d.taken, token, own);
  }
}

int launch_verify(const VerifyArgs& a, hipStream_t st) {
  const unsigned chunks = static_cast<unsigned>(a.chunks);
  const unsigned rows = a.n_rows < 65535 ? a.n_rows : 65535, seqs = a.n_seqs < 65535 ? a.n_seqs : 65535;
  if (rows > 0) {
    if (a.kind == MMVQ_TARGET_LOGITS)
      hipLaunchKernelGGL((verify_stats_kernel<true>), dim3(chunks, rows), dim3(kSThreads), 0, st, a);
    else
      hipLaunchKernelGGL((verify_stats_kernel<false>), dim3(chunks, rows), dim3(kSThreads), 0, st, a);
    const int rc = check_launch();
    if (rc) return rc;
  }
  if (!a.draft_probs) {
    hipLaunchKernelGGL(verify_finish_kernel, dim3(seqs), dim3(kVThreads), 0, st, a);
    return check_launch();
  }
  hipLaunchKernelGGL(verify_decide_kernel, dim3(chunks, seqs), dim3(kVThreads), 0, st, a);
  const int rc = check_launch();
  if (rc) return rc;
  hipLaunchKernelGGL(verify_draw_kernel, dim3(seqs), dim3(kVThreads), 0, st, a);
  return check_launch();
}

}  // namespace qmv
