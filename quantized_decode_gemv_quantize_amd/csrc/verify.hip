// verify.hip - verification of drafted tokens (speculative sampling).
//
// Three launches over the target's rows, cut into chunks of kChunk logits:
//   stats    per row and chunk: largest logit, its lowest index, and the sum
//            of e_i = exp((l_i - largest) / T) (or of the weights);
//   decide   per sequence: the rows' sums joined over the chunks, the drafts
//            accepted one after the other, and per chunk the sums of the
//            weights to draw from, max(e_i - q_i Z, 0) and e_i;
//   draw     per sequence: the chunk and then the index in which the running
//            sum passes u * total.
// Everything that a token depends on is in 64 bits: with 10^5 logits a
// running sum in 32 bits moves a border by more than the probability of many
// tokens. The stats launch reads every row once and is bound by that read
// and by the 64-bit exponentials; the other two read one row a sequence
// again, mostly from cache.
#include "decode_args.hpp"
#include "launch.hpp"

namespace qmv {

constexpr int kVThreads = 256;
constexpr int kVPer = 8;                       // elements a lane
constexpr int kChunk = kVThreads * kVPer;

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
  int pad;
  double z, inv_t;                             // inv_t 0: greedy
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

// 1/T of a sequence; 0 for a greedy one.
__device__ __forceinline__ double inv_temperature(const VerifyArgs& a, int s) {
  if (!a.temperature) return 1.0;
  const float t = a.temperature[s];
  return t > 0.0f ? 1.0 / static_cast<double>(t) : 0.0;
}
// T = +inf gives 1/T = 0, too: a softmax of equal weights, not a greedy row.
__device__ __forceinline__ bool greedy(const VerifyArgs& a, int s) {
  return a.kind == MMVQ_TARGET_LOGITS && a.temperature && !(a.temperature[s] > 0.0f);
}

// Unnormalised weight of element i of a row whose largest logit is `top` (at
// its lowest index `best`).
__device__ __forceinline__ double weight(const VerifyArgs& a, float v, int i, float top, int best, double inv_t,
                                         bool greedy_row) {
  if (a.kind == MMVQ_TARGET_WEIGHTS) return v > 0.0f && v < INFINITY ? static_cast<double>(v) : 0.0;
  if (greedy_row) return i == best ? 1.0 : 0.0;
  if (!(v > -INFINITY)) return 0.0;            // -inf, NaN
  if (v == top) return 1.0;                    // +inf among them
  if (top == INFINITY) return 0.0;
  return exp((static_cast<double>(v) - static_cast<double>(top)) * inv_t);
}

// A probability of the draft; what is not positive counts as 0.
__device__ __forceinline__ double draft_weight(float q) { return q > 0.0f ? static_cast<double>(q) : 0.0; }

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
  return v;
}
__device__ __forceinline__ void wave_top(float& top, int& at) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    const float t = __shfl_xor(top, m);
    const int i = __shfl_xor(at, m);
    if (t > top || (t == top && i < at)) { top = t; at = i; }
  }
}

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

// Four elements at i, `fill` behind the row's end.
__device__ __forceinline__ void load_quad(const float* row, int i, int n, float fill, float (&v)[4]) {
  if (i + 4 <= n) {
    const u32x4 r = ld_x4(reinterpret_cast<const uint8_t*>(row + i));
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(r[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = i + e < n ? row[i + e] : fill;
  }
}

__global__ void __launch_bounds__(kVThreads) verify_stats_kernel(VerifyArgs a) {
  __shared__ float tops[4];
  __shared__ int ats[4];
  __shared__ double sums[4];
  const int tid = threadIdx.x, wave = tid >> 6, c = blockIdx.x;
  for (int r = blockIdx.y; r < a.n_rows; r += gridDim.y) {
    float v[kVPer];
#pragma unroll
    for (int k = 0; k < kVPer / 4; ++k) {
      float t[4];
      load_quad(a.target + r * a.ldt, c * kChunk + 4 * (k * kVThreads + tid), a.vocab, -INFINITY, t);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * k + e] = t[e];
    }
    const int s = sequence_of(a, r);
    if (s < 0) continue;                       // uniform: every wave finds the same
    float top = -INFINITY;
    int at = 0x7fffffff;
#pragma unroll
    for (int k = 0; k < kVPer; ++k) {
      const int i = c * kChunk + 4 * ((k / 4) * kVThreads + tid) + k % 4;
      if (v[k] > top) { top = v[k]; at = i; }
    }
    double sum = 0.0;
    if (a.kind == MMVQ_TARGET_LOGITS) {
      wave_top(top, at);
      __syncthreads();                         // the row before is written
      if ((tid & 63) == 0) { tops[wave] = top; ats[wave] = at; }
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 4; ++w)
        if (tops[w] > top || (tops[w] == top && ats[w] < at)) { top = tops[w]; at = ats[w]; }
    } else {
      __syncthreads();
    }
    const bool gr = greedy(a, s);
    const double inv_t = inv_temperature(a, s);
    if (!gr) {
#pragma unroll
      for (int k = 0; k < kVPer; ++k) sum += weight(a, v[k], 0, top, 0, inv_t, false);
      sum = wave_sum(sum);
      if ((tid & 63) == 0) sums[wave] = sum;
    }
    __syncthreads();
    if (tid == 0) {
      RowStat st;
      st.top = top;
      st.at = at;
      st.sum = gr ? 0.0 : sums[0] + sums[1] + sums[2] + sums[3];
      row_stats(a)[static_cast<int64_t>(r) * a.chunks + c] = st;
    }
  }
}

// A row's chunks joined, by one wave: the same in all lanes.
__device__ __forceinline__ void join_row(const VerifyArgs& a, int r, double inv_t, bool gr, float& top, int& at, double& z) {
  const RowStat* st = row_stats(a) + static_cast<int64_t>(r) * a.chunks;
  top = -INFINITY;
  at = 0x7fffffff;
  z = 0.0;
  if (a.kind == MMVQ_TARGET_LOGITS) {
    for (int c = lane_id(); c < a.chunks; c += kWave)
      if (st[c].top > top) { top = st[c].top; at = st[c].at; }
    wave_top(top, at);
  }
  if (gr) {
    z = top > -INFINITY ? 1.0 : 0.0;
    return;
  }
  for (int c = lane_id(); c < a.chunks; c += kWave) {
    if (a.kind == MMVQ_TARGET_WEIGHTS) z += st[c].sum;
    else if (st[c].top > -INFINITY && (st[c].top == top || top < INFINITY))
      z += st[c].top == top ? st[c].sum
                            : st[c].sum * exp((static_cast<double>(st[c].top) - static_cast<double>(top)) * inv_t);
  }
  z = wave_sum(z);
}

// The weight to draw from and the plain one, of element i of the decided row.
__device__ __forceinline__ void draw_weights(const VerifyArgs& a, const Decision& d, bool gr, int x, float v, float q,
                                             int i, double& rest, double& all) {
  all = weight(a, v, i, d.top, d.best, d.inv_t, gr);
  const double off = a.draft_probs ? draft_weight(q) * d.z : i == x ? d.z : 0.0;
  rest = all - off;
  rest = rest > 0.0 ? rest : 0.0;
}

__global__ void __launch_bounds__(kVThreads) verify_decide_kernel(VerifyArgs a) {
  __shared__ Decision dec;
  __shared__ int ok[4];
  __shared__ float tops[4];
  __shared__ int ats[4];
  __shared__ double zs[4], sums[8];
  const int tid = threadIdx.x, wave = tid >> 6, c = blockIdx.x;
  for (int s = blockIdx.y; s < a.n_seqs; s += gridDim.y) {
    int first, count;
    seq_rows(a, s, first, count);
    const bool gr = greedy(a, s);
    const double inv_t = inv_temperature(a, s);
    __syncthreads();
    if (tid == 0) {
      dec.row = -1;
      dec.taken = 0;
      dec.last = 0;
      dec.inv_t = inv_t;
    }
    bool open = true;                          // uniform: every draft so far accepted
    for (int i0 = 0; i0 < count && open; i0 += 4) {
      const int i = i0 + wave, r = first + i;
      if (i < count) {
        float top;
        int at;
        double z;
        join_row(a, r, inv_t, gr, top, at, z);
        bool yes = false;
        if (i + 1 < count) {
          const int x = a.draft_tokens[r];
          if (x >= 0 && x < a.vocab) {
            const double e = weight(a, a.target[r * a.ldt + x], x, top, at, inv_t, gr);
            const double q = a.draft_probs ? draft_weight(a.draft_probs[r * a.ldd + x]) : 1.0;
            yes = static_cast<double>(a.u_accept[r]) * q * z < e;
          }
        }
        if ((tid & 63) == 0) {
          ok[wave] = yes && z > 0.0 && z < INFINITY;
          tops[wave] = top;
          ats[wave] = at;
          zs[wave] = z;
        }
      }
      __syncthreads();
      if (tid == 0) {
        for (int w = 0; w < 4 && i0 + w < count; ++w) {
          if (ok[w]) {
            ++dec.taken;
            continue;
          }
          const bool valid = zs[w] > 0.0 && zs[w] < INFINITY;
          dec.row = valid ? first + i0 + w : -2;
          dec.last = i0 + w + 1 == count;
          dec.top = tops[w];
          dec.best = ats[w];
          dec.z = zs[w];
          break;
        }
      }
      __syncthreads();
      open = dec.row == -1;
    }
    __syncthreads();
    const Decision d = dec;
    if (c == 0 && tid == 0) decisions(a)[s] = d;
    double rest = 0.0, all = 0.0;
    if (d.row >= 0) {
      const int x = d.last ? -1 : a.draft_tokens[d.row];
#pragma unroll
      for (int k = 0; k < kVPer / 4; ++k) {
        const int i = c * kChunk + 4 * (k * kVThreads + tid);
        float v[4], q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        load_quad(a.target + d.row * a.ldt, i, a.vocab, -INFINITY, v);
        if (a.draft_probs && !d.last) load_quad(a.draft_probs + d.row * a.ldd, i, a.vocab, 0.0f, q);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          double re, al;
          draw_weights(a, d, gr, x, v[e], q[e], i + e, re, al);
          rest += re;
          all += al;
        }
      }
    }
    rest = wave_sum(rest);
    all = wave_sum(all);
    if ((tid & 63) == 0) {
      sums[2 * wave] = rest;
      sums[2 * wave + 1] = all;
    }
    __syncthreads();
    if (tid == 0) {
      SeqSum ss;
      ss.rest = sums[0] + sums[2] + sums[4] + sums[6];
      ss.all = sums[1] + sums[3] + sums[5] + sums[7];
      seq_sums(a)[static_cast<int64_t>(s) * a.chunks + c] = ss;
    }
  }
}

__device__ __forceinline__ double wave_scan(double v) {   // inclusive
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) {
    const double o = __shfl_up(v, m);
    if (lane_id() >= m) v += o;
  }
  return v;
}

__global__ void __launch_bounds__(kVThreads) verify_draw_kernel(VerifyArgs a) {
  __shared__ double wsum[4], before_s, goal_s;
  __shared__ int chunk_s, rest_s, hit_s, last_s;
  const int tid = threadIdx.x, wave = tid >> 6;
  for (int s = blockIdx.x; s < a.n_seqs; s += gridDim.x) {
    const Decision d = decisions(a)[s];
    int first, count;
    seq_rows(a, s, first, count);
    const bool gr = greedy(a, s);
    const SeqSum* cs = seq_sums(a) + static_cast<int64_t>(s) * a.chunks;
    int token = -1;
    if (d.row >= 0) {                          // uniform
      __syncthreads();
      if (wave == 0) {
        double rest = 0.0, all = 0.0;
        for (int c = lane_id(); c < a.chunks; c += kWave) {
          rest += cs[c].rest;
          all += cs[c].all;
        }
        rest = wave_sum(rest);
        all = wave_sum(all);
        const bool use = !d.last && rest > 0.0;
        const double goal = static_cast<double>(a.u_sample[s]) * (use ? rest : all);
        // first chunk in which the running sum passes the goal; behind the
        // last border, the last chunk that has a weight
        double run = 0.0, before = 0.0, last_before = 0.0;
        int found = -1, last = 0;
        for (int c0 = 0; c0 < a.chunks && found < 0; c0 += kWave) {
          const int c = c0 + lane_id();
          const double w = c < a.chunks ? (use ? cs[c].rest : cs[c].all) : 0.0;
          const double up = wave_scan(w) + run;
          const uint64_t hit = __ballot(up > goal), some = __ballot(w > 0.0);
          if (some) {
            const int l = 63 - __builtin_clzll(some);
            last = c0 + l;
            last_before = __shfl(up - w, l);
          }
          if (hit) {
            const int l = __builtin_ctzll(hit);
            found = c0 + l;
            before = __shfl(up - w, l);
          }
          run = __shfl(up, kWave - 1);
        }
        if (lane_id() == 0) {
          chunk_s = found >= 0 ? found : last;
          before_s = found >= 0 ? before : last_before;
          goal_s = goal;
          rest_s = use;
          hit_s = 0x7fffffff;
          last_s = -1;
        }
      }
      __syncthreads();
      // the chunk again, a run of consecutive elements a lane
      const int base = chunk_s * kChunk + kVPer * tid, x = d.last ? -1 : a.draft_tokens[d.row];
      double w[kVPer], own = 0.0;
#pragma unroll
      for (int k = 0; k < kVPer; k += 4) {
        float v[4], q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        load_quad(a.target + d.row * a.ldt, base + k, a.vocab, -INFINITY, v);
        if (a.draft_probs && !d.last) load_quad(a.draft_probs + d.row * a.ldd, base + k, a.vocab, 0.0f, q);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          double re, al;
          draw_weights(a, d, gr, x, v[e], q[e], base + k + e, re, al);
          w[k + e] = rest_s ? re : al;
          own += w[k + e];
        }
      }
      const double up = wave_scan(own);
      if ((tid & 63) == 63) wsum[wave] = up;
      __syncthreads();
      double run = before_s + (up - own);
      for (int v = 0; v < wave; ++v) run += wsum[v];
      int hit = 0x7fffffff, last = -1;
#pragma unroll
      for (int k = 0; k < kVPer; ++k) {
        run += w[k];
        if (w[k] > 0.0) {
          last = base + k;
          if (run > goal_s && hit == 0x7fffffff) hit = base + k;
        }
      }
      if (hit != 0x7fffffff) atomicMin(&hit_s, hit);
      if (last >= 0) atomicMax(&last_s, last);
      __syncthreads();
      token = hit_s != 0x7fffffff ? hit_s : last_s;
    }
    for (int i = tid; i < a.max_out; i += kVThreads)
      a.tokens[static_cast<int64_t>(s) * a.max_out + i] =
          i < d.taken ? a.draft_tokens[first + i] : i == d.taken ? token : -1;
    if (tid == 0) a.n_accepted[s] = d.taken;
  }
}

int launch_verify(const VerifyArgs& a, hipStream_t st) {
  const unsigned chunks = static_cast<unsigned>(a.chunks);
  const unsigned rows = a.n_rows < 65535 ? a.n_rows : 65535, seqs = a.n_seqs < 65535 ? a.n_seqs : 65535;
  if (rows > 0) {
    hipLaunchKernelGGL(verify_stats_kernel, dim3(chunks, rows), dim3(kVThreads), 0, st, a);
    const int rc = check_launch();
    if (rc) return rc;
  }
  hipLaunchKernelGGL(verify_decide_kernel, dim3(chunks, seqs), dim3(kVThreads), 0, st, a);
  const int rc = check_launch();
  if (rc) return rc;
  hipLaunchKernelGGL(verify_draw_kernel, dim3(seqs), dim3(kVThreads), 0, st, a);
  return check_launch();
}

}  // namespace qmv
