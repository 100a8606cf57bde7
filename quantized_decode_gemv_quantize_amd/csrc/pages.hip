// pages.hip - page tables of many requests: pages given back, and a step's
// pages, descriptor arrays and row maps from the requests' lengths.
//
//   start = running sum of the new tokens; want[s] = max(0, ceil(len / page) -
//   held) for requests with new tokens; off = running sum of want; entry
//   held + i of request s is free page n_free - given + off[s] + i.
//
// Sums go over requests (one workgroup, 1024 at a time); rows and pages find
// their request by bisection in the running sums, in LDS up to 1024 requests.
// All of it is a chain of latencies: two scans, ten steps of a bisection, a
// table entry. Up to kPlanRows rows one workgroup does everything in one
// launch (64 requests, 318 rows: 4.0 us); more rows take a second launch over
// all of them (512 requests, 58 336 rows, 0.9 MB of maps: 2.7 + 5.5 us).
#include "draw.hpp"
#include "launch.hpp"
#include "serve_args.hpp"

namespace qmv {

constexpr int kPThreads = 1024;
constexpr int kPWaves = kPThreads / kWave;
constexpr int kPlanRows = 4096;                // rows that one workgroup maps beside the sums
constexpr int kFThreads = 256;

// Sum of the values of the lanes before this one over the workgroup (they and
// their sum below 2^31), and the sum of all. lds: kPWaves numbers that no
// other scan uses before the next barrier.
__device__ __forceinline__ int block_scan(int v, int* lds, int& total) {
  const int wave = threadIdx.x >> 6, up = wave_scan(v);
  if (lane_id() == kWave - 1) lds[wave] = up;
  __syncthreads();
  const int part = lane_id() < kPWaves ? lds[lane_id()] : 0, sums = wave_scan(part);
  total = __builtin_amdgcn_readlane(sums, kPWaves - 1);
  const int before = __shfl(sums - part, wave);
  return before + up - v;
}

__device__ __forceinline__ int clamp_to(int v, int most) { return v < 0 ? 0 : v > most ? most : v; }

// Pages of the request that a position's length needs, at most its table's.
__device__ __forceinline__ int pages_of(const PoolArgs& p, int64_t len) {
  const int64_t n = (len + (int64_t(1) << p.shift) - 1) >> p.shift;
  return n < p.pages_per_seq ? static_cast<int>(n) : p.pages_per_seq;
}

// Largest s < n with sums[s] <= v (sums[0] <= v).
template <class T>
__device__ __forceinline__ int bisect(const T* sums, int n, int64_t v) {
  int at = 0;
  for (int step = 1 << (31 - __builtin_clz(n)); step > 0; step >>= 1)
    if (at + step < n && sums[at + step] <= v) at += step;
  return at;
}

struct Given {
  int64_t pages;           // of those needed
  int before;              // free pages before the step
};
__device__ __forceinline__ int page_taken(const PlanArgs& a, Given g, int64_t i) {
  return i < g.pages ? a.p.free[g.before - g.pages + i] : -1;
}

// Table entries and row maps, by `threads` threads of which this is number
// `tid`. start, off: n_seqs + 1 running sums, held and len: per request.
template <class Off>
__device__ __forceinline__ void fill(const PlanArgs& a, const int* start, const Off* off, const int* held, const int* len, Given g,
                                     int tid, int threads) {
  for (int64_t i = tid; i < off[a.n_seqs]; i += threads) {
    const int s = bisect(off, a.n_seqs, i);
    a.p.table[s * a.p.stride + held[s] + (i - off[s])] = page_taken(a, g, i);
  }
  if (!a.row_seq && !a.row_pos && !a.row_slot) return;
  const int live = start[a.n_seqs];
  for (int r = tid; r < a.n_rows; r += threads) {
    int s = -1, pos = -1;
    int64_t slot = -1;
    if (r < live) {
      s = bisect(start, a.n_seqs, r);
      pos = len[s] - (start[s + 1] - r);
      const int p = pos >> a.p.shift;
      if (a.row_slot && p < a.p.pages_per_seq) {
        const int page = p < held[s] ? a.p.table[s * a.p.stride + p] : page_taken(a, g, off[s] + p - held[s]);
        if (page >= 0 && page < a.p.n_pages) slot = (static_cast<int64_t>(page) << a.p.shift) + (pos & ((1 << a.p.shift) - 1));
      }
    }
    if (a.row_seq) a.row_seq[r] = s;
    if (a.row_pos) a.row_pos[r] = pos;
    if (a.row_slot) a.row_slot[r] = slot;
  }
}

// One request of the sums.
struct Need {
  int cached, fresh, held;
};
__device__ __forceinline__ Need need_of(const PlanArgs& a, int s) {
  constexpr int kMaxLen = 1 << 30;
  if (s >= a.n_seqs) return Need{0, 0, 0};
  return Need{clamp_to(a.cached[s], kMaxLen), clamp_to(a.n_new[s], a.n_rows), clamp_to(a.p.held[s], a.p.pages_per_seq)};
}

// The sums, and with FILL (n_seqs <= kPThreads) everything else.
template <bool FILL>
__global__ void __launch_bounds__(kPThreads) plan_kernel(PlanArgs a) {
  __shared__ int lds[4][kPWaves];
  __shared__ int l_start[FILL ? kPThreads + 1 : 1], l_held[FILL ? kPThreads : 1], l_len[FILL ? kPThreads : 1];
  __shared__ int64_t l_off[FILL ? kPThreads + 1 : 1];
  const int tid = threadIdx.x;
  const int before = clamp_to(*a.p.n_free, a.p.n_pages);
  int64_t rows = 0, wanted = 0;
  for (int s0 = 0; s0 < a.n_seqs; s0 += kPThreads) {
    const int s = s0 + tid;
    const Need n = need_of(a, s);
    int total;
    // 1024 counts of at most 2^20 stay below 2^31
    const int64_t at = rows + block_scan(n.fresh, lds[0], total);
    const int first = static_cast<int>(at < a.n_rows ? at : a.n_rows);
    const int fresh = n.fresh < a.n_rows - first ? n.fresh : a.n_rows - first;
    rows += total;
    const int len = n.cached + fresh, pages = fresh > 0 ? pages_of(a.p, len) : 0;
    const int want = pages > n.held ? pages - n.held : 0;
    // 1024 tables may name more than 2^31 pages: low and high parts apart
    int low, high;
    const int64_t low_at = block_scan(want & 0xFFFF, lds[1], low), high_at = block_scan(want >> 16, lds[2], high);
    const int64_t off = wanted + low_at + (high_at << 16);
    wanted += low + (static_cast<int64_t>(high) << 16);
    if (s < a.n_seqs) {
      a.start[s] = first;
      a.len[s] = len;
      if (FILL) {
        l_start[s] = first;
        l_off[s] = off;
        l_held[s] = n.held;
        l_len[s] = len;
      } else {
        a.off[s] = off;
        a.held[s] = n.held;
      }
    }
    __syncthreads();                           // lds is free again
  }
  const int live = static_cast<int>(rows < a.n_rows ? rows : a.n_rows);
  const Given g{wanted < before ? wanted : before, before};
  if (tid == 0) {
    a.start[a.n_seqs] = live;
    *a.p.n_free = static_cast<int>(before - g.pages);
    const int64_t lack = wanted - g.pages;
    if (a.missing) *a.missing = static_cast<int>(lack < 0x7fffffff ? lack : 0x7fffffff);
    if (FILL) {
      l_start[a.n_seqs] = live;
      l_off[a.n_seqs] = wanted;
    } else {
      a.off[a.n_seqs] = wanted;
      a.off[a.n_seqs + 1] = g.pages;
      a.off[a.n_seqs + 2] = before;
    }
  }
  __syncthreads();
  const int64_t* offs = FILL ? l_off : a.off;
  for (int s = tid; s < a.n_seqs; s += kPThreads) {
    const int64_t from = offs[s], to = offs[s + 1];
    const int64_t got = (to < g.pages ? to : g.pages) - (from < g.pages ? from : g.pages);
    a.p.held[s] = (FILL ? l_held[s] : a.held[s]) + static_cast<int>(got);
  }
  if constexpr (FILL) fill(a, l_start, l_off, l_held, l_len, g, tid, kPThreads);
}

__global__ void __launch_bounds__(kFThreads) plan_fill_kernel(PlanArgs a) {
  __shared__ int l_start[kPThreads + 1], l_held[kPThreads], l_len[kPThreads];
  __shared__ int64_t l_off[kPThreads + 1];
  const int tid = threadIdx.x, all = static_cast<int>(gridDim.x) * kFThreads, me = static_cast<int>(blockIdx.x) * kFThreads + tid;
  const Given g{a.off[a.n_seqs + 1], static_cast<int>(a.off[a.n_seqs + 2])};
  if (a.n_seqs > kPThreads) {
    fill(a, a.start, a.off, a.held, a.len, g, me, all);
    return;
  }
  for (int s = tid; s <= a.n_seqs; s += kFThreads) {
    l_start[s] = a.start[s];
    l_off[s] = a.off[s];
    if (s < a.n_seqs) {
      l_held[s] = a.held[s];
      l_len[s] = a.len[s];
    }
  }
  __syncthreads();
  fill(a, l_start, l_off, l_held, l_len, g, me, all);
}

int64_t plan_bytes(int n_seqs) { return (static_cast<int64_t>(n_seqs) * 12 + 24 + 15) / 16 * 16; }

int launch_plan(const PlanArgs& a, hipStream_t st) {
  if (a.n_seqs <= kPThreads && a.n_rows <= kPlanRows) {
    hipLaunchKernelGGL((plan_kernel<true>), dim3(1), dim3(kPThreads), 0, st, a);
    return check_launch();
  }
  hipLaunchKernelGGL((plan_kernel<false>), dim3(1), dim3(kPThreads), 0, st, a);
  const int rc = check_launch();
  if (rc) return rc;
  const int most = a.n_rows > a.n_seqs ? a.n_rows : a.n_seqs, blocks = (most + kFThreads - 1) / kFThreads;
  hipLaunchKernelGGL(plan_fill_kernel, dim3(blocks < 4 * kCus ? blocks : 4 * kCus), dim3(kFThreads), 0, st, a);
  return check_launch();
}

// ---------------------------------------------------------------------------

// Entries that a request gives up: keep .. held - 1.
__device__ __forceinline__ void given_up(const ReleaseArgs& a, int s, int& from, int& to) {
  from = to = 0;
  if (s >= a.n_seqs) return;
  const int held = clamp_to(a.p.held[s], a.p.pages_per_seq), keep = a.keep[s];
  if (keep < 0 || keep >= held) return;
  from = keep;
  to = held;
}

// One workgroup; the requests that give pages up are listed, and each of
// them is a wave's: first their pages are counted, and with the counts'
// running sum they are put behind the free ones in order. A chain of
// latencies, too, six barriers and two walks of a table row: 3.1 us for 3 of 64
// requests with up to 250 pages, 5.5 for 40 of 512 with up to 187.
__global__ void __launch_bounds__(kPThreads) release_kernel(ReleaseArgs a) {
  __shared__ int lds[2][kPWaves];
  __shared__ int list[kPThreads], from[kPThreads], to[kPThreads], count[kPThreads];
  const int tid = threadIdx.x, wave = tid >> 6;
  int64_t n_free = clamp_to(*a.p.n_free, a.p.n_pages);
  for (int s0 = 0; s0 < a.n_seqs; s0 += kPThreads) {
    int f, t, n;
    given_up(a, s0 + tid, f, t);
    const int at = block_scan(t > f, lds[0], n);
    if (t > f) {
      list[at] = s0 + tid;
      from[at] = f;
      to[at] = t;
    }
    __syncthreads();
    const auto page = [&](int s, int p, int end) QMV_INLINE {   // -1: none to give back
      if (p >= end || (a.shared && p < a.shared[s])) return -1;
      const int id = a.p.table[s * a.p.stride + p];
      return id >= 0 && id < a.p.n_pages ? id : -1;
    };
    for (int i = wave; i < n; i += kPWaves) {
      int c = 0;
      for (int p = from[i]; p < to[i]; p += kWave) c += __builtin_popcountll(__ballot(page(list[i], p + lane_id(), to[i]) >= 0));
      if (lane_id() == 0) count[i] = c;
    }
    __syncthreads();
    // a page is in the pool once, so that more than n_pages of them are mistakes that are dropped
    const int mine = tid < n ? (count[tid] < a.p.n_pages ? count[tid] : a.p.n_pages) : 0;
    int low, high;
    const int64_t low_at = block_scan(mine & 0xFFFF, lds[1], low);
    __syncthreads();
    const int64_t high_at = block_scan(mine >> 16, lds[0], high);
    const int64_t first = n_free + low_at + (high_at << 16);
    if (tid < n) count[tid] = static_cast<int>(first < a.p.n_pages ? first : a.p.n_pages);
    __syncthreads();
    for (int i = wave; i < n; i += kPWaves) {
      const int s = list[i];
      int64_t dst = count[i];
      for (int p = from[i]; p < to[i]; p += kWave) {
        const int id = page(s, p + lane_id(), to[i]);
        const uint64_t some = __ballot(id >= 0);
        const int64_t mark = dst + __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(some >> 32),
                                                             __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(some), 0));
        if (id >= 0 && mark < a.p.n_pages) a.p.free[mark] = id;
        if (p + lane_id() < to[i]) a.p.table[s * a.p.stride + p + lane_id()] = -1;
        dst += __builtin_popcountll(some);
      }
      if (lane_id() == 0) a.p.held[s] = from[i];
    }
    n_free += low + (static_cast<int64_t>(high) << 16);
    if (n_free > a.p.n_pages) n_free = a.p.n_pages;
    __syncthreads();                           // the lists are free again
  }
  if (tid == 0) *a.p.n_free = static_cast<int>(n_free);
}

int launch_release(const ReleaseArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(release_kernel, dim3(1), dim3(kPThreads), 0, st, a);
  return check_launch();
}

}  // namespace qmv
