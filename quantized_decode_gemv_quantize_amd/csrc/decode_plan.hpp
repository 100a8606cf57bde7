// decode_plan.hpp - launch arithmetic of the operators between the mat-vecs:
// shapes of an attention launch, the ranges that the keys are cut into, the
// units that new tokens touch, and division by numbers the host knows. Shared
// by the launchers, the kernels and the host model of the tests.
#pragma once

#include <stdint.h>

#include "kv_layout.hpp"

namespace qmv {

// Division of 0 <= n < 2^31: q = (mulhi(n, mul) + n) >> s with 2^s >= d and
// mul = floor(2^32 (2^s - d) / d) + 1. A 32-bit division on the device is
// some forty dependent instructions, and a workgroup's place takes a dozen of
// them before its first load.
struct FastDiv {
  uint32_t d, mul, shift;
  FastDiv() = default;
  explicit FastDiv(uint32_t n) : d(n), mul(0), shift(0) {
    while ((uint64_t(1) << shift) < n) ++shift;
    mul = static_cast<uint32_t>((((uint64_t(1) << shift) - n) << 32) / n + 1);
  }
#ifndef QMV_HOST_MODEL
  __device__ __forceinline__ int div(int n) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(n), mul) + static_cast<uint32_t>(n)) >> shift);
  }
#else
  int div(int n) const {
    const uint32_t hi = static_cast<uint32_t>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul) >> 32);
    return static_cast<int>((hi + static_cast<uint32_t>(n)) >> shift);
  }
#endif
};

constexpr int kStep = 32;                       // keys a step of the attention kernels
constexpr int kMaxSplits = 128;                 // two a lane in the join

// Range `split` of `splits` over the keys beg..end-1, in steps: first and
// past-the-last key, both on steps counted from beg.
struct KeyRange {
  int beg, end;
};
KV_DEV KeyRange split_keys(int beg, int end, FastDiv splits, int split) {
  const int steps = end > beg ? (end - beg + kStep - 1) / kStep : 0;
  const int per = splits.div(steps + static_cast<int>(splits.d) - 1);
  const int s0 = split * per < steps ? split * per : steps, s1 = s0 + per < steps ? s0 + per : steps;
  return KeyRange{beg + s0 * kStep, beg + s1 * kStep};
}

// Units of 16 tokens that a run of n tokens touches at most.
KV_HD int units_of(int n) { return (n + 14) / 16 + 1; }

struct AttnShape {
  int mt;                                       // 16-row tiles a wave
  bool rows;                                    // waves own rows (else they share the keys)
  int tiles, splits;
};

constexpr int kSplitKeys = 256;                 // fewest keys worth a workgroup of their own
constexpr int kLongKeys = 2048;                 // and where they are cut beyond one round of workgroups
constexpr int kCus = 256;

// Rows of one key/value head (new tokens times query heads that share it):
// up to 16, 32 or (D = 64) 48 fit the tiles of one wave, and the four waves
// share the keys; beyond 64 each wave takes rows of its own. Tiles go by the
// batch's largest count: a sequence with fewer rows works on empty ones, too.
// 40 rows of D = 64 in one wave's three tiles against two workgroups of two
// (16 users of 5 tokens): Q4_0 over 5300..16000 keys 63 us against 86, Q8_0
// over 2700..8000 47 against 59, F16 46 against 56. Three tiles of 128 dims
// leave a compute unit one workgroup: 97 us with two, 115 with three. Of 96
// dims they would gain as well (Q4_0 107 -> 83, Q8_0 82 -> 64) and are not in
// this rule yet.
//
// The keys are cut until the chip is filled once: two workgroups a compute
// unit, one for heads of 256 dims, whose waves need more than half of the
// registers (20 us with 256 workgroups against 29 with 512 for 3 tokens of 16
// heads of 256 over 20000). No range is shorter than kSplitKeys: at 8191 keys of
// one user 11.0 us, 13.6 with ranges of 512 and 11.9 with 128. Several rows a
// wave over quantized keys are bound by arithmetic, and there twice as many
// ranges even out sequences of different lengths as long as they stay long
// (16 users of 5300..16000 keys 70 -> 64 us; ranges of 250 keys 28 -> 39 us).
inline AttnShape attn_shape(int nb, int n_seqs, int n_kv_heads, int group, int max_new, int max_len, int window) {
  const int64_t rows = static_cast<int64_t>(max_new) * group;
  AttnShape s;
  s.rows = rows > 64;
  s.mt = nb < 8 && rows > 16 ? 2 : 1;
  if (nb == 2 && rows > 32 && rows <= 48) s.mt = 3;
  const int rt = 16 * s.mt * (s.rows ? 4 : 1);
  s.tiles = static_cast<int>((rows + rt - 1) / rt);
  const int64_t groups = static_cast<int64_t>(n_seqs) * n_kv_heads * s.tiles;
  const int64_t keys = window > 0 && window + static_cast<int64_t>(max_new) < max_len
                           ? window + static_cast<int64_t>(max_new) : max_len;
  const bool heavy = !s.rows && nb == 8;        // one wave a SIMD
  const auto cut = [&](int64_t target, int64_t least) {
    const int64_t want = (target + groups - 1) / groups, most = (keys + least - 1) / least;
    return want < most ? want : most;
  };
  int64_t splits = cut(heavy ? kCus : 2 * kCus, kSplitKeys);
  if (!s.rows && s.mt > 1 && !heavy) {
    const int64_t more = cut(4 * kCus, kLongKeys);
    splits = more > splits ? more : splits;
  }
  if (splits > kMaxSplits) splits = kMaxSplits;
  s.splits = static_cast<int>(splits < 1 ? 1 : splits);
  return s;
}

}  // namespace qmv
