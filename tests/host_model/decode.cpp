// decode.cpp - host model of the launch arithmetic and the cache layout of the
// operators between the mat-vecs: the kernels' own headers, run on the CPU.
#include <cstdio>
#include <vector>

#include "decode_plan.hpp"

using namespace qmv;

static long bad = 0;
#define CHECK(c, ...) do { if (!(c)) { if (++bad < 20) { printf("FAIL %s: ", #c); printf(__VA_ARGS__); printf("\n"); } } } while (0)

// Every byte of a unit is one value's (or scale's), and operand loads find the
// values that the writer put there, aligned as they need it.
static void layout(int kind, int nb) {
  const int unit = kv_unit_bytes(kind, nb), code = kv_code_bytes(kind, nb), ps = kv_piece(kind, nb), run = kv_run(kind);
  const int esize = kind == kKvF16 ? 2 : 1, dims = kind == kKvQ4 ? 16 : 32;
  CHECK(unit % 16 == 0 && code % 16 == 0, "kind %d nb %d", kind, nb);
  for (int keys = 0; keys < 2; ++keys) {
    std::vector<int> owner(unit, 0);
    for (int tt = 0; tt < 16; ++tt)
      for (int b = 0; b < nb; ++b) {
        for (int c = 0; c < dims; ++c) {
          const int at = keys ? kv_key_at(kind, nb, tt, b, c) : kv_value_at(kind, tt, b, c);
          for (int e = 0; e < esize; ++e)
            if (at + e >= 0 && at + e < code) ++owner[at + e];
            else CHECK(false, "kind %d nb %d at %d", kind, nb, at);
          if (kind == kKvQ4) CHECK(at == (keys ? kv_key_at(kind, nb, tt, b, c + 16) : kv_value_at(kind, tt, b, c + 16)), "nibble pair");
        }
        if (kind != kKvF16)
          for (int e = 0; e < 2; ++e) ++owner[kv_scale_at(kind, nb, b, tt) + e];
      }
    for (int i = 0; i < unit; ++i) CHECK(owner[i] == 1, "kind %d nb %d keys %d byte %d owned %d times", kind, nb, keys, i, owner[i]);
  }
  // keys: run b of lane (g, rr) of tile m holds 8 dims of token 8 (rr / 4) + 4 m + rr % 4
  for (int m = 0; m < 2; ++m)
    for (int g = 0; g < 4; ++g)
      for (int rr = 0; rr < 8; ++rr)
        for (int b = 0; b < nb; ++b) {
          const int off = b * run, at = kv_key_piece(kind, nb, m, off / ps, g, rr) + off % ps, tt = rr / 4 * 8 + m * 4 + rr % 4;
          CHECK(at + run <= code && kv_key_piece(kind, nb, m, off / ps, g, rr) % ps == 0 && at % run == 0, "run at %d", at);
          for (int j = 0; j < (kind == kKvQ4 ? 4 : 8); ++j)
            CHECK(kv_key_at(kind, nb, tt, b, kind == kKvQ4 ? 4 * g + j : 8 * g + j) == at + j * esize, "key run m %d g %d rr %d b %d", m, g, rr, b);
        }
  // values: the lane of dim r, tokens 8 h8..
  for (int b = 0; b < nb; ++b)
    for (int half = 0; half < 2; ++half)
      for (int h8 = 0; h8 < 2; ++h8)
        for (int r = 0; r < 16; ++r) {
          const int at = kv_value_run(kind, b, half, h8, r) + (kind == kKvQ8 ? 8 * half : 0);
          CHECK(kv_value_run(kind, b, half, h8, r) % (kind == kKvQ4 ? 8 : 16) == 0, "value run alignment");
          for (int j = 0; j < 8; ++j)
            CHECK(kv_value_at(kind, 8 * h8 + j, b, 16 * half + r) == at + j * esize, "value run b %d half %d h8 %d r %d", b, half, h8, r);
        }
  for (int b = 0; b < nb; ++b)
    for (int h8 = 0; h8 < 2 && kind != kKvF16; ++h8) CHECK(kv_scale_at(kind, nb, b, 8 * h8) % 16 == 0, "scale alignment");
}

static void division() {
  const int ns[] = {0, 1, 2, 3, 31, 32, 33, 1000, 65535, 65536, 1 << 20, (1 << 30) - 1, 1 << 30, (1 << 30) + 127, 0x7fffffff};
  for (uint32_t d = 1; d < 5000; ++d) {
    const FastDiv f(d);
    for (int n : ns) CHECK(f.div(n) == n / static_cast<int>(d), "%d / %u", n, d);
    for (int n = 0; n < 4000; n += 1 + d % 7) CHECK(f.div(n) == n / static_cast<int>(d), "%d / %u", n, d);
    for (int64_t k = 1; k * d < 0x7fffffff; k = k * 3 + 1)
      for (int64_t n = k * d - 1; n <= k * d + 1 && n < 0x7fffffff; ++n) CHECK(f.div(static_cast<int>(n)) == n / d, "%ld / %u", static_cast<long>(n), d);
  }
  for (uint32_t d : {65535u, 65536u, 65537u, (1u << 22) - 1, 1u << 22, (1u << 30) - 1})
    for (int n : ns) CHECK(FastDiv(d).div(n) == n / static_cast<int>(d), "%d / %u", n, d);
}

// The ranges cover the keys' steps once, in order, wherever they start.
static void ranges() {
  for (int splits = 1; splits <= kMaxSplits; splits = splits < 9 ? splits + 1 : splits * 2 - 3)
    for (int beg : {0, 32, 960})
      for (int n : {-5, 0, 1, 31, 32, 33, 64, 100, 1000, 4096, 8191, 70000, 1 << 30}) {
        const int end = n > (1 << 29) ? n : beg + n;
        const int steps = end > beg ? (end - beg + kStep - 1) / kStep : 0;
        int at = beg;
        for (int s = 0; s < splits; ++s) {
          const KeyRange r = split_keys(beg, end, FastDiv(splits), s);
          CHECK(r.beg == at || (r.beg == r.end && r.beg == beg + steps * kStep), "splits %d n %d s %d: %d..%d at %d", splits, n, s, r.beg, r.end, at);
          CHECK(r.end >= r.beg && (r.beg - beg) % kStep == 0, "range");
          at = r.end > at ? r.end : at;
        }
        CHECK(at == beg + steps * kStep, "splits %d n %d: ends at %d", splits, n, at);
      }
}

// Launch shapes: rows are covered, waves and splits are in their limits.
static void shapes() {
  for (int nb : {2, 3, 4, 8})
    for (int n_seqs : {1, 3, 64, 5000})
      for (int heads : {1, 8, 1024})
        for (int group : {1, 5, 8, 64})
          for (int new_ : {1, 2, 5, 17, 300, 1 << 20})
            for (int len : {1, 255, 257, 8191, 1 << 20, 1 << 30})
              for (int window : {0, 1, 128, 1 << 30}) {
                const AttnShape s = attn_shape(nb, n_seqs, heads, group, new_, len, window);
                const int64_t rows = static_cast<int64_t>(new_) * group, rt = 16 * s.mt * (s.rows ? 4 : 1);
                CHECK(s.splits >= 1 && s.splits <= kMaxSplits, "splits %d", s.splits);
                CHECK(s.tiles >= 1 && s.tiles * rt >= rows && (s.tiles - 1) * rt < rows, "tiles %d of %ld", s.tiles, static_cast<long>(rt));
                CHECK(s.mt == 1 || (s.mt == 2 && nb < 8) || (s.mt == 3 && nb == 2), "mt %d nb %d", s.mt, nb);
                CHECK(!(s.rows && s.mt != (nb < 8 ? 2 : 1)), "rows mt %d nb %d", s.mt, nb);
                // the workspace is asked for without a window: never smaller
                CHECK(s.splits <= attn_shape(nb, n_seqs, heads, group, new_, len, 0).splits, "window %d", window);
              }
  for (int n = 1; n < 200; ++n)
    for (int first = 0; first < 16; ++first) CHECK((first + n - 1) / 16 - first / 16 + 1 <= units_of(n), "%d tokens from %d", n, first);
}

int main() {
  for (int kind : {kKvF16, kKvQ8, kKvQ4})
    for (int nb : {2, 3, 4, 8}) layout(kind, nb);
  division();
  ranges();
  shapes();
  printf("%ld failing check(s)\n", bad);
  return bad != 0;
}
