// attn_kernel.hpp - attention of new tokens over the paged cache.
//
//   out = sum_t softmax(scale q.k_t) v_t over the visible keys t
//
// The query heads that share a key/value head are rows of one product
// (row = token * group + head of the group), so a cache byte is read once for
// all of them. A wave owns MT tiles of 16 rows and walks the keys 32 at a
// time with the running maximum M, sum l and unnormalised O of a softmax:
//   S^T = K q^T     two 16x16 tiles of 16x16x32 fp16 products; a lane then
//                   holds the scores of ONE row (lane % 16) for the 8 tokens
//                   8g..8g+7 of the step (g = lane / 16)
//   O^T += V^T P^T  whose right operand is exactly that: the probabilities
//                   stay in their lanes, and M, l and the rescaling of O are
//                   one value a lane
// The cache is stored in operand order (kv_layout.hpp). Quantized codes are
// exact in fp16; a key's block scale is applied to the block's partial score,
// a value's block scale d to the probability.
//
// Precision: q (times scale * log2 e, in fp32) is carried as two fp16 parts
// of the row scaled by a power of two, 21 bits of the row's largest value; a
// probability (times d) as two fp16 parts, 20 bits. fp16 parts need their
// factor in range: the reference M of a row is the maximum of s + e over the
// keys, e the exponent field of the token's largest |d| (0 for F16), and the
// weight w = 2^(s + e - M + K) enters l times 2^(16 - e) and O times
// d 2^(16 - e), which is below 4: fp16 numbers, off by 2^-32 of the largest at
// most however small they are. The factor 2^(K + 16 - M) cancels in O / l. A
// token's scales that lie so far below its largest that the factor takes bits
// from them have these added apart (lost_f16). Scores, M, l and O are fp32.
//
// Two kernels: with few rows the four waves of a workgroup take every fourth
// step of the same rows, read operands from memory straight into registers
// (the cache is the traffic, nothing would be shared) and join O through
// LDS; with many rows each wave has rows of its own, and the workgroup turns
// each step's codes into operands once, in LDS, for all four. Either way the
// keys can be cut into ranges whose partial (M, l, O) a second
// launch joins, so that few rows over a long cache still fill the chip.
//
// Measured: F16, 64 sequences of one token over 1500..4500 keys of 8 heads of
// 128, 154 us, 5.3 TB/s, bound by memory (Q8_0 95, Q4_0 88); Q4_0, 16 of 2 to 5
// tokens and 64 query heads of 64 over 5300..16000, 64 us, bound by vector issue
// (79 %, a third of it for rows that a sequence does not have); Q8_0, 2048
// tokens of 32 heads of 128 over 8192, 543 us, 442 TFLOP/s of the formula's
// operations (the parts double them), vector issue 70 % and the chain of one
// wave's own reads and products: a compute unit with one workgroup instead of
// two takes as long for it.
#pragma once

#include "decode_args.hpp"
#include "launch.hpp"

namespace qmv {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kAttnThreads = 256;

// K above, with the 16 of a quantized token's factor: w <= 2^14 (F16), 2^13
// where its product is below 4 times that. M may lag the true maximum by
// kLag, so that O is rescaled a few times a walk instead of at every new
// maximum; K leaves room for it.
constexpr float kLag = 4.0f;
__host__ __device__ constexpr float weight_shift(int kind) { return (kind == kKvF16 ? 14.0f : 13.0f + 16.0f) - kLag; }

__device__ __forceinline__ f32x4 mfma_f16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}
// Maximum and sum over the four lanes that share a row.
__device__ __forceinline__ float row_max(float v) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float row_sum(float v) {
  v = swap_pair_sum<32>(v, v);
  return swap_pair_sum<16>(v, v);
}

// Two values as fp16 parts: hi toward zero, lo the nearest of the rest
// (together 21 bits). The rest as a * 1 - hi: a fused multiply-add takes hi
// as it is (v_fma_mix_f32), a difference would convert it first.
__device__ __forceinline__ void split_f16(float a, float b, uint32_t& hi, uint32_t& lo) {
  const auto h = __builtin_amdgcn_cvt_pkrtz(a, b);
  hi = __builtin_bit_cast(uint32_t, h);
  float one = 1.0f;
  asm("" : "+s"(one));
  float ra = fmaf(a, one, -static_cast<float>(h[0])), rb = fmaf(b, one, -static_cast<float>(h[1]));
  asm("" : "+v"(ra), "+v"(rb));                 // or fma and conversion in one, at half the rate
  const half2v r = {static_cast<_Float16>(ra), static_cast<_Float16>(rb)};
  lo = __builtin_bit_cast(uint32_t, r);
}
// Parts of the products (ph + pl) d of two values: hi the nearest fp16 of
// ph d, lo of its rest (exact in fp16) and pl d.
__device__ __forceinline__ void scale_parts(uint32_t ph, uint32_t pl, uint32_t d, uint32_t& hi, uint32_t& lo) {
  const half2v p = __builtin_bit_cast(half2v, ph), q = __builtin_bit_cast(half2v, pl), f = __builtin_bit_cast(half2v, d);
  const half2v h = p * f;
  hi = __builtin_bit_cast(uint32_t, h);
  lo = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(q, f, __builtin_elementwise_fma(p, f, -h)));
}

// fp16 of four biased codes (bytes): 1024 + u by its bits, less the bias.
__device__ __forceinline__ void codes_f16(uint32_t w, float bias, uint32_t& lo, uint32_t& hi) {
  const _Float16 b = static_cast<_Float16>(-1024.0f - bias);
  const half2v off = {b, b};
  lo = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) + off);
  hi = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) + off);
}
// Operand of 8 codes in two words (Q8_0), or in the low or high nibbles of them.
__device__ __forceinline__ u32x4 operand_q8(uint32_t a, uint32_t b) {
  uint32_t t[4];
  codes_f16(a, 128.0f, t[0], t[1]);
  codes_f16(b, 128.0f, t[2], t[3]);
  return u32x4{t[0], t[1], t[2], t[3]};
}
__device__ __forceinline__ u32x4 operand_q4(uint32_t a, uint32_t b) {   // nibbles in bytes
  uint32_t t[4];
  codes_f16(a & 0x0F0F0F0Fu, 8.0f, t[0], t[1]);
  codes_f16(b & 0x0F0F0F0Fu, 8.0f, t[2], t[3]);
  return u32x4{t[0], t[1], t[2], t[3]};
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// Of two tokens' largest scales: fp16 factors 2^(16 - e), e the exponent
// field, at least 1 (a subnormal's unit is that of the field 1), and e. A
// scale of the token times its factor is below 4, without any rounding that
// the largest would notice.
__device__ __forceinline__ uint32_t token_factors(uint32_t top) { return 0x7C007C00u - max_u16x2(top & 0x7C007C00u, 0x04000400u); }
__device__ __forceinline__ float factor_field(uint32_t word, int half) {   // e
  return static_cast<float>(static_cast<int>(31u - ((word >> (16 * half + 10)) & 31u)));
}
__device__ __forceinline__ uint32_t pk_mul_f16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, a) * __builtin_bit_cast(half2v, b));
}

// A factor below 1 (a largest scale of 4 and more) takes the token's scales
// that are 2^-15 of the largest and less under fp16's 2^-14, where they lose
// up to 2^-25 of a product that is 2 and more for the largest. What they lose
// is exact in fp32, and times 2^kLost in fp16; with the first part of the
// weight times 2^-kLost it is one more product, below 2^-12 and so off by
// 2^-25 itself. Rare; either kernel takes it where it costs its walk least.
constexpr int kLost = 14;
__device__ __forceinline__ uint32_t min_u16x2(uint32_t a, uint32_t b) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ bool below_one(uint32_t factors) { return (factors & 0xFFFFu) < 0x3C00u || (factors >> 16) < 0x3C00u; }
__device__ __forceinline__ uint32_t lost_f16(uint32_t d, uint32_t factor) {
  constexpr float up = static_cast<float>(1 << kLost);
  const uint32_t kept = pk_mul_f16(d, factor);
  const half2v r = {static_cast<_Float16>(up * fmaf(h2f(d), h2f(factor), -h2f(kept))),
                    static_cast<_Float16>(up * fmaf(h2f(d >> 16), h2f(factor >> 16), -h2f(kept >> 16)))};
  return __builtin_bit_cast(uint32_t, r);
}

// Words of 8 fp16 whose elements c.. are cleared.
__device__ __forceinline__ uint32_t keep_mask(int e, int c) {
  return c >= 2 * e + 2 ? ~0u : c == 2 * e + 1 ? 0xFFFFu : 0u;
}
// Nonzero if one of the two fp16 is infinite or NaN.
__device__ __forceinline__ uint32_t wild_bits(uint32_t w) { return ((w & 0x7FFF7FFFu) + 0x04000400u) & 0x80008000u; }
// The two fp16, zero where infinite or NaN.
__device__ __forceinline__ uint32_t tamed(uint32_t w) { return w & ~((wild_bits(w) >> 15) * 0xFFFFu); }

// Loads of a wave's 32-key step, as they lie in the cache.
template <int KIND, int NB>
struct KeyRegs {
  static constexpr int kWords = 2 * kv_lane_bytes(KIND, NB) / 4;
  uint32_t w[kWords];                           // [m][run bytes of the blocks in turn]
  u32x4 sc[KIND == kKvF16 ? 1 : NB];            // scales of tokens 8g..8g+7 per block

  // unit: the 16-token unit of this lane's row as keys; sunit: of tokens 8g..
  __device__ __forceinline__ void load(const uint8_t* unit, const uint8_t* sunit) {
    constexpr int PS = kv_piece(KIND, NB), PW = PS / 4, NP = kv_lane_bytes(KIND, NB) / PS;
    const int l = lane_id(), g = l >> 4;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const uint8_t* src = unit + kv_key_piece(KIND, NB, m, p, g, l & 7);
        uint32_t* dst = w + (m * NP + p) * PW;
        if constexpr (PS == 16) {
          const u32x4 r = ld_a16_x4(src);
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[e] = r[e];
        } else if constexpr (PS == 8) {
          const u32x2 r = ld_x2(src);
          dst[0] = r.x;
          dst[1] = r.y;
        } else {
          dst[0] = ld_u32(src);
        }
      }
    if constexpr (KIND != kKvF16) {
#pragma unroll
      for (int b = 0; b < NB; ++b) sc[b] = ld_a16_x4(sunit + kv_scale_at(KIND, NB, b, 8 * (g & 1)));
    }
  }
  // fp16 operand of block b, tile m
  __device__ __forceinline__ u32x4 operand(int m, int b) const {
    constexpr int LW = kv_lane_bytes(KIND, NB) / 4;
    if constexpr (KIND == kKvF16) {
      return u32x4{w[m * LW + 4 * b], w[m * LW + 4 * b + 1], w[m * LW + 4 * b + 2], w[m * LW + 4 * b + 3]};
    } else if constexpr (KIND == kKvQ8) {
      return operand_q8(w[m * LW + 2 * b], w[m * LW + 2 * b + 1]);
    } else {
      return operand_q4(w[m * LW + b], w[m * LW + b] >> 4);
    }
  }
};

template <int KIND, int NB>
struct ValueRegs {
  static constexpr int kPer = KIND == kKvF16 ? 8 : KIND == kKvQ8 ? 4 : 2;   // words a block
  uint32_t w[NB * kPer];
  u32x4 sc[KIND == kKvF16 ? 1 : NB];

  // unit: of tokens 8g..8g+7
  __device__ __forceinline__ void load(const uint8_t* unit) {
    const int l = lane_id(), h8 = (l >> 4) & 1, r = l & 15;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if constexpr (KIND == kKvF16) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const u32x4 v = ld_a16_x4(unit + kv_value_run(KIND, b, half, h8, r));
#pragma unroll
          for (int e = 0; e < 4; ++e) w[8 * b + 4 * half + e] = v[e];
        }
      } else if constexpr (KIND == kKvQ8) {
        const u32x4 v = ld_a16_x4(unit + kv_value_run(KIND, b, 0, h8, r));
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * b + e] = v[e];
      } else {
        const u32x2 v = ld_x2(unit + kv_value_run(KIND, b, 0, h8, r));
        w[2 * b] = v.x;
        w[2 * b + 1] = v.y;
      }
      if constexpr (KIND != kKvF16) sc[b] = ld_a16_x4(unit + kv_scale_at(KIND, NB, b, 8 * h8));
    }
  }
  // fp16 operand of dims 32 b + 16 half ..
  __device__ __forceinline__ u32x4 operand(int b, int half) const {
    if constexpr (KIND == kKvF16) {
      const uint32_t* p = w + 8 * b + 4 * half;
      return u32x4{p[0], p[1], p[2], p[3]};
    } else if constexpr (KIND == kKvQ8) {
      return operand_q8(w[4 * b + 2 * half], w[4 * b + 2 * half + 1]);
    } else {
      return operand_q4(w[2 * b] >> (4 * half), w[2 * b + 1] >> (4 * half));
    }
  }
  // The tokens' factors and exponent fields; their scales times the factors.
  __device__ __forceinline__ void normalise(u32x4& factor, float (&e5)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t top = sc[0][e] & 0x7FFF7FFFu;
#pragma unroll
      for (int b = 1; b < NB; ++b) top = max_u16x2(top, sc[b][e] & 0x7FFF7FFFu);
      factor[e] = token_factors(top);
      e5[2 * e] = factor_field(factor[e], 0);
      e5[2 * e + 1] = factor_field(factor[e], 1);
#pragma unroll
      for (int b = 0; b < NB; ++b) sc[b][e] = pk_mul_f16(sc[b][e], factor[e]);
    }
  }
  // Tokens c.. of this lane's 8 do not exist: what lies there is no value
  // (F16) or scale, and 0 times it need not be 0.
  __device__ __forceinline__ void keep(int c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t mask = keep_mask(e, c);
      if constexpr (KIND == kKvF16) {
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t) w[4 * t + e] &= mask;
      } else {
#pragma unroll
        for (int b = 0; b < NB; ++b) sc[b][e] &= mask;
      }
    }
  }
  // F16: whether any value is infinite or NaN; zeros in their place
  __device__ __forceinline__ bool wild() const {
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < NB * kPer; ++i) any |= wild_bits(w[i]);
    return any != 0;
  }
  __device__ __forceinline__ void tame() {
#pragma unroll
    for (int i = 0; i < NB * kPer; ++i) w[i] = tamed(w[i]);
  }
};

// Table entries of a 32-key step's two 16-token halves, read a step ahead of
// its loads. They stay in vector registers as they come (`zero` keeps the
// compiler from seeing that they are the same in all lanes): turned into
// scalars at once they would make the wave wait for every load in flight.
struct StepIds {
  int id[2];
};

__device__ __forceinline__ int vector_zero() {
  int z;
  asm("v_mov_b32 %0, 0" : "=v"(z));
  return z;
}

__device__ __forceinline__ StepIds step_ids(const AttnArgs& a, int s, int t0, int zero) {
  const int32_t* row = a.b.page_table + static_cast<int64_t>(s) * a.b.table_stride;
  const int last = a.b.pages_per_seq - 1, p0 = t0 >> a.b.page_shift, p1 = (t0 + 16) >> a.b.page_shift;
  return StepIds{{row[(p0 < last ? p0 : last) + zero], row[(p1 < last ? p1 : last) + zero]}};
}

// Where the units of a step's halves lie, from the cache's start; a half may
// be a hole.
struct StepPages {
  int64_t off[2];
  bool ok[2];
};

template <int KIND, int NB>
__device__ __forceinline__ StepPages step_pages(const AttnArgs& a, StepIds ids, int head, int t0) {
  constexpr int U = kv_unit_bytes(KIND, NB);
  const int upp = 1 << (a.b.page_shift - 4);
  const uint32_t page_bytes = static_cast<uint32_t>(a.b.n_kv_heads * upp) * U;   // 2^29 at most
  StepPages p;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int pos = t0 + 16 * h;
    p.ok[h] = (pos >> a.b.page_shift) < a.b.pages_per_seq && static_cast<uint32_t>(ids.id[h]) < static_cast<uint32_t>(a.b.n_pages);
    const uint32_t page = p.ok[h] ? static_cast<uint32_t>(ids.id[h]) : 0u;   // a hole's loads go to page 0 and are masked
    p.off[h] = static_cast<int64_t>(static_cast<uint64_t>(page) * page_bytes +
                                    static_cast<uint32_t>(head * upp + ((pos >> 4) & (upp - 1))) * U);
  }
  return p;
}

// Factor that turns a row's O into its result: 1 / l with the sink's share
// in l; 0 for a row that saw no key (l is NaN where all scores were). l and O
// are in units of 2^(m - shift), in which a sink 2^128 above is infinite: it
// leaves the keys nothing.
__device__ __forceinline__ float row_factor(const AttnArgs& a, int head, float m, float l, float shift) {
  if (l == 0.0f) return 0.0f;
  if (!a.sinks) return 1.0f / l;
  return 1.0f / (l + __builtin_amdgcn_exp2f(fmaf(a.sinks[head], 1.44269504088896340736f, shift - m)));
}

// A finished row to out, or a split's share of it to the workspace. `write`
// stores this lane's values times a factor from the row's first float on.
template <int D, class W>
__device__ __forceinline__ void store_row(const AttnArgs& a, int token, int head, int split, float m, float l,
                                          float shift, W write, bool lead) {
  if (a.splits.d == 1) {
    write(a.out + token * a.ldo + static_cast<int64_t>(head) * D, row_factor(a, head, m, l, shift));
  } else {
    const int64_t at = (static_cast<int64_t>(token) * a.n_heads + head) * static_cast<int>(a.splits.d) + split;
    write(a.part_o + at * D, 1.0f);
    if (lead) a.part_ml[at] = make_float2(m, l);
  }
}

// What a workgroup works on: a tile of rows of one sequence and key/value
// head, and a range of the keys.
struct Place {
  int head, split, s, tile0;
  int first, count, len, keys, rows, base;      // base: position of new token 0
  // The sequence with n longer ones (of equals the first is the longer). Up
  // to 64 of them, a lane each.
  static __device__ __forceinline__ int nth_longest(const AttnArgs& a, int n) {
    const int lane = lane_id(), count = a.b.n_seqs, own = lane < count ? a.b.seq_len[lane] : 0;
    int before = 0;
    for (int j = 0; j < count; ++j) {
      const int other = __builtin_amdgcn_readlane(own, j);
      before += other > own || (other == own && j < lane);
    }
    return __builtin_ctzll(__ballot(lane < count && before == n));
  }
  template <bool ROWS>
  __device__ __forceinline__ bool find(const AttnArgs& a) {
    // Workgroups go to the 8 XCDs in turn: those that read the same keys (the
    // tiles of one sequence, head and range) get the same XCD and its L2.
    const int slot = blockIdx.x >> 3;
    const int slot_group = a.tiles.div(slot), tiles = static_cast<int>(a.tiles.d);
    int id = slot_group * 8 + static_cast<int>(blockIdx.x & 7);
    // Later rows see more keys. The longest first; where all workgroups of the
    // launch run at once, two a compute unit, the second half from the
    // shortest on, so that a long one has a short one beside it.
    const int j = slot - slot_group * tiles, back = tiles - tiles / 2;
    tile0 = gridDim.x <= 512 && j >= back ? j - back : tiles - 1 - j;
    const int per_head = a.heads.div(id);
    head = id - per_head * static_cast<int>(a.heads.d);
    s = a.splits.div(per_head);
    split = per_head - s * static_cast<int>(a.splits.d);
    if (s >= a.b.n_seqs) return false;
    if (ROWS && a.by_length) s = nth_longest(a, s);
    const int from = a.b.token_start[s], to = a.b.token_start[s + 1], l = a.b.seq_len[s];
    a.b.clamp_rows(from, to, first, count);
    len = l < 0 ? 0 : l > (1 << 30) ? (1 << 30) : l;
    const int64_t table_end = static_cast<int64_t>(a.b.pages_per_seq) << a.b.page_shift;
    keys = len < table_end ? len : static_cast<int>(table_end);
    rows = count * static_cast<int>(a.group.d);   // n_tokens * n_heads <= 2^30
    base = len - count;
    return true;
  }
  // The split's range of the keys that rows r0..r1 see, in whole steps.
  __device__ __forceinline__ void range(const AttnArgs& a, int r0, int r1, int& beg, int& end) const {
    const int lo = base + a.group.div(r0), hi = base + a.group.div(r1);
    const int k_end = hi + 1 < keys ? hi + 1 : keys;
    const int k_beg = a.window > 0 && lo - a.window + 1 > 0 ? (lo - a.window + 1) & ~(kStep - 1) : 0;
    const KeyRange k = split_keys(k_beg, k_end, a.splits, split);
    beg = k.beg;
    end = k.end;
  }
};

// A wave's rows: q as operands, and the running softmax. QLDS: q in LDS, where
// the four waves of the keys kernel share it, [tile][block][lo, hi][lane].
// AHEAD: keys and values come from LDS, and a block's are read before the
// products of the block before it: a wave waits for its own chain of reads and
// products, two waves a SIMD do not cover it all (2048 tokens over 8192: F16
// of 96 dims 418 -> 400 us, Q8_0 492 -> 469, of 256 1746 -> 1586). The keys of
// quantized heads of 128 dims are read in place, for they have no registers
// left to be read ahead to (Q8_0 577 us as it was, 538 with the values ahead,
// 593 with both).
template <int KIND, int NB, int MT, bool QLDS = false, bool AHEAD = false>
struct Rows {
  static constexpr bool kKeysAhead = AHEAD && (KIND == kKvF16 || NB != 4);
  static constexpr int DT = 2 * NB;
  static constexpr float kTop = KIND == kKvF16 ? weight_shift(KIND) : weight_shift(KIND) - 16.0f;   // the factors' 16
  u32x4 qh[QLDS ? 1 : MT][QLDS ? 1 : NB], ql[QLDS ? 1 : MT][QLDS ? 1 : NB];
  const u32x4* q_lds;
  float to_log2[MT];                            // 2^-k of the row's scaling
  int qpos[MT];                                 // position; -1: no row, or one before position 0
  float m[MT], l[MT];
  f32x4 o[MT][DT];

  __device__ __forceinline__ u32x4 q(int t, int b, int hi) const {
    if constexpr (QLDS) return q_lds[((t * NB + b) * 2 + hi) * kWave + lane_id()];
    else return hi ? qh[t][b] : ql[t][b];
  }

  __device__ __forceinline__ void init(const AttnArgs& a, const Place& w, int row0, u32x4* lds = nullptr) {
    const int lane = lane_id(), g = lane >> 4, col = lane & 15;
    q_lds = lds;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int row = row0 + 16 * t + col;
      const bool live = row < w.rows;
      const int group = static_cast<int>(a.group.d), tok = live ? a.group.div(row) : 0;
      const int hd = w.head * group + (live ? row - tok * group : 0);
      qpos[t] = live && w.base + tok >= 0 ? w.base + tok : -1;
      const float* src = a.q + (w.first + tok) * a.ldq + static_cast<int64_t>(hd) * (32 * NB);
      float v[NB][8], top = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int d0 = 32 * b + (KIND == kKvQ4 ? 4 * g : 8 * g), d1 = KIND == kKvQ4 ? d0 + 16 : d0 + 4;
        const u32x4 x = ld_x4(reinterpret_cast<const uint8_t*>(src + d0));
        const u32x4 y = ld_x4(reinterpret_cast<const uint8_t*>(src + d1));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[b][e] = live ? __uint_as_float(x[e]) * a.scale_log2 : 0.0f;
          v[b][4 + e] = live ? __uint_as_float(y[e]) * a.scale_log2 : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[b][e]));
      }
      top = row_max(top);
      int ex = static_cast<int>((__float_as_uint(top) >> 23) & 0xFFu) - 127;   // 2^ex <= top < 2^(ex+1)
      ex = top == 0.0f || ex == 128 ? 13 : ex < -100 ? -100 : ex;
      const float up = __uint_as_float(static_cast<uint32_t>(13 - ex + 127) << 23);   // to 2^13..2^14
      to_log2[t] = __uint_as_float(static_cast<uint32_t>(ex - 13 + 127) << 23);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        u32x4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t h, r;
          split_f16(v[b][2 * e] * up, v[b][2 * e + 1] * up, h, r);
          hi[e] = h;
          lo[e] = r;
        }
        if constexpr (QLDS) {                   // all waves have the same rows: each stores its blocks
          if ((b & 3) == static_cast<int>(threadIdx.x >> 6)) {
            lds[((t * NB + b) * 2 + 0) * kWave + lane] = lo;
            lds[((t * NB + b) * 2 + 1) * kWave + lane] = hi;
          }
        } else {
          qh[t][b] = hi;
          ql[t][b] = lo;
        }
      }
      m[t] = -INFINITY;
      l[t] = 0.0f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[t][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
  }

  // Scores of the step. key(mm, b): operand of key tile mm, block b; scale(b):
  // the 8 tokens' scales of the block. The products of one block are
  // independent chains, and a block's partial scores are scaled while the
  // next block's products run.
  template <class K, class S>
  __device__ __forceinline__ void scores(K key, S scale, f32x4 (&s)[MT][2]) const {
#pragma unroll
    for (int t = 0; t < MT; ++t) s[t][0] = s[t][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 n0, n1, ns;                           // the next block's, where they are read ahead
    if constexpr (kKeysAhead) {
      n0 = key(0, 0);
      n1 = key(1, 0);
      ns = scale(0);
    }
    const auto next = [&](int b, u32x4& k0, u32x4& k1) QMV_INLINE {
      if constexpr (QLDS || kKeysAhead) __builtin_amdgcn_sched_barrier(0);   // a block after the other: registers
      if constexpr (kKeysAhead) {
        k0 = n0;
        k1 = n1;
        if (b + 1 < NB) {
          n0 = key(0, b + 1);
          n1 = key(1, b + 1);
          if constexpr (KIND != kKvF16) ns = scale(b + 1);
        }
        __builtin_amdgcn_sched_barrier(0);
      } else {
        k0 = key(0, b);
        k1 = key(1, b);
      }
    };
    if constexpr (KIND == kKvF16) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        u32x4 k0, k1;
        next(b, k0, k1);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          s[t][0] = mfma_f16(k0, q(t, b, 0), s[t][0]);
          s[t][1] = mfma_f16(k1, q(t, b, 0), s[t][1]);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          s[t][0] = mfma_f16(k0, q(t, b, 1), s[t][0]);
          s[t][1] = mfma_f16(k1, q(t, b, 1), s[t][1]);
        }
      }
    } else {
      f32x4 acc[2][MT][2];
      u32x4 sc_now, sc_done = {};               // of block b and of the one before it
#pragma unroll
      for (int b = 0; b <= NB; ++b) {
        sc_now = ns;
        if (b < NB) {
          u32x4 k0, k1;
          next(b, k0, k1);
          f32x4 (&c)[MT][2] = acc[b & 1];
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            c[t][0] = mfma_f16(k0, q(t, b, 0), f32x4{0.0f, 0.0f, 0.0f, 0.0f});
            c[t][1] = mfma_f16(k1, q(t, b, 0), f32x4{0.0f, 0.0f, 0.0f, 0.0f});
          }
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            c[t][0] = mfma_f16(k0, q(t, b, 1), c[t][0]);
            c[t][1] = mfma_f16(k1, q(t, b, 1), c[t][1]);
          }
        }
        if (b > 0) {
          const u32x4 sc = kKeysAhead ? sc_done : scale(b - 1);
#pragma unroll
          for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              s[t][j / 4][j & 3] = fmaf(acc[(b - 1) & 1][t][j / 4][j & 3], h2f(sc[j / 2] >> (16 * (j & 1))), s[t][j / 4][j & 3]);
        }
        sc_done = sc_now;
      }
    }
  }

  // What tile t's row does not see of tokens k0..k0+7, of which `real` exist.
  __device__ __forceinline__ void hide(const AttnArgs& a, int t, int k0, int real, f32x4 (&s)[MT][2]) const {
    const int end = qpos[t] - k0 + 1 < real ? qpos[t] - k0 + 1 : real;
    const int beg = a.window > 0 ? qpos[t] - a.window + 1 - k0 : -1;
#pragma unroll
    for (int j = 0; j < 8; ++j) s[t][j / 4][j & 3] = j < end && j >= beg ? s[t][j / 4][j & 3] : -INFINITY;
  }

  // Scores to weights; M, l and O follow. factor, e5: of the 8 tokens (F16: not read).
  // shift: kTop, less kLost in a walk for what scales lost.
  __device__ __forceinline__ void weigh(int t, u32x4 factor, const float (&e5)[8], float shift, f32x4 (&s)[MT][2]) {
    float top;
    if constexpr (KIND == kKvF16) {
      top = s[t][0][0];
#pragma unroll
      for (int j = 1; j < 8; ++j) top = fmaxf(top, s[t][j / 4][j & 3]);
      top = row_max(top) * to_log2[t];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[t][j / 4][j & 3] = fmaf(s[t][j / 4][j & 3], to_log2[t], e5[j]);
      top = s[t][0][0];
#pragma unroll
      for (int j = 1; j < 8; ++j) top = fmaxf(top, s[t][j / 4][j & 3]);
      top = row_max(top);
    }
    if (__any(top > m[t] + kLag)) {
      top = fmaxf(m[t], top);
      const float al = __builtin_amdgcn_exp2f(m[t] - (top == -INFINITY ? 0.0f : top));
      l[t] *= al;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][d][i] *= al;
      m[t] = top;
    }
    const float off = shift - (m[t] == -INFINITY ? 0.0f : m[t]);   // a row that has seen nothing yet: all weights 0
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = s[t][j / 4][j & 3], w = __builtin_amdgcn_exp2f(KIND == kKvF16 ? fmaf(x, to_log2[t], off) : x + off);
      s[t][j / 4][j & 3] = w;
      if constexpr (KIND == kKvF16) l[t] += w;
      else l[t] = fmaf(w, h2f(factor[j / 2] >> (16 * (j & 1))), l[t]);
    }
  }

  // Parts of weights times scales.
  static __device__ __forceinline__ void scaled(u32x4 wh, u32x4 wl, u32x4 d, u32x4& hi, u32x4& lo) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t h, r;
      scale_parts(wh[e], wl[e], d[e], h, r);
      hi[e] = h;
      lo[e] = r;
    }
  }

  // O of the step. value(d): operand of dims 16 d ..; scale(b): the 8 tokens'
  // scales of block b, times the tokens' factors; first: where to leave the
  // weights' first parts. A quantized block's weights are formed while the
  // products of the block before run.
  template <class V, class S>
  __device__ __forceinline__ void accumulate(V value, S scale, const f32x4 (&s)[MT][2], u32x4* first = nullptr) {
    u32x4 wh[MT], wl[MT], ph[2][MT], pl[2][MT];
    u32x4 n0, n1, ns;                           // the next block's values and the scales of its weights, read ahead
    if constexpr (AHEAD) {
      n0 = value(0);
      n1 = value(1);
      if constexpr (KIND != kKvF16) ns = scale(1);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t h, r;
        split_f16(s[t][e / 2][2 * (e & 1)], s[t][e / 2][2 * (e & 1) + 1], h, r);
        wh[t][e] = h;
        wl[t][e] = r;
      }
      if (first) first[t] = wh[t];
      if constexpr (KIND == kKvF16) {
        ph[0][t] = wh[t];
        pl[0][t] = wl[t];
      } else {
        scaled(wh[t], wl[t], scale(0), ph[0][t], pl[0][t]);
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if constexpr (QLDS || AHEAD) __builtin_amdgcn_sched_barrier(0);
      const int now = KIND == kKvF16 ? 0 : b & 1;
      u32x4 v0, v1, vs;
      if constexpr (AHEAD) {
        v0 = n0;
        v1 = n1;
        vs = ns;
        if (b + 1 < NB) {
          n0 = value(2 * b + 2);
          n1 = value(2 * b + 3);
        }
        if (KIND != kKvF16 && b + 2 < NB) ns = scale(b + 2);
        __builtin_amdgcn_sched_barrier(0);
      } else {
        v0 = value(2 * b);
        v1 = value(2 * b + 1);
        if (KIND != kKvF16 && b + 1 < NB) vs = scale(b + 1);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        o[t][2 * b] = mfma_f16(v0, pl[now][t], o[t][2 * b]);
        o[t][2 * b + 1] = mfma_f16(v1, pl[now][t], o[t][2 * b + 1]);
      }
      if (KIND != kKvF16 && b + 1 < NB) {
#pragma unroll
        for (int t = 0; t < MT; ++t) scaled(wh[t], wl[t], vs, ph[now ^ 1][t], pl[now ^ 1][t]);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        o[t][2 * b] = mfma_f16(v0, ph[now][t], o[t][2 * b]);
        o[t][2 * b + 1] = mfma_f16(v1, ph[now][t], o[t][2 * b + 1]);
      }
    }
  }

  // F16: the infinities and NaN among the step's values, which accumulate()
  // meets as zeros, token by token and only into the rows that see them (a
  // weight of 0 times one of them is NaN). Read from the cache again: rare,
  // and few registers.
  __device__ __forceinline__ void add_wild(const AttnArgs& a, const Place& w, int t, int t0, const f32x4 (&s)[MT][2]) {
    const int lane = lane_id(), g = lane >> 4, col = lane & 15;
#pragma unroll 1
    for (int tok = 0; tok < kStep; ++tok) {
      const int pos = t0 + tok, page = a.b.page(w.s, pos);
      if (pos >= w.keys || page < 0) continue;  // uniform
      float own = s[t][0][0];
#pragma unroll
      for (int j = 1; j < 8; ++j) own = (tok & 7) == j ? s[t][j / 4][j & 3] : own;
      const float weight = __shfl(own, (tok >> 3) * 16 + col);
      const bool see = pos <= qpos[t] && (a.window <= 0 || pos > qpos[t] - a.window);
      const uint8_t* unit = a.v + a.b.unit(page, w.head, pos) * kv_unit_bytes(KIND, NB);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        asm volatile("" ::: "memory");          // one tile's loads at a time: registers, not speed
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t v = ld_u16(unit + kv_value_at(KIND, tok & 15, d / 2, 16 * (d & 1) + 4 * g + i));
          if (see && (v & 0x7C00u) == 0x7C00u) o[t][d][i] = fmaf(weight, h2f(v), o[t][d][i]);
        }
      }
    }
  }

  // Quantized: what the step's scales lost by their factors. Read from the
  // cache again: few registers.
  template <class V>
  __device__ __forceinline__ void add_lost(const AttnArgs& a, const Place& w, int t0, V value, u32x4 factor, const u32x4 (&wh)[MT]) {
    const int g = lane_id() >> 4, pos = t0 + 8 * g, page = a.b.page(w.s, pos), real = page < 0 ? 0 : w.keys - pos;
    const uint8_t* unit = a.v + a.b.unit(page < 0 ? 0 : page, w.head, pos) * kv_unit_bytes(KIND, NB);   // a hole's is masked
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      asm volatile("" ::: "memory");            // one block's loads at a time
      u32x4 rest = ld_a16_x4(unit + kv_scale_at(KIND, NB, b, 8 * (g & 1)));
#pragma unroll
      for (int e = 0; e < 4; ++e) rest[e] = lost_f16(rest[e] & keep_mask(e, real), factor[e]);
      if (!__any((rest[0] | rest[1] | rest[2] | rest[3]) != 0)) continue;
      constexpr uint32_t down = ((15u - kLost) << 10) * 0x10001u;
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        u32x4 p;
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = pk_mul_f16(pk_mul_f16(wh[t][e], down), rest[e]);
        o[t][2 * b] = mfma_f16(value(2 * b), p, o[t][2 * b]);
        o[t][2 * b + 1] = mfma_f16(value(2 * b + 1), p, o[t][2 * b + 1]);
      }
    }
  }
};

// Few rows: the waves share the keys.
template <int KIND, int NB, int MT>
__global__ void __launch_bounds__(kAttnThreads, NB < 8 ? 2 : 1) attn_keys_kernel(AttnArgs a) {
  constexpr bool QLDS = NB * MT >= 8 || (KIND == kKvF16 && NB == 4);   // else its registers would leave one wave a SIMD, or spill
  constexpr int D = 32 * NB, DT = 2 * NB, RW = 16 * MT, DP = D + 4;   // rows a bank apart
  // q, and after the walk the waves' O
  __shared__ __attribute__((aligned(16))) float lds_o[4 * RW * DP];
  __shared__ float lds_ml[4 * RW * 2];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id(), g = lane >> 4, col = lane & 15;
  Place w;
  if (!w.find<false>(a)) return;
  for (int tile = w.tile0; tile * RW < w.rows; tile += static_cast<int>(a.tiles.d)) {
    const int row0 = tile * RW, row1 = (row0 + RW < w.rows ? row0 + RW : w.rows) - 1;
    int t_beg, t_end;
    w.range(a, row0, row1, t_beg, t_end);
    const int lo = w.base + a.group.div(row0), hi = w.base + a.group.div(row1);
    int t0 = t_beg + wave * kStep;
    KeyRegs<KIND, NB> kr;
    StepPages pg;
    StepIds next;
    const int zero = vector_zero();
    const int kh = col >> 3, vh = g >> 1;       // halves of the step: of the lane's key row, of its tokens
    if (t0 < t_end) {
      const StepIds ids = step_ids(a, w.s, t0, zero);
      next = step_ids(a, w.s, t0 + 4 * kStep, zero);
      pg = step_pages<KIND, NB>(a, ids, w.head, t0);
      kr.load(a.k + (kh ? pg.off[1] : pg.off[0]), a.k + (vh ? pg.off[1] : pg.off[0]));
    }
    Rows<KIND, NB, MT, QLDS> r;
    if (QLDS) __syncthreads();                  // the tile before is read out
    r.init(a, w, row0, reinterpret_cast<u32x4*>(lds_o));
    if (QLDS) __syncthreads();
    for (; t0 < t_end; t0 += 4 * kStep) {
      if (QLDS) asm volatile("" ::: "memory");  // q is read each step, not kept
      ValueRegs<KIND, NB> vr;
      vr.load(a.v + (vh ? pg.off[1] : pg.off[0]));
      f32x4 s[MT][2];
      r.scores([&](int mm, int b) QMV_INLINE { return kr.operand(mm, b); },
               [&](int b) QMV_INLINE { return kr.sc[KIND == kKvF16 ? 0 : b]; }, s);
      const bool ok0 = pg.ok[0], ok1 = pg.ok[1];
      if (t0 + 4 * kStep < t_end) {
        pg = step_pages<KIND, NB>(a, next, w.head, t0 + 4 * kStep);
        kr.load(a.k + (kh ? pg.off[1] : pg.off[0]), a.k + (vh ? pg.off[1] : pg.off[0]));
        next = step_ids(a, w.s, t0 + 8 * kStep, zero);
      }
      // steps that every row sees whole need no masks
      const bool whole = __all(ok0 && ok1) && t0 + kStep - 1 <= lo && t0 + kStep <= w.keys && (a.window <= 0 || t0 > hi - a.window);
      bool wild = false;
      if (!whole) {
        const int real = (vh ? ok1 : ok0) ? w.keys - (t0 + 8 * g) : 0;   // tokens of this lane that exist
#pragma unroll
        for (int t = 0; t < MT; ++t) r.hide(a, t, t0 + 8 * g, real, s);
        vr.keep(real);
        if constexpr (KIND == kKvF16) {
          wild = __any(vr.wild());              // (of a whole step every row sees them)
          if (wild) vr.tame();
        }
      }
      float e5[8];
      u32x4 factor;
      if constexpr (KIND != kKvF16) vr.normalise(factor, e5);
#pragma unroll
      for (int t = 0; t < MT; ++t) r.weigh(t, factor, e5, r.kTop, s);
      const auto value = [&](int d) QMV_INLINE { return vr.operand(d / 2, d & 1); };
      if constexpr (KIND == kKvF16) {
        if (wild) {
#pragma unroll
          for (int t = 0; t < MT; ++t) r.add_wild(a, w, t, t0, s);
        }
      }
      u32x4 wh[MT];
      r.accumulate(value, [&](int b) QMV_INLINE { return vr.sc[KIND == kKvF16 ? 0 : b]; }, s, wh);
      if constexpr (KIND != kKvF16) {
        const uint32_t low = min_u16x2(min_u16x2(factor[0], factor[1]), min_u16x2(factor[2], factor[3]));
        if (__builtin_expect(__any(below_one(low)), 0)) r.add_lost(a, w, t0, value, factor, wh);
      }
    }

    // the waves' shares joined: each scaled to the common maximum
    __syncthreads();                            // q is not needed any more, the tile before is read out
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const float l = row_sum(r.l[t]);
      if (g == 0) {
        lds_ml[(wave * RW + 16 * t + col) * 2] = r.m[t];
        lds_ml[(wave * RW + 16 * t + col) * 2 + 1] = l;
      }
#pragma unroll
      for (int d = 0; d < DT; ++d)
        *reinterpret_cast<f32x4*>(&lds_o[(wave * RW + 16 * t + col) * DP + 16 * d + 4 * g]) = r.o[t][d];
    }
    __syncthreads();
    for (int it = threadIdx.x; it < RW * (D / 4); it += kAttnThreads) {
      const int rr = it / (D / 4), d = it % (D / 4) * 4, row = row0 + rr;
      if (row >= w.rows) continue;
      float mx = -INFINITY;
#pragma unroll
      for (int v = 0; v < 4; ++v) mx = fmaxf(mx, lds_ml[(v * RW + rr) * 2]);
      const float from = mx == -INFINITY ? 0.0f : mx;
      float ls = 0.0f;
      f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float f = __builtin_amdgcn_exp2f(lds_ml[(v * RW + rr) * 2] - from);
        ls = fmaf(lds_ml[(v * RW + rr) * 2 + 1], f, ls);
        const f32x4 x = *reinterpret_cast<const f32x4*>(&lds_o[(v * RW + rr) * DP + d]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(x[i], f, acc[i]);
      }
      const int tok = a.group.div(row), hd = (w.head - tok) * static_cast<int>(a.group.d) + row;
      store_row<D>(a, w.first + tok, hd, w.split, mx, ls, weight_shift(KIND), [&](float* dst, float f) QMV_INLINE {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = f == 0.0f ? 0.0f : acc[i] * f;
        __builtin_memcpy(__builtin_assume_aligned(dst + d, 4), v, 16);
      }, d == 0);
    }
  }
}

// A 32-key step as operands, in LDS.
template <int KIND, int NB>
struct StepLds {
  u32x4 k[2][NB][kWave];                        // key operands
  u32x4 v[2 * NB][kWave];                       // value operands
  uint32_t ksc[KIND == kKvF16 ? 1 : NB][16];    // scales of the 32 tokens, two a word
  uint32_t vsc[KIND == kKvF16 ? 1 : NB][16];    // times the tokens' factors
  uint32_t factor[16];                          // the factors
  float e5[kStep];                              // and their exponent fields
  int wild[4];                                  // F16, of each wave's share: an infinity or NaN was among the values
                                                // quantized, [0]: a factor of the walk was below 1
};

// A lane's share of a step on its way to LDS: runs of block b of operand lane
// `at`, NB * 64 of them over the workgroup.
template <int KIND, int NB>
struct StepRegs {
  static constexpr int kItems = (NB * kWave + kAttnThreads - 1) / kAttnThreads;
  static constexpr int kKeyWords = kv_run(KIND) / 4;
  static constexpr int kValueWords = KIND == kKvF16 ? 8 : KIND == kKvQ8 ? 4 : 2;
  uint32_t k[kItems][2][kKeyWords], v[kItems][kValueWords];
  uint32_t ksc, vsc[KIND == kKvF16 ? 1 : NB];   // of lanes 0..16 NB-1: word lane % 16, of block lane / 16 and of all blocks
  uint32_t low = ~0u;                           // of lanes 0..15: smallest factors stored
  bool ok[2];

  __device__ __forceinline__ void load(const AttnArgs& a, StepIds ids, int head, int t0) {
    const StepPages pg = step_pages<KIND, NB>(a, ids, head, t0);
    ok[0] = pg.ok[0];
    ok[1] = pg.ok[1];
    const int tid = threadIdx.x;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int it = tid + i * kAttnThreads;
      if (NB * kWave % kAttnThreads && it >= NB * kWave) break;
      const int b = it >> 6, at = it & 63, g = at >> 4, row = at & 15;
      const uint8_t* ku = a.k + (row >> 3 ? pg.off[1] : pg.off[0]);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        constexpr int PS = kv_piece(KIND, NB);
        const int off = b * kv_run(KIND);
        const uint8_t* src = ku + kv_key_piece(KIND, NB, m, off / PS, g, row & 7) + off % PS;
        if constexpr (KIND == kKvF16) {
          const u32x4 r = ld_a16_x4(src);
#pragma unroll
          for (int e = 0; e < 4; ++e) k[i][m][e] = r[e];
        } else if constexpr (KIND == kKvQ8) {
          const u32x2 r = ld_x2(src);
          k[i][m][0] = r.x;
          k[i][m][1] = r.y;
        } else {
          k[i][m][0] = ld_u32(src);
        }
      }
      const uint8_t* vu = a.v + (g >> 1 ? pg.off[1] : pg.off[0]);
      if constexpr (KIND == kKvF16) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const u32x4 r = ld_a16_x4(vu + kv_value_run(KIND, b, half, g & 1, row));
#pragma unroll
          for (int e = 0; e < 4; ++e) v[i][4 * half + e] = r[e];
        }
      } else if constexpr (KIND == kKvQ8) {
        const u32x4 r = ld_a16_x4(vu + kv_value_run(KIND, b, 0, g & 1, row));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] = r[e];
      } else {
        const u32x2 r = ld_x2(vu + kv_value_run(KIND, b, 0, g & 1, row));
        v[i][0] = r.x;
        v[i][1] = r.y;
      }
    }
    if constexpr (KIND != kKvF16) {
      if (tid < 16 * NB) {
        const int b = tid >> 4, word = tid & 15;
        const int64_t off = word >> 3 ? pg.off[1] : pg.off[0];
        ksc = ld_u32(a.k + off + kv_scale_at(KIND, NB, b, 2 * (word & 7)));
#pragma unroll
        for (int i = 0; i < NB; ++i) vsc[i] = ld_u32(a.v + off + kv_scale_at(KIND, NB, i, 2 * (word & 7)));
      }
    }
  }

  // lost: what the value scales lose by their factors, in their place
  __device__ __forceinline__ void store(StepLds<KIND, NB>& lds, int t0, int keys, bool lost) {
    const int tid = threadIdx.x;
    const bool part = !__all(ok[0] && ok[1]) || t0 + kStep > keys;   // slots without a token
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int it = tid + i * kAttnThreads;
      if (NB * kWave % kAttnThreads && it >= NB * kWave) break;
      const int b = it >> 6, at = it & 63, g = at >> 4;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if constexpr (KIND == kKvF16) lds.k[m][b][at] = u32x4{k[i][m][0], k[i][m][1], k[i][m][2], k[i][m][3]};
        else if constexpr (KIND == kKvQ8) lds.k[m][b][at] = operand_q8(k[i][m][0], k[i][m][1]);
        else lds.k[m][b][at] = operand_q4(k[i][m][0], k[i][m][0] >> 4);
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if constexpr (KIND == kKvF16) {
          u32x4 x = {v[i][4 * half], v[i][4 * half + 1], v[i][4 * half + 2], v[i][4 * half + 3]};
          if (part) {
            const int real = (g >> 1 ? ok[1] : ok[0]) ? keys - (t0 + 8 * g) : 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] &= keep_mask(e, real);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            any |= wild_bits(x[e]);
            x[e] = tamed(x[e]);
          }
          lds.v[2 * b + half][at] = x;
        } else if constexpr (KIND == kKvQ8) {
          lds.v[2 * b + half][at] = operand_q8(v[i][2 * half], v[i][2 * half + 1]);
        } else {
          lds.v[2 * b + half][at] = operand_q4(v[i][0] >> (4 * half), v[i][1] >> (4 * half));
        }
      }
    }
    if constexpr (KIND == kKvF16) {
      const bool w = __any(any != 0);
      if (lane_id() == 0) lds.wild[tid >> 6] = w;
    } else {
      if (tid < 16 * NB) {
        const int b = tid >> 4, word = tid & 15;
        lds.ksc[b][word] = ksc;
        const uint32_t mask = part ? keep_mask(0, (word >> 3 ? ok[1] : ok[0]) ? keys - (t0 + 2 * word) : 0) : ~0u;
        uint32_t own = 0, top = 0;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          vsc[i] &= mask;
          own = i == b ? vsc[i] : own;
          top = max_u16x2(top, vsc[i] & 0x7FFF7FFFu);
        }
        const uint32_t f = token_factors(top);
        lds.vsc[b][word] = __builtin_expect(lost, 0) ? lost_f16(own, f) : pk_mul_f16(own, f);
        if (b == 0) {
          low = min_u16x2(low, f);
          lds.factor[word] = f;
          lds.e5[2 * word] = factor_field(f, 0);
          lds.e5[2 * word + 1] = factor_field(f, 1);
        }
      }
    }
  }
};

// Many rows: the waves have rows of their own and share each step's operands.
template <int KIND, int NB, int MT>
__global__ void __launch_bounds__(kAttnThreads, 2) attn_rows_kernel(AttnArgs a) {
  constexpr int D = 32 * NB, DT = 2 * NB, RW = 16 * MT, RT = 4 * RW;
  // Quantized heads of 256 dims: the next step's operands go to LDS before
  // the second product and free their registers for it, and no wave skips a
  // step that none of its rows sees, for the compiler keeps O in memory
  // across that branch (1586 -> 1119 us, 2048 tokens over 8192). Others lose
  // by it, F16 of 256 dims 1238 -> 1664, half-filled tiles of 128 dims 86 -> 93.
  constexpr bool kStraight = KIND != kKvF16 && NB == 8;
  __shared__ StepLds<KIND, NB> lds[2];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id(), g = lane >> 4, col = lane & 15;
  Place w;
  if (!w.find<true>(a)) return;
  for (int tile = w.tile0; tile * RT < w.rows; tile += static_cast<int>(a.tiles.d)) {
    const int row0 = tile * RT + wave * RW;
    int t_beg, t_end;
    w.range(a, tile * RT, (tile * RT + RT < w.rows ? tile * RT + RT : w.rows) - 1, t_beg, t_end);
    // positions of the wave's first and last row; lo > hi where it has none
    const int lo = row0 < w.rows ? w.base + a.group.div(row0) : 1;
    const int hi = row0 < w.rows ? w.base + a.group.div((row0 + RW < w.rows ? row0 + RW : w.rows) - 1) : 0;
    StepRegs<KIND, NB> in;
    StepIds next;
    const int zero = vector_zero();
    const auto begin = [&]() QMV_INLINE {       // the first step's loads
      if (t_beg >= t_end) return;
      const StepIds ids = step_ids(a, w.s, t_beg, zero);
      next = step_ids(a, w.s, t_beg + kStep, zero);
      in.load(a, ids, w.head, t_beg);
    };
    begin();
    Rows<KIND, NB, MT, false, true> r;
    r.init(a, w, row0);
    // What scales lost is added by a second walk: a branch for it in the first
    // costs every step (Q8_0, 2048 tokens over 8192: 128 dims 543 -> 686 us
    // behind the second product and 554 before it, 256 dims 1150 -> 1213). Its
    // weights are those of the first, whose M stands; l is the first one's.
    constexpr bool kTwice = KIND != kKvF16;
    bool again = false;
    float l_first[MT];
    while (true) {
      const bool lost = kTwice && again;
      const float shift = lost ? r.kTop - kLost : r.kTop;
      __syncthreads();                          // the tile or walk before is done with LDS
      if (t_beg < t_end) in.store(lds[0], t_beg, w.keys, lost);
      __syncthreads();
      int buf = 0;
      for (int t0 = t_beg; t0 < t_end; t0 += kStep, buf ^= 1) {
        const bool ok0 = in.ok[0], ok1 = in.ok[1], more = t0 + kStep < t_end;
        if (more) {
          in.load(a, next, w.head, t0 + kStep);
          next = step_ids(a, w.s, t0 + 2 * kStep, zero);
        }
        const StepLds<KIND, NB>& st = lds[buf];
        if (kStraight || (lo <= hi && t0 <= hi && (a.window <= 0 || t0 + kStep > lo - a.window + 1))) {   // some row sees some of it
          f32x4 s[MT][2];
          // products first: of the two waves of a SIMD, one multiplies while the
          // other weighs (2048 tokens over 8192, Q4_0: 597 us without, 580 with
          // the scores first, 544 with both products; of 256 dims Q8_0 1745 us
          // so, 1785 with both)
          __builtin_amdgcn_s_setprio(1);
          r.scores([&](int mm, int b) QMV_INLINE { return st.k[mm][b][lane]; },
                   [&](int b) QMV_INLINE { return *reinterpret_cast<const u32x4*>(&st.ksc[KIND == kKvF16 ? 0 : b][4 * g]); }, s);
          __builtin_amdgcn_s_setprio(0);
          const bool whole = __all(ok0 && ok1) && t0 + kStep - 1 <= lo && t0 + kStep <= w.keys && (a.window <= 0 || t0 > hi - a.window);
          if (!whole) {
            const int real = (g >> 1 ? ok1 : ok0) ? w.keys - (t0 + 8 * g) : 0;
#pragma unroll
            for (int t = 0; t < MT; ++t) r.hide(a, t, t0 + 8 * g, real, s);
          }
          float e5[8];
          u32x4 factor;
          if constexpr (KIND != kKvF16) {
            factor = *reinterpret_cast<const u32x4*>(&st.factor[4 * g]);
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
              const f32x4 x = *reinterpret_cast<const f32x4*>(&st.e5[8 * g + j]);
#pragma unroll
              for (int i = 0; i < 4; ++i) e5[j + i] = x[i];
            }
          }
#pragma unroll
          for (int t = 0; t < MT; ++t) r.weigh(t, factor, e5, shift, s);
          const auto value = [&](int d) QMV_INLINE { return st.v[d][lane]; };
          if constexpr (KIND == kKvF16) {
            if (st.wild[0] | st.wild[1] | st.wild[2] | st.wild[3]) {
#pragma unroll
              for (int t = 0; t < MT; ++t) r.add_wild(a, w, t, t0, s);
            }
          }
          if (kStraight && more) in.store(lds[buf ^ 1], t0 + kStep, w.keys, lost);
          if constexpr (NB < 8) __builtin_amdgcn_s_setprio(1);
          r.accumulate(value, [&](int b) QMV_INLINE {
            return *reinterpret_cast<const u32x4*>(&st.vsc[KIND == kKvF16 ? 0 : b][4 * g]);
          }, s);
          if constexpr (NB < 8) __builtin_amdgcn_s_setprio(0);
        }
        if (!kStraight && more) in.store(lds[buf ^ 1], t0 + kStep, w.keys, lost);
        __syncthreads();
      }
      if (!kTwice || again) break;
      if (wave == 0) {
        const bool low = __any(below_one(in.low));
        if (lane == 0) lds[0].wild[0] = low;
      }
      __syncthreads();
      if (!__builtin_amdgcn_readfirstlane(lds[0].wild[0])) break;
      again = true;
#pragma unroll
      for (int t = 0; t < MT; ++t) l_first[t] = r.l[t];
      begin();
    }
    if (again) {
#pragma unroll
      for (int t = 0; t < MT; ++t) r.l[t] = l_first[t];
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const float l = row_sum(r.l[t]);
      const int row = row0 + 16 * t + col;
      if (row >= w.rows) continue;
      const int tok = a.group.div(row), hd = (w.head - tok) * static_cast<int>(a.group.d) + row;
      store_row<D>(a, w.first + tok, hd, w.split, r.m[t], l, weight_shift(KIND), [&](float* dst, float f) QMV_INLINE {
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          float v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = f == 0.0f ? 0.0f : r.o[t][d][i] * f;
          __builtin_memcpy(__builtin_assume_aligned(dst + 16 * d + 4 * g, 4), v, 16);
        }
      }, g == 0);
    }
  }
}

template <int KIND, int NB, int MT, bool ROWS>
int launch_attn_as(const AttnArgs& a, hipStream_t st) {
  const int64_t groups = static_cast<int64_t>(a.b.n_seqs) * a.splits.d * a.b.n_kv_heads;
  const int64_t grid = (groups + 7) / 8 * 8 * a.tiles.d;
  if (grid > (1 << 23)) return MMVQ_ERR_SHAPE;   // 2^32 lanes in a launch
  const dim3 g(static_cast<unsigned>(grid)), b(kAttnThreads);
  if constexpr (ROWS) {
    // More workgroups than run at once: those of the longest sequences first,
    // so that none of them is what the chip waits for in the end (12 of 200
    // new tokens over 1300..4000: 327 -> 271 us). Few rows gain nothing by it
    // (16 of 5 over 5300..16000: 63.2 and 64.5 us), and short ones lose the
    // time that the order takes (30 of 2 over 700: 20.4 and 23.3).
    AttnArgs args = a;
    args.by_length = a.b.n_seqs > 1 && a.b.n_seqs <= kWave && grid > 2 * kCus;
    hipLaunchKernelGGL((attn_rows_kernel<KIND, NB, MT>), g, b, 0, st, args);
  } else {
    hipLaunchKernelGGL((attn_keys_kernel<KIND, NB, MT>), g, b, 0, st, a);
  }
  return check_launch();
}

template <int KIND, int NB>
int launch_attn_nb(const AttnShape& s, const AttnArgs& a, hipStream_t st) {
  if (s.rows) return launch_attn_as<KIND, NB, NB < 8 ? 2 : 1, true>(a, st);
  if constexpr (NB < 8)
    if (s.mt == 2) return launch_attn_as<KIND, NB, 2, false>(a, st);
  if constexpr (NB == 2)
    if (s.mt == 3) return launch_attn_as<KIND, NB, 3, false>(a, st);
  return launch_attn_as<KIND, NB, 1, false>(a, st);
}

template <int KIND>
int launch_attn_kind(int nb, const AttnShape& s, const AttnArgs& a, hipStream_t st) {
  switch (nb) {
    case 2: return launch_attn_nb<KIND, 2>(s, a, st);
    case 3: return launch_attn_nb<KIND, 3>(s, a, st);
    case 4: return launch_attn_nb<KIND, 4>(s, a, st);
    case 8: return launch_attn_nb<KIND, 8>(s, a, st);
    default: return MMVQ_ERR_SHAPE;
  }
}

}  // namespace qmv
