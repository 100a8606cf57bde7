// attn_kernel.hpp - attention of new tokens over the paged cache.
//
//   out = sum_t softmax(scale q.k_t) v_t over the visible keys t
//
// The query heads that share a key/value head are rows of one product
// (row = token * group + head of the group), so a cache byte is read once for
// all of them. A wave owns MT tiles of 16 rows and walks the keys 32 at a
// time with the running maximum m, sum l and unnormalised O of a softmax:
//   S^T = K q^T     two 16x16 tiles of 16x16x32 fp16 products; a lane then
//                   holds the scores of ONE row (lane % 16) for the 8 tokens
//                   8g..8g+7 of the step (g = lane / 16)
//   O^T += V^T P^T  whose right operand is exactly that: the probabilities
//                   stay in their lanes, and m, l and the rescaling of O are
//                   one value a lane
// The cache is stored in operand order (kv_layout.hpp): operands go from
// memory to registers in full 4 to 16-byte runs, without LDS. Quantized
// codes are exact in fp16 (keys) and bf16 (values); a key's block scale is
// applied to the block's partial score, a value's block scale to P.
//
// Precision: fp32 q is carried as two fp16 parts of the row scaled by a
// power of two (21 bits of the row's largest value); P as two fp16 parts
// (F16 cache, P scaled by 2^14 so that small ones keep their bits; the scale
// cancels in O / l) or, P times the value's scale, as two bf16 parts (2^-16;
// bf16 for its range, since scales reach from 2^-24 to 65504). Scores, m, l
// and O are fp32.
//
// Two splits of the work over a workgroup's 4 waves: with few rows the waves
// take every fourth step of the same rows and join O through LDS (ROWS =
// false); with many each wave has rows of its own and the waves meet in the
// cache only (ROWS = true). Either way the keys can be cut into a.splits
// ranges whose partial (m, l, O) a second launch joins, so that few rows over
// a long cache still fill the chip.
#pragma once

#include "decode_args.hpp"
#include "launch.hpp"

namespace qmv {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kAttnThreads = 256;
constexpr int kStep = 32;                       // keys a step
constexpr float kPShift = 14.0f;                // P of an F16 cache is scaled by 2^14

__device__ __forceinline__ f32x4 mfma_f16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
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

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const half2v h = {static_cast<_Float16>(a), static_cast<_Float16>(b)};
  return __builtin_bit_cast(uint32_t, h);
}
// Two values as fp16 parts: hi toward zero, lo the nearest of the rest (together 21 bits).
__device__ __forceinline__ void split_f16(float a, float b, uint32_t& hi, uint32_t& lo) {
  const auto h = __builtin_amdgcn_cvt_pkrtz(a, b);
  hi = __builtin_bit_cast(uint32_t, h);
  lo = pack_f16(a - static_cast<float>(h[0]), b - static_cast<float>(h[1]));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {   // nearest
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 h = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, h);
}
// Two values as bf16 parts, each the nearest: together within 2^-16. Cutting
// toward zero would cost as much and lean every probability the same way.
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(a, b);
  lo = pack_bf16(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {   // values that are exact in bf16
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

// fp16 of four biased codes (bytes): 1024 + u by its bits, less the bias.
__device__ __forceinline__ void codes_f16(uint32_t w, float bias, uint32_t& lo, uint32_t& hi) {
  const _Float16 b = static_cast<_Float16>(-1024.0f - bias);
  const half2v off = {b, b};
  lo = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) + off);
  hi = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) + off);
}
__device__ __forceinline__ void codes_bf16(uint32_t w, float bias, uint32_t& lo, uint32_t& hi) {
  lo = bf16_pair(static_cast<float>(w & 0xFFu) - bias, static_cast<float>((w >> 8) & 0xFFu) - bias);
  hi = bf16_pair(static_cast<float>((w >> 16) & 0xFFu) - bias, static_cast<float>(w >> 24) - bias);
}

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
        const uint8_t* src = unit + (((m * NP + p) * 4 + g) * 8 + (l & 7)) * PS;
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
    u32x4 r;
    if constexpr (KIND == kKvF16) {
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = w[m * LW + 4 * b + e];
    } else if constexpr (KIND == kKvQ8) {
      uint32_t t[4];
      codes_f16(w[m * LW + 2 * b], 128.0f, t[0], t[1]);
      codes_f16(w[m * LW + 2 * b + 1], 128.0f, t[2], t[3]);
      r = u32x4{t[0], t[1], t[2], t[3]};
    } else {
      const uint32_t v = w[m * LW + b];
      uint32_t t[4];
      codes_f16(v & 0x0F0F0F0Fu, 8.0f, t[0], t[1]);
      codes_f16((v >> 4) & 0x0F0F0F0Fu, 8.0f, t[2], t[3]);
      r = u32x4{t[0], t[1], t[2], t[3]};
    }
    return r;
  }
  __device__ __forceinline__ float scale(int b, int j) const { return h2f(sc[b][j / 2] >> (16 * (j & 1))); }
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
          const u32x4 v = ld_a16_x4(unit + (((b * 2 + half) * 2 + h8) * 16 + r) * 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[8 * b + 4 * half + e] = v[e];
        }
      } else if constexpr (KIND == kKvQ8) {
        const u32x4 v = ld_a16_x4(unit + ((b * 2 + h8) * 16 + r) * 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * b + e] = v[e];
      } else {
        const u32x2 v = ld_x2(unit + ((b * 2 + h8) * 16 + r) * 8);
        w[2 * b] = v.x;
        w[2 * b + 1] = v.y;
      }
      if constexpr (KIND != kKvF16) sc[b] = ld_a16_x4(unit + kv_scale_at(KIND, NB, b, 8 * h8));
    }
  }
  // operand of dims 32 b + 16 half ..: fp16 (F16) or bf16
  __device__ __forceinline__ u32x4 operand(int b, int half) const {
    u32x4 r;
    if constexpr (KIND == kKvF16) {
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = w[8 * b + 4 * half + e];
    } else {
      uint32_t t[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t v;
        if constexpr (KIND == kKvQ8) v = w[4 * b + 2 * half + e];
        else v = (w[2 * b + e] >> (4 * half)) & 0x0F0F0F0Fu;
        codes_bf16(v, KIND == kKvQ8 ? 128.0f : 8.0f, t[2 * e], t[2 * e + 1]);
      }
      r = u32x4{t[0], t[1], t[2], t[3]};
    }
    return r;
  }
  __device__ __forceinline__ float scale(int b, int j) const { return h2f(sc[b][j / 2] >> (16 * (j & 1))); }

  // F16: tokens c.. of this lane's 8 do not exist (what lies there is no value): zero.
  __device__ __forceinline__ void keep(int c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t mask = c >= 2 * e + 2 ? ~0u : c == 2 * e + 1 ? 0xFFFFu : 0u;
#pragma unroll
      for (int t = 0; t < 2 * NB; ++t) w[4 * t + e] &= mask;
    }
  }
  // F16: whether any value is infinite or NaN
  __device__ __forceinline__ bool wild() const {
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < NB * kPer; ++i) any |= ((w[i] & 0x7FFF7FFFu) + 0x04000400u) & 0x80008000u;
    return any != 0;
  }
};

// Where the units of a 32-key step lie; 16-token halves may be holes.
struct StepPages {
  const uint8_t* k[2];
  const uint8_t* v[2];
  bool ok[2];
};

template <int KIND, int NB>
__device__ __forceinline__ StepPages step_pages(const AttnArgs& a, int s, int head, int t0) {
  constexpr int U = kv_unit_bytes(KIND, NB);
  StepPages p;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int pos = t0 + 16 * h, page = a.b.page(s, pos);
    p.ok[h] = page >= 0;
    const int64_t off = a.b.unit(page < 0 ? 0 : page, head, pos) * U;   // a hole's loads go to page 0 and are masked
    p.k[h] = a.k + off;
    p.v[h] = a.v + off;
  }
  return p;
}

// 1 / (sum of the row's probabilities), its sink among them; 0 for a row
// that saw no key. m and l are in units of log2, l scaled by 2^shift.
__device__ __forceinline__ float row_factor(const AttnArgs& a, int head, float m, float l, float shift) {
  if (m == -INFINITY) return 0.0f;
  if (a.sinks) l += __builtin_amdgcn_exp2f(fmaf(a.sinks[head], 1.44269504088896340736f, shift - m));
  return 1.0f / l;
}

// A finished row to out, or a split's share of it to the workspace. `write`
// stores this lane's values times a factor from the row's first float on.
template <int D, class W>
__device__ __forceinline__ void store_row(const AttnArgs& a, int token, int head, int split, float m, float l,
                                          float shift, W write, bool lead) {
  if (a.splits == 1) {
    write(a.out + token * a.ldo + static_cast<int64_t>(head) * D, row_factor(a, head, m, l, shift));
  } else {
    const int64_t at = (static_cast<int64_t>(token) * a.n_heads + head) * a.splits + split;
    write(a.part_o + at * D, 1.0f);
    if (lead) a.part_ml[at] = make_float2(m, l);
  }
}

template <int KIND, int NB, int MT, bool ROWS>
__global__ void __launch_bounds__(kAttnThreads) attn_kernel(AttnArgs a) {
  constexpr int D = 32 * NB, DT = 2 * NB;
  constexpr int RW = 16 * MT;                   // rows a wave
  constexpr int RT = ROWS ? 4 * RW : RW;        // rows a workgroup
  constexpr float kShift = KIND == kKvF16 ? kPShift : 0.0f;
  __shared__ float lds_o[ROWS ? 1 : 4 * RW * D];
  __shared__ float lds_ml[ROWS ? 1 : 4 * RW * 2];

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane_id(), g = l >> 4, col = l & 15;
  // Workgroups go to the 8 XCDs in turn: those that read the same keys (the
  // tiles of one sequence, head and range) get the same XCD and its L2.
  const int slot = blockIdx.x >> 3;
  int group_id = (slot / a.tiles) * 8 + (blockIdx.x & 7);
  const int tile0 = a.tiles - 1 - slot % a.tiles;   // the longest rows first
  if (group_id >= a.b.n_seqs * a.splits * a.b.n_kv_heads) return;
  const int head = group_id % a.b.n_kv_heads;
  group_id /= a.b.n_kv_heads;
  const int split = group_id % a.splits, s = group_id / a.splits;

  int first, count;
  a.b.rows(s, first, count);
  const int len = a.b.seq_len[s] < 0 ? 0 : a.b.seq_len[s] > (1 << 30) ? (1 << 30) : a.b.seq_len[s];
  const int64_t table_end = static_cast<int64_t>(a.b.pages_per_seq) << a.b.page_shift;
  const int keys = len < table_end ? len : static_cast<int>(table_end);
  const int rows = count * a.group;             // count <= 2^20, group <= 2^16: see the host check

  for (int tile = tile0; tile * RT < rows; tile += a.tiles) {
    const int row0 = tile * RT + (ROWS ? wave * RW : 0);
    // positions of the workgroup's and the wave's rows
    const int wg_last = (tile * RT + RT < rows ? tile * RT + RT : rows) - 1;
    const int w_last = row0 + RW - 1 < rows ? row0 + RW - 1 : rows - 1;
    const int base = len - count;               // position of new token 0
    const int hi_wg = base + wg_last / a.group, lo_wg = base + tile * RT / a.group;
    const int hi = base + w_last / a.group;
    const int lo = base + (row0 < rows ? row0 : rows - 1) / a.group;
    // the split's range of the keys that the workgroup sees, in steps
    int k_end = hi_wg + 1 < keys ? hi_wg + 1 : keys;
    const int k_beg = a.window > 0 && lo_wg - a.window + 1 > 0 ? (lo_wg - a.window + 1) & ~(kStep - 1) : 0;
    const int steps = k_end > k_beg ? (k_end - k_beg + kStep - 1) / kStep : 0;
    const int per = (steps + a.splits - 1) / a.splits;
    int t_beg = k_beg + split * per * kStep;
    int t_end = k_beg + (split + 1 < a.splits ? (split + 1) * per : steps) * kStep;
    if (t_end > k_beg + steps * kStep) t_end = k_beg + steps * kStep;
    if constexpr (ROWS) {                       // and of those the wave's own
      if (row0 >= rows) t_end = t_beg;
      else if (hi + 1 < t_end) t_end = hi + 1;
      if (a.window > 0 && lo - a.window + 1 > t_beg) t_beg += (lo - a.window + 1 - t_beg) & ~(kStep - 1);
    }

    // q as fp16 parts of its row scaled to 2^13..2^14
    u32x4 qh[MT][NB], ql[MT][NB];
    float to_log2[MT];
    int qpos[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int row = row0 + 16 * t + col;
      const bool live = row < rows;
      const int tok = live ? row / a.group : 0, hd = head * a.group + (live ? row - tok * a.group : 0);
      qpos[t] = live ? base + tok : -1;
      const float* src = a.q + (first + tok) * a.ldq + static_cast<int64_t>(hd) * D;
      float v[NB][8], top = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int d0 = 32 * b + (KIND == kKvQ4 ? 4 * g : 8 * g), d1 = KIND == kKvQ4 ? d0 + 16 : d0 + 4;
        const u32x4 x = ld_x4(reinterpret_cast<const uint8_t*>(src + d0));
        const u32x4 y = ld_x4(reinterpret_cast<const uint8_t*>(src + d1));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[b][e] = live ? __uint_as_float(x[e]) : 0.0f;
          v[b][4 + e] = live ? __uint_as_float(y[e]) : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[b][e]));
      }
      top = row_max(top);
      int ex = static_cast<int>((__float_as_uint(top) >> 23) & 0xFFu) - 127;   // 2^ex <= top < 2^(ex+1)
      ex = top == 0.0f || ex == 128 ? 13 : ex < -100 ? -100 : ex;
      const float up = __uint_as_float(static_cast<uint32_t>(13 - ex + 127) << 23);
      to_log2[t] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(ex - 13 + 127) << 23);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t h, lo2;
          split_f16(v[b][2 * e] * up, v[b][2 * e + 1] * up, h, lo2);
          qh[t][b][e] = h;
          ql[t][b][e] = lo2;
        }
    }

    float m[MT], lsum[MT];
    f32x4 o[MT][DT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      m[t] = -INFINITY;
      lsum[t] = 0.0f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[t][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    const int stride = ROWS ? kStep : 4 * kStep;
    int t0 = t_beg + (ROWS ? 0 : wave * kStep);
    KeyRegs<KIND, NB> kr;
    StepPages pg;
    const int kh = col >> 3, vh = g >> 1;       // halves of the step: of the lane's key row, of its tokens
    if (t0 < t_end) {
      pg = step_pages<KIND, NB>(a, s, head, t0);
      kr.load(kh ? pg.k[1] : pg.k[0], vh ? pg.k[1] : pg.k[0]);
    }
    for (; t0 < t_end; t0 += stride) {
      ValueRegs<KIND, NB> vr;
      vr.load(vh ? pg.v[1] : pg.v[0]);
      // scores
      float p[MT][8];
#pragma unroll
      for (int mm = 0; mm < 2; ++mm) {
        f32x4 sc[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) sc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const u32x4 kop = kr.operand(mm, b);
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            if constexpr (KIND == kKvF16) {
              sc[t] = mfma_f16(kop, ql[t][b], sc[t]);
              sc[t] = mfma_f16(kop, qh[t][b], sc[t]);
            } else {
              f32x4 acc = mfma_f16(kop, ql[t][b], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
              acc = mfma_f16(kop, qh[t][b], acc);
#pragma unroll
              for (int i = 0; i < 4; ++i) sc[t][i] = fmaf(acc[i], kr.scale(b, 4 * mm + i), sc[t][i]);
            }
          }
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) p[t][4 * mm + i] = sc[t][i] * to_log2[t];
      }
      const bool ok0 = pg.ok[0], ok1 = pg.ok[1];
      const int tn = t0 + stride;
      if (tn < t_end) {
        pg = step_pages<KIND, NB>(a, s, head, tn);
        kr.load(kh ? pg.k[1] : pg.k[0], vh ? pg.k[1] : pg.k[0]);
      }
      // what a row does not see; steps that every row sees whole skip this
      const bool whole = ok0 && ok1 && t0 + kStep - 1 <= lo && t0 + kStep <= keys &&
                         (a.window <= 0 || t0 > hi - a.window);
      bool wild = false;
      const int kpos = t0 + 8 * g;
      if (!whole) {
        const bool ok = vh ? ok1 : ok0;
        const int real = ok ? keys - kpos : 0;  // tokens of this lane that exist
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int k = kpos + j;
            const bool see = j < real && k <= qpos[t] && (a.window <= 0 || k > qpos[t] - a.window);
            p[t][j] = see ? p[t][j] : -INFINITY;
          }
        if constexpr (KIND == kKvF16) {
          vr.keep(real);
          wild = __any(vr.wild());
        }
      }
      // running maximum and sum
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        float top = p[t][0];
#pragma unroll
        for (int j = 1; j < 8; ++j) top = fmaxf(top, p[t][j]);
        top = fmaxf(m[t], row_max(top));
        const float from = top == -INFINITY ? 0.0f : top;   // a row that has seen nothing yet
        if (__any(top != m[t])) {
          const float al = __builtin_amdgcn_exp2f(m[t] - from);
          lsum[t] *= al;
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[t][d][i] *= al;
          m[t] = top;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          p[t][j] = __builtin_amdgcn_exp2f(p[t][j] - from + kShift);
          lsum[t] += p[t][j];
        }
      }
      // O
      if constexpr (KIND == kKvF16) {
        u32x4 ph[MT], pl[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t h, lo2;
            split_f16(p[t][2 * e], p[t][2 * e + 1], h, lo2);
            ph[t][e] = h;
            pl[t][e] = lo2;
          }
        if (!wild) {
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const u32x4 vop = vr.operand(b, half);
#pragma unroll
              for (int t = 0; t < MT; ++t) {
                o[t][2 * b + half] = mfma_f16(vop, pl[t], o[t][2 * b + half]);
                o[t][2 * b + half] = mfma_f16(vop, ph[t], o[t][2 * b + half]);
              }
            }
        } else {
          // an infinity or NaN among the values: one token after the other,
          // added only to the rows that see it (0 * inf is NaN)
          for (int tok = 0; tok < kStep; ++tok) {
            const bool mine = (tok >> 3) == g;
            const int k = t0 + tok;
            u32x4 mask = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mask[e] = mine && (tok & 7) >> 1 == e ? (tok & 1 ? 0xFFFF0000u : 0xFFFFu) : 0u;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              const bool see = k <= qpos[t] && (a.window <= 0 || k > qpos[t] - a.window);
#pragma unroll
              for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                  const u32x4 vop = vr.operand(b, half) & mask;
                  f32x4 acc = mfma_f16(vop, pl[t] & mask, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
                  acc = mfma_f16(vop, ph[t] & mask, acc);
#pragma unroll
                  for (int i = 0; i < 4; ++i) o[t][2 * b + half][i] += see ? acc[i] : 0.0f;
                }
            }
          }
        }
      } else {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          u32x4 ph[MT], pl[MT];
#pragma unroll
          for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float x = p[t][2 * e] * vr.scale(b, 2 * e), y = p[t][2 * e + 1] * vr.scale(b, 2 * e + 1);
              if (!whole) {                     // an unseen token's scale may be anything
                x = p[t][2 * e] == 0.0f ? 0.0f : x;
                y = p[t][2 * e + 1] == 0.0f ? 0.0f : y;
              }
              uint32_t h, lo2;
              split_bf16(x, y, h, lo2);
              ph[t][e] = h;
              pl[t][e] = lo2;
            }
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const u32x4 vop = vr.operand(b, half);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              o[t][2 * b + half] = mfma_bf16(vop, pl[t], o[t][2 * b + half]);
              o[t][2 * b + half] = mfma_bf16(vop, ph[t], o[t][2 * b + half]);
            }
          }
        }
      }
    }

#pragma unroll
    for (int t = 0; t < MT; ++t) lsum[t] = row_sum(lsum[t]);

    if constexpr (ROWS) {
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int row = row0 + 16 * t + col;
        if (row >= rows) continue;
        const int tok = row / a.group, hd = head * a.group + row - tok * a.group;
        store_row<D>(a, first + tok, hd, split, m[t], lsum[t], kShift, [&](float* dst, float f) QMV_INLINE {
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = f == 0.0f ? 0.0f : o[t][d][i] * f;
            __builtin_memcpy(__builtin_assume_aligned(dst + 16 * d + 4 * g, 4), v, 16);
          }
        }, g == 0);
      }
    } else {
      // the waves' shares joined: each scaled to the common maximum
      __syncthreads();                          // the tile before is read out
#pragma unroll
      for (int t = 0; t < MT; ++t)
        if (g == 0) {
          lds_ml[(wave * RW + 16 * t + col) * 2] = m[t];
          lds_ml[(wave * RW + 16 * t + col) * 2 + 1] = lsum[t];
        }
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int d = 0; d < DT; ++d)
          *reinterpret_cast<f32x4*>(&lds_o[(wave * RW + 16 * t + col) * D + 16 * d + 4 * g]) = o[t][d];
      __syncthreads();
      for (int it = threadIdx.x; it < RW * (D / 4); it += kAttnThreads) {
        const int r = it / (D / 4), d = it % (D / 4) * 4, row = row0 + r;
        if (row >= rows) continue;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) mx = fmaxf(mx, lds_ml[(w * RW + r) * 2]);
        const float from = mx == -INFINITY ? 0.0f : mx;
        float ls = 0.0f;
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float f = __builtin_amdgcn_exp2f(lds_ml[(w * RW + r) * 2] - from);
          ls = fmaf(lds_ml[(w * RW + r) * 2 + 1], f, ls);
          const f32x4 x = *reinterpret_cast<const f32x4*>(&lds_o[(w * RW + r) * D + d]);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = fmaf(x[i], f, acc[i]);
        }
        const int tok = row / a.group, hd = head * a.group + row - tok * a.group;
        store_row<D>(a, first + tok, hd, split, mx, ls, kShift, [&](float* dst, float f) QMV_INLINE {
          float v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = f == 0.0f ? 0.0f : acc[i] * f;
          __builtin_memcpy(__builtin_assume_aligned(dst + d, 4), v, 16);
        }, d == 0);
      }
    }
  }
}

template <int KIND, int NB, int MT, bool ROWS>
int launch_attn_as(const AttnArgs& a, hipStream_t st) {
  const int64_t groups = static_cast<int64_t>(a.b.n_seqs) * a.splits * a.b.n_kv_heads;
  const int64_t grid = (groups + 7) / 8 * 8 * a.tiles;
  if (grid > (1 << 23)) return MMVQ_ERR_SHAPE;   // 2^32 lanes in a launch
  hipLaunchKernelGGL((attn_kernel<KIND, NB, MT, ROWS>), dim3(static_cast<unsigned>(grid)), dim3(kAttnThreads), 0, st, a);
  return check_launch();
}

template <int KIND, int NB>
int launch_attn_nb(const AttnShape& s, const AttnArgs& a, hipStream_t st) {
  if constexpr (NB < 8) {
    if (s.mt == 2) return s.rows ? launch_attn_as<KIND, NB, 2, true>(a, st) : launch_attn_as<KIND, NB, 2, false>(a, st);
    return launch_attn_as<KIND, NB, 1, false>(a, st);
  } else {
    return s.rows ? launch_attn_as<KIND, NB, 1, true>(a, st) : launch_attn_as<KIND, NB, 1, false>(a, st);
  }
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
