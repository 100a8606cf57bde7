// kv_cache.hip - new tokens' keys and values into the paged cache, and back.
//
// Writer: eight lanes hold a 32-value block, 4 dims each, of 8 consecutive
// tokens: eight loads at once, reductions over the block by DPP. Keys go out
// token by token, values, which a unit holds transposed, as runs of 8 tokens
// after a transposition in registers (in LDS it meets 8-way bank
// conflicts). A run that is not all new is stored as the new tokens' own
// bytes. Reader: a workgroup takes a unit through LDS. Long prompts are bound
// by memory bandwidth (4 bytes a value in, 0.56 to 2 out: 8058 tokens of 8
// heads of 128, each alone, F16 22.0 us written and 22.7 read, Q8_0 16.8 and
// 20.9, Q4_0 19.3 and 16.6; F16 in turn 29 and 18, where the reader finds some
// of it in the caches), single tokens by latency.
#include "decode_args.hpp"
#include "launch.hpp"
#include "q8.hpp"

namespace qmv {

// Four code nibbles of a value quad (Q4_0): min(15, floor(x/d + 8.5)), 8
// where d is 0, in the low four bits of each byte.
__device__ __forceinline__ uint32_t q4_codes(const float (&x)[4], float d) {
  const bool z = d == 0.0f;
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float t = floorf(x[e] / (z ? 1.0f : d) + 8.5f);
    const int q = z ? 8 : static_cast<int>(fminf(fmaxf(t, 0.0f), 15.0f));
    w |= static_cast<uint32_t>(q) << (8 * e);
  }
  return w;
}

// Word of the lane 4 away in the group of 8.
__device__ __forceinline__ uint32_t from_half(uint32_t v) {
  const int m = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), kDppMirror8, 0xF, 0xF, false);   // lane ^ 7
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, m, 0x1B, 0xF, 0xF, false));            // lane ^ 3
}

// The value of largest magnitude of the block, the first of equals.
__device__ __forceinline__ float q4_most(const float (&x)[4]) {
  float m = x[0];
#pragma unroll
  for (int e = 1; e < 4; ++e) m = fabsf(x[e]) > fabsf(m) ? x[e] : m;
  // lane order is value order: across a lane bit the lower lane wins a tie
  const int l = lane_id();
  const auto step = [&](float o, bool upper) QMV_INLINE {
    const bool take = upper ? fabsf(o) >= fabsf(m) : fabsf(o) > fabsf(m);
    m = take ? o : m;
  };
  step(dpp_f<kDppXor1>(m), l & 1);
  step(dpp_f<kDppXor2>(m), l & 2);
  // every lane of a quad holds the quad's value now: any lane of the other quad will do
  step(dpp_f<kDppMirror8>(m), l & 4);
  return m;
}

template <int KIND, int NB>
struct UnitLds {
  alignas(16) uint8_t bytes[kv_unit_bytes(KIND, NB)];
};

__device__ __forceinline__ uint32_t scale_bits(float d) { return f2h_bits(fminf(fmaxf(d, -65504.0f), 65504.0f)); }

// Codes of the lane's quad of a block, as a unit stores them (a byte each),
// and the block's d.
template <int KIND>
__device__ __forceinline__ float quad_codes(const float (&x)[4], uint32_t& w) {
  if constexpr (KIND == kKvQ8) {
    const u32x4 raw[1] = {{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])}};
    float amax = absmax4(raw[0]);
    amax = fmaxf(amax, dpp_f<kDppXor1>(amax));
    amax = fmaxf(amax, dpp_f<kDppXor2>(amax));
    amax = fmaxf(amax, dpp_f<kDppMirror8>(amax));
    const float d = q8_scale_product(amax);
    uint32_t packed[1];
    int sum = 0;
    q8_quant_block(raw, d, packed, sum);
    w = packed[0] ^ 0x80808080u;                   // q + 128
    return d;
  } else {
    const float d = q4_most(x) / -8.0f;
    w = q4_codes(x, d);
    return d;
  }
}

// The values of quad `sub`, from the image of a unit.
template <int KIND, int NB, bool KEYS>
__device__ __forceinline__ void get_quad(const uint8_t* img, int tt, int b, int sub, float (&x)[4]) {
  const int c = 4 * sub;
  const float d = KIND == kKvF16 ? 1.0f : h2f(ld_u16(img + kv_scale_at(KIND, NB, b, tt)));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint8_t* p = img + (KEYS ? kv_key_at(KIND, NB, tt, b, c + e) : kv_value_at(KIND, tt, b, c + e));
    if constexpr (KIND == kKvF16) x[e] = h2f(ld_u16(p));
    else if constexpr (KIND == kKvQ8) x[e] = d * static_cast<float>(static_cast<int>(*p) - 128);
    else x[e] = d * static_cast<float>((c < 16 ? *p & 15 : *p >> 4) - 8);
  }
}

// Units that a sequence's new tokens touch.
struct Run {
  int row0, count, len, p0;
  __device__ __forceinline__ Run(const BatchArgs& b, int s) {
    const int from = b.token_start[s], to = b.token_start[s + 1], l = b.seq_len[s];
    b.clamp_rows(from, to, row0, count);
    len = l < 0 ? 0 : l > (1 << 30) ? (1 << 30) : l;
    p0 = len - count;
  }
};

// 4x4 bytes: word e of the result holds byte e of the four words.
__device__ __forceinline__ void transpose4(const uint32_t (&w)[4], uint32_t (&t)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
  const uint32_t c = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
  t[0] = __builtin_amdgcn_perm(b, a, 0x05040100u);
  t[1] = __builtin_amdgcn_perm(b, a, 0x07060302u);
  t[2] = __builtin_amdgcn_perm(d, c, 0x05040100u);
  t[3] = __builtin_amdgcn_perm(d, c, 0x07060302u);
}

template <int KIND, int NB, bool KEYS>
__device__ __forceinline__ void write_units(const KvIoArgs& a) {
  constexpr int W = KEYS ? 0 : 1;
  constexpr int U = kv_unit_bytes(KIND, NB), L = 16 * NB, GROUPS = 256 / L;   // lanes a unit, units a workgroup
  const int head = blockIdx.x >> 1, tid = threadIdx.x, grp = tid / L, lane = tid - grp * L;
  const int h8 = lane / (8 * NB), b = lane / 8 % NB, sub = lane & 7;
  if (grp >= GROUPS) return;
  for (int s = blockIdx.z; s < a.b.n_seqs; s += gridDim.z) {
    const Run r(a.b, s);
    const int first = (r.p0 >> 4) + static_cast<int>(blockIdx.y) * GROUPS + grp;
    for (int base = first * 16; base < r.len; base += 16 * GROUPS * static_cast<int>(gridDim.y)) {
      const int ta = r.p0 - base - 8 * h8, tb = r.len - base - 8 * h8;   // tokens j of the lane's 8: ta <= j < tb
      if (r.count == 0 || ta >= 8 || tb <= 0) continue;
      u32x4 raw[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        raw[j] = u32x4{0u, 0u, 0u, 0u};
        if (j >= ta && j < tb)
          raw[j] = ld_x4(reinterpret_cast<const uint8_t*>(
              a.act[W] + (r.row0 + (base + 8 * h8 + j - r.p0)) * a.ld[W] + head * (32 * NB) + 32 * b + 4 * sub));
      }
      const int page = a.b.page(s, base);          // the rows are on their way
      if (page < 0) continue;
      float x[8][4];
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[j][e] = __uint_as_float(raw[j][e]);
      uint8_t* dst = a.cache[W] + a.b.unit(page, head, base) * U;
      const bool full = ta <= 0 && tb >= 8;
      if constexpr (KIND == kKvF16 && KEYS) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j >= ta && j < tb)
            *reinterpret_cast<u32x2*>(dst + kv_key_at(KIND, NB, 8 * h8 + j, b, 4 * sub)) =
                u32x2{f2h_bits(x[j][0]) | (f2h_bits(x[j][1]) << 16), f2h_bits(x[j][2]) | (f2h_bits(x[j][3]) << 16)};
      } else if constexpr (KIND == kKvF16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = f2h_bits(x[2 * j][e]) | (f2h_bits(x[2 * j + 1][e]) << 16);
          uint8_t* to = dst + kv_value_at(KIND, 8 * h8, b, 4 * sub + e);
          if (full) *reinterpret_cast<u32x4*>(to) = u32x4{w[0], w[1], w[2], w[3]};
          else
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j >= ta && j < tb) reinterpret_cast<uint16_t*>(to)[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
        }
      } else {
        uint32_t code[8], ds[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          code[j] = 0;
          if (j >= ta && j < tb)                   // the same for the block's 8 lanes; one token's step does one
            ds[j / 2] |= scale_bits(quad_codes<KIND>(x[j], code[j])) << (16 * (j & 1));
        }
        if constexpr (KEYS) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j >= ta && j < tb) {
              // the lower half of the lanes: its nibbles and those 16 dims on
              if constexpr (KIND == kKvQ4) code[j] |= from_half(code[j]) << 4;
              if (KIND == kKvQ8 || sub < 4)
                *reinterpret_cast<uint32_t*>(dst + kv_key_at(KIND, NB, 8 * h8 + j, b, 4 * sub)) = code[j];
            }
        } else {
          uint32_t lo[4], hi[4];
          transpose4({code[0], code[1], code[2], code[3]}, lo);
          transpose4({code[4], code[5], code[6], code[7]}, hi);
          if constexpr (KIND == kKvQ4) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              lo[e] |= from_half(lo[e]) << 4;
              hi[e] |= from_half(hi[e]) << 4;
            }
          }
          if (KIND == kKvQ8 || sub < 4) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint8_t* to = dst + kv_value_at(KIND, 8 * h8, b, 4 * sub + e);
              if (full) *reinterpret_cast<u32x2*>(to) = u32x2{lo[e], hi[e]};
              else
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  if (j >= ta && j < tb) to[j] = static_cast<uint8_t>((j < 4 ? lo[e] : hi[e]) >> (8 * (j & 3)));
            }
          }
        }
        if (sub == 0) {
          uint8_t* to = dst + kv_scale_at(KIND, NB, b, 8 * h8);
          if (full) *reinterpret_cast<u32x4*>(to) = u32x4{ds[0], ds[1], ds[2], ds[3]};
          else
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j >= ta && j < tb) reinterpret_cast<uint16_t*>(to)[j] = static_cast<uint16_t>(ds[j / 2] >> (16 * (j & 1)));
        }
      }
    }
  }
}

template <int KIND, int NB, bool KEYS>
__device__ __forceinline__ void read_units(const KvIoArgs& a, uint8_t* img) {
  constexpr int U = kv_unit_bytes(KIND, NB);
  const int head = blockIdx.y >> 1, tid = threadIdx.x;
  float* act = a.act[KEYS ? 0 : 1];
  const int64_t ld = a.ld[KEYS ? 0 : 1];
  if (!act) return;
  const uint8_t* cache = a.cache[KEYS ? 0 : 1];
  for (int s = blockIdx.z; s < a.b.n_seqs; s += gridDim.z) {
    const Run r(a.b, s);
    const int row0 = r.row0, count = r.count, len = r.len, p0 = r.p0;
    for (int base = ((p0 >> 4) + static_cast<int>(blockIdx.x)) * 16; base < len; base += 16 * static_cast<int>(gridDim.x)) {
      if (count == 0) continue;
      const int page = a.b.page(s, base);
      const int ta = p0 > base ? p0 - base : 0, tb = len - base < 16 ? len - base : 16;
      __syncthreads();                             // the image before is read
      if (page >= 0) {
        const uint8_t* src = cache + a.b.unit(page, head, base) * U;
        for (int o = 16 * tid; o < U; o += 16 * 256)
          *reinterpret_cast<u32x4*>(img + o) = *reinterpret_cast<const u32x4*>(src + o);
      }
      __syncthreads();
      for (int it = tid; it < (tb - ta) * NB * 8; it += 256) {
        const int tt = ta + it / (NB * 8), b = it / 8 % NB, sub = it & 7;
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (page >= 0) get_quad<KIND, NB, KEYS>(img, tt, b, sub, x);
        float* p = act + (row0 + (base + tt - p0)) * ld + head * (32 * NB) + 32 * b + 4 * sub;
        __builtin_memcpy(__builtin_assume_aligned(p, 4), x, 16);
      }
    }
  }
}

template <int KIND, int NB, bool WRITE>
__global__ void __launch_bounds__(256) kv_io_kernel(KvIoArgs a) {
  if constexpr (WRITE) {
    if (blockIdx.x & 1) write_units<KIND, NB, false>(a);
    else write_units<KIND, NB, true>(a);
  } else {
    __shared__ UnitLds<KIND, NB> img;
    if (blockIdx.y & 1) read_units<KIND, NB, false>(a, img.bytes);
    else read_units<KIND, NB, true>(a, img.bytes);
  }
}

template <int KIND, int NB, bool WRITE>
int launch_io_as(const KvIoArgs& a, int max_new, hipStream_t st) {
  const int units = units_of(max_new);
  constexpr int PER = WRITE ? 256 / (16 * NB) : 1; // units a workgroup
  // The writer has the heads side by side, so that the rows of one unit's
  // tokens are read together (31.7 -> 29.5 us for 8192 F16 tokens of 8 heads
  // of 128); the reader goes along a head's pages (20.0 against 18.1).
  const unsigned groups = static_cast<unsigned>((units + PER - 1) / PER), heads = static_cast<unsigned>(2 * a.b.n_kv_heads);
  const unsigned seqs = static_cast<unsigned>(a.b.n_seqs < 65535 ? a.b.n_seqs : 65535);
  const dim3 grid = WRITE ? dim3(heads, groups < 65535 ? groups : 65535, seqs) : dim3(groups, heads, seqs);
  hipLaunchKernelGGL((kv_io_kernel<KIND, NB, WRITE>), grid, dim3(256), 0, st, a);
  return check_launch();
}

template <int KIND, bool WRITE>
int launch_io(int nb, const KvIoArgs& a, int max_new, hipStream_t st) {
  switch (nb) {
    case 2: return launch_io_as<KIND, 2, WRITE>(a, max_new, st);
    case 3: return launch_io_as<KIND, 3, WRITE>(a, max_new, st);
    case 4: return launch_io_as<KIND, 4, WRITE>(a, max_new, st);
    case 8: return launch_io_as<KIND, 8, WRITE>(a, max_new, st);
    default: return MMVQ_ERR_SHAPE;
  }
}

int launch_kv_write(int kind, int nb, const KvIoArgs& a, int max_new, hipStream_t st) {
  return kind == kKvF16  ? launch_io<kKvF16, true>(nb, a, max_new, st)
         : kind == kKvQ8 ? launch_io<kKvQ8, true>(nb, a, max_new, st)
                         : launch_io<kKvQ4, true>(nb, a, max_new, st);
}

int launch_kv_read(int kind, int nb, const KvIoArgs& a, int max_new, hipStream_t st) {
  return kind == kKvF16  ? launch_io<kKvF16, false>(nb, a, max_new, st)
         : kind == kKvQ8 ? launch_io<kKvQ8, false>(nb, a, max_new, st)
                         : launch_io<kKvQ4, false>(nb, a, max_new, st);
}

}  // namespace qmv
