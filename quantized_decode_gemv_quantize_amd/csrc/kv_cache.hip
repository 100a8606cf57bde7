// kv_cache.hip - new tokens' keys and values into the paged cache, and back.
//
// A workgroup owns one unit (16 tokens of one head, keys or values): it
// quantizes the rows that fall into it (8 lanes a 32-value block, 4 values a
// lane, reductions over the 8 lanes by DPP), arranges the unit in LDS and
// copies out what belongs to the new tokens: 16-byte stores where the unit
// is all new, the tokens' own bytes otherwise. The arrangement transposes
// the values, which in memory would be stores of single bytes. Long prompts
// are bound by memory bandwidth (4 bytes a value in, 0.56 to 2 out), single
// tokens by latency.
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

// Quantizes value quad `sub` of block b of token tt into the unit image.
template <int KIND, int NB, bool KEYS>
__device__ __forceinline__ void put_quad(uint8_t* img, int tt, int b, int sub, const float (&x)[4]) {
  const int c = 4 * sub;
  if constexpr (KIND == kKvF16) {
    uint16_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = static_cast<uint16_t>(f2h_bits(x[e]));
    if constexpr (KEYS) {
      *reinterpret_cast<u32x2*>(img + kv_key_at(KIND, NB, tt, b, c)) =
          u32x2{h[0] | static_cast<uint32_t>(h[1]) << 16, h[2] | static_cast<uint32_t>(h[3]) << 16};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) *reinterpret_cast<uint16_t*>(img + kv_value_at(KIND, tt, b, c + e)) = h[e];
    }
  } else {
    float d;
    uint32_t w;
    bool mine = true;
    if constexpr (KIND == kKvQ8) {
      const u32x4 raw[1] = {{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])}};
      float amax = absmax4(raw[0]);
      amax = fmaxf(amax, dpp_f<kDppXor1>(amax));
      amax = fmaxf(amax, dpp_f<kDppXor2>(amax));
      amax = fmaxf(amax, dpp_f<kDppMirror8>(amax));
      d = q8_scale(amax);
      uint32_t packed[1];
      int sum = 0;
      q8_quant_block(raw, d, packed, sum);
      w = packed[0] ^ 0x80808080u;                 // q + 128
    } else {
      d = q4_most(x) / -8.0f;
      w = q4_codes(x, d);
      const uint32_t o = from_half(w);
      w = w | (o << 4);                            // lower half of the lanes: its nibbles and those 16 dims on
      mine = sub < 4;
    }
    if (mine) {
      if constexpr (KEYS) {
        *reinterpret_cast<uint32_t*>(img + kv_key_at(KIND, NB, tt, b, c)) = w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) img[kv_value_at(KIND, tt, b, c + e)] = static_cast<uint8_t>(w >> (8 * e));
      }
    }
    if (sub == 0) *reinterpret_cast<uint16_t*>(img + kv_scale_at(KIND, NB, b, tt)) = static_cast<uint16_t>(f2h_bits(fminf(fmaxf(d, -65504.0f), 65504.0f)));
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

template <int KIND, int NB, bool KEYS>
__device__ __forceinline__ void write_units(const KvIoArgs& a, uint8_t* img) {
  constexpr int U = kv_unit_bytes(KIND, NB), C = kv_code_bytes(KIND, NB);
  const int head = blockIdx.y >> 1, tid = threadIdx.x;
  const float* act = a.act[KEYS ? 0 : 1];
  const int64_t ld = a.ld[KEYS ? 0 : 1];
  uint8_t* cache = a.cache[KEYS ? 0 : 1];
  for (int s = blockIdx.z; s < a.b.n_seqs; s += gridDim.z) {
    int row0, count;
    a.b.rows(s, row0, count);
    const int len = a.b.seq_len[s] > 0 ? a.b.seq_len[s] : 0;
    const int p0 = len - count;
    for (int base = ((p0 >> 4) + static_cast<int>(blockIdx.x)) * 16; base < len; base += 16 * static_cast<int>(gridDim.x)) {
      const int page = a.b.page(s, base);
      if (count == 0 || page < 0) continue;
      const int ta = p0 > base ? p0 - base : 0, tb = len - base < 16 ? len - base : 16;
      __syncthreads();                             // the image of the unit before is copied out
      for (int it = tid; it < (tb - ta) * NB * 8; it += 256) {
        const int tt = ta + it / (NB * 8), b = it / 8 % NB, sub = it & 7;
        const u32x4 r = ld_x4(reinterpret_cast<const uint8_t*>(
            act + (row0 + (base + tt - p0)) * ld + head * (32 * NB) + 32 * b + 4 * sub));
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(r[e]);
        put_quad<KIND, NB, KEYS>(img, tt, b, sub, x);
      }
      __syncthreads();
      uint8_t* dst = cache + a.b.unit(page, head, base) * U;
      if (ta == 0 && tb == 16) {
        for (int o = 16 * tid; o < U; o += 16 * 256)
          *reinterpret_cast<u32x4*>(dst + o) = *reinterpret_cast<const u32x4*>(img + o);
      } else {
        if constexpr (KEYS) {
          for (int w = tid; w < C / 4; w += 256) {
            const int tt = kv_key_token(KIND, NB, w);
            if (tt >= ta && tt < tb) reinterpret_cast<uint32_t*>(dst)[w] = reinterpret_cast<const uint32_t*>(img)[w];
          }
        } else {
          // elements of 8 tokens lie together: element e is of token 8 h8 + e % 8
          const int n = tb - ta;
          for (int it = tid; it < n * (C / 16 / (KIND == kKvF16 ? 2 : 1)); it += 256) {
            const int tt = ta + it % n, e = it / n;
            const int run = KIND == kKvQ8 ? e / 32 * 4 + tt / 8 * 2 + 0 : e / 16 * 2 + tt / 8;
            int at;
            if constexpr (KIND == kKvQ8) at = ((run >> 1) * 32 + e % 32) * 8 + tt % 8;
            else at = (run * 16 + e % 16) * 8 + tt % 8;
            if constexpr (KIND == kKvF16) reinterpret_cast<uint16_t*>(dst)[at] = reinterpret_cast<const uint16_t*>(img)[at];
            else dst[at] = img[at];
          }
        }
        if constexpr (KIND != kKvF16) {
          const int n = tb - ta;
          for (int it = tid; it < n * NB; it += 256) {
            const int o = kv_scale_at(KIND, NB, it / n, ta + it % n);
            *reinterpret_cast<uint16_t*>(dst + o) = *reinterpret_cast<const uint16_t*>(img + o);
          }
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
    int row0, count;
    a.b.rows(s, row0, count);
    const int len = a.b.seq_len[s] > 0 ? a.b.seq_len[s] : 0;
    const int p0 = len - count;
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
  __shared__ UnitLds<KIND, NB> img;
  if constexpr (WRITE) {
    if (blockIdx.y & 1) write_units<KIND, NB, false>(a, img.bytes);
    else write_units<KIND, NB, true>(a, img.bytes);
  } else {
    if (blockIdx.y & 1) read_units<KIND, NB, false>(a, img.bytes);
    else read_units<KIND, NB, true>(a, img.bytes);
  }
}

template <int KIND, bool WRITE>
int launch_io(int nb, const KvIoArgs& a, int max_new, hipStream_t st) {
  const int units = (max_new + 14) / 16 + 1;       // a run of max_new tokens touches at most so many
  const dim3 grid(static_cast<unsigned>(units), static_cast<unsigned>(2 * a.b.n_kv_heads),
                  static_cast<unsigned>(a.b.n_seqs < 65535 ? a.b.n_seqs : 65535));
  switch (nb) {
    case 2: hipLaunchKernelGGL((kv_io_kernel<KIND, 2, WRITE>), grid, dim3(256), 0, st, a); break;
    case 3: hipLaunchKernelGGL((kv_io_kernel<KIND, 3, WRITE>), grid, dim3(256), 0, st, a); break;
    case 4: hipLaunchKernelGGL((kv_io_kernel<KIND, 4, WRITE>), grid, dim3(256), 0, st, a); break;
    case 8: hipLaunchKernelGGL((kv_io_kernel<KIND, 8, WRITE>), grid, dim3(256), 0, st, a); break;
    default: return MMVQ_ERR_SHAPE;
  }
  return check_launch();
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
