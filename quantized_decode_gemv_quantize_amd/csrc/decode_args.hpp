// decode_args.hpp - kernel arguments and launchers of the operators between
// the mat-vecs (include/mmvq_decode.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mmvq_decode.h"
#include "decode_plan.hpp"
#include "kv_layout.hpp"

namespace qmv {

// Ragged batch and page geometry on the device side; the checks of the
// values that the host cannot see are here.
struct BatchArgs {
  const int32_t* token_start;
  const int32_t* seq_len;
  const int32_t* page_table;
  int64_t table_stride;
  int n_seqs, n_tokens, pages_per_seq, n_pages;
  int page_shift;     // log2(page_size)
  int n_kv_heads;

  // First row and row count of the sequence with rows a..b-1, inside the activation buffers.
  __device__ __forceinline__ void clamp_rows(int a, int b, int& first, int& count) const {
    first = a < 0 ? 0 : a > n_tokens ? n_tokens : a;
    const int end = b > n_tokens ? n_tokens : b;
    count = end > first ? end - first : 0;
  }
  // Page of a position, -1 for a hole.
  __device__ __forceinline__ int page(int s, int pos) const {
    const int p = pos >> page_shift;
    if (pos < 0 || p >= pages_per_seq) return -1;
    const int id = page_table[static_cast<int64_t>(s) * table_stride + p];
    return id >= 0 && id < n_pages ? id : -1;
  }
  // Unit of a position's 16 tokens in the cache, in units.
  __device__ __forceinline__ int64_t unit(int page, int head, int pos) const {
    const int upp = 1 << (page_shift - 4);
    return (static_cast<int64_t>(page) * n_kv_heads + head) * upp + ((pos >> 4) & (upp - 1));
  }
};

struct KvIoArgs {
  BatchArgs b;
  uint8_t* cache[2];       // keys, values
  float* act[2];           // fp32 rows (read by the writer, written by the reader)
  int64_t ld[2];
};

struct AttnArgs {
  BatchArgs b;
  const uint8_t* k;
  const uint8_t* v;
  const float* q;
  float* out;
  const float* sinks;
  int64_t ldq, ldo;
  float scale_log2;        // scale * log2(e)
  int window, n_heads, head_dim;
  bool by_length;          // workgroups of the longest sequences first
  FastDiv group, tiles, splits, heads;   // query heads a key/value head, ..., key/value heads
  float* part_o;           // [row][head][split][head_dim]
  float2* part_ml;         // [row][head][split]
};

struct VerifyArgs {
  const float* target;
  const float* temperature;
  const float* draft_probs;
  const float* u_accept;
  const float* u_sample;
  const int32_t* draft_tokens;
  const int32_t* row_start;
  int32_t* n_accepted;
  int32_t* tokens;
  int64_t ldt, ldd;
  int vocab, kind, n_seqs, n_rows, max_out, chunks;
  uint8_t* ws;
};

struct NormArgs {
  const float* x;
  const float* res;
  const float* w;
  float* sum;
  float* y;
  uint8_t* yq;
  int64_t ldx, ldr, lds, ldy, n;
  int K;
  double eps, inv_K;
};

int launch_norm(const NormArgs& a, hipStream_t st);
int launch_dequantize_q8_1(const uint8_t* yq, int64_t K, int64_t n, float* x, int64_t ldx, hipStream_t st);
int launch_kv_write(int kind, int nb, const KvIoArgs& a, int max_new, hipStream_t st);
int launch_kv_read(int kind, int nb, const KvIoArgs& a, int max_new, hipStream_t st);
int launch_attn_f16(int nb, const AttnShape& s, const AttnArgs& a, hipStream_t st);
int launch_attn_q8_0(int nb, const AttnShape& s, const AttnArgs& a, hipStream_t st);
int launch_attn_q4_0(int nb, const AttnShape& s, const AttnArgs& a, hipStream_t st);
int launch_attn_join(const AttnArgs& a, bool f16, hipStream_t st);
int64_t verify_bytes(int n_seqs, int n_rows, int vocab, int* chunks);
int launch_verify(const VerifyArgs& a, hipStream_t st);

}  // namespace qmv
