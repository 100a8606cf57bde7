// kv_layout.hpp - layout of a paged key/value cache: where a token's value
// lies in its page. Shared by the cache's writer and reader, the attention
// kernels and the host model of the tests.
//
// A page holds, for every key/value head, page_size/16 units of 16 tokens. A
// unit is its codes followed (quantized types) by fp16 block scales
// [head_dim/32][16 tokens]. The attention kernels multiply 32 keys a step
// with 16x16x32 matrix instructions, S^T = K q^T and O^T = V^T P^T, whose
// operands hold 8 consecutive contraction elements a lane (lane = 16 g + r):
//   keys    row r of tile m is token 8 (r/4) + 4 m + r%4, so that the score
//           tiles leave lane group g with tokens 8g..8g+7 of its query, which
//           is the operand layout of P in the second product: no value moves
//           between lanes. A lane's runs of the head's 32-value blocks lie
//           together and the pieces of the 8 rows of a lane group side by
//           side: [m][piece][g][rr = r%8][piece bytes].
//   values  transposed, 8 tokens together: [block][half of 16][tokens 8 h8..]
//           [r][8 tokens], the two halves of a block interleaved for Q8_0
//           (one 16-byte load) and in the two nibbles of a byte for Q4_0.
// Every operand load is then one aligned, fully used run of 4 to 16 bytes,
// and a 32-token step may span two pages (pages of 16 tokens) because each
// half of it comes from its own unit.
#pragma once

#include <stdint.h>

#ifndef QMV_HOST_MODEL
#include <hip/hip_runtime.h>
#define KV_HD __host__ __device__ __forceinline__
#define KV_DEV __device__ __forceinline__
#else
#define KV_HD inline
#define KV_DEV inline
#endif

namespace qmv {

enum KvKind { kKvF16 = 0, kKvQ8 = 1, kKvQ4 = 2 };

constexpr int kUnitTokens = 16;

// Bytes of a lane's run of one 32-value block (8 values).
KV_HD constexpr int kv_run(int kind) { return kind == kKvF16 ? 16 : kind == kKvQ8 ? 8 : 4; }
KV_HD constexpr int kv_lane_bytes(int kind, int nb) { return kv_run(kind) * nb; }
// Widest load that divides a lane's bytes.
KV_HD constexpr int kv_piece(int kind, int nb) {
  return kv_lane_bytes(kind, nb) % 16 == 0 ? 16 : kv_lane_bytes(kind, nb) % 8 == 0 ? 8 : 4;
}
KV_HD constexpr int kv_code_bytes(int kind, int nb) { return 64 * kv_lane_bytes(kind, nb); }   // 2 m, 4 g, 8 rr
KV_HD constexpr int kv_unit_bytes(int kind, int nb) {
  return kv_code_bytes(kind, nb) + (kind == kKvF16 ? 0 : 32 * nb);
}
// Byte of block b's scale of token tt (quantized types).
KV_HD constexpr int kv_scale_at(int kind, int nb, int b, int tt) {
  return kv_code_bytes(kind, nb) + (b * kUnitTokens + tt) * 2;
}

// Byte of the key element: dim 32 b + c of token tt (Q4_0: the byte whose low
// nibble is dim c % 16 and whose high nibble is 16 dims further).
KV_HD constexpr int kv_key_at(int kind, int nb, int tt, int b, int c) {
  const int ps = kv_piece(kind, nb);
  const int g = kind == kKvQ4 ? c % 16 / 4 : c / 8;
  const int off = b * kv_run(kind) + (kind == kKvQ4 ? c % 4 : kind == kKvF16 ? c % 8 * 2 : c % 8);
  const int m = tt / 4 % 2, rr = tt / 8 * 4 + tt % 4;
  return (((m * (kv_lane_bytes(kind, nb) / ps) + off / ps) * 4 + g) * 8 + rr) * ps + off % ps;
}
// Byte of the value element (Q4_0: as above).
KV_HD constexpr int kv_value_at(int kind, int tt, int b, int c) {
  const int half = c / 16, r = c % 16, h8 = tt / 8, j = tt % 8;
  return kind == kKvF16  ? ((((b * 2 + half) * 2 + h8) * 16 + r) * 8 + j) * 2
         : kind == kKvQ8 ? (((b * 2 + h8) * 16 + r) * 2 + half) * 8 + j
                         : ((b * 2 + h8) * 16 + r) * 8 + j;
}
// Byte of piece p of lane group g, row rr of key tile m; a lane's pieces in
// turn are its runs of the blocks in turn.
KV_HD constexpr int kv_key_piece(int kind, int nb, int m, int p, int g, int rr) {
  const int ps = kv_piece(kind, nb);
  return (((m * (kv_lane_bytes(kind, nb) / ps) + p) * 4 + g) * 8 + rr) * ps;
}
// Byte of a lane's values of block b (F16: of each 16-dim half) for tokens
// 8 h8..: 8 tokens of dim r, of both halves for the quantized types.
KV_HD constexpr int kv_value_run(int kind, int b, int half, int h8, int r) {
  return kind == kKvF16 ? (((b * 2 + half) * 2 + h8) * 16 + r) * 16
                        : ((b * 2 + h8) * 16 + r) * (kind == kKvQ8 ? 16 : 8);
}

}  // namespace qmv
