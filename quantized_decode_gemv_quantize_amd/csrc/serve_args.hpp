// serve_args.hpp - kernel arguments and launchers of the operators of a step
// over many requests (include/mmvq_serve.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mmvq_serve.h"
#include "serve_plan.hpp"

namespace qmv {

struct EmbedArgs {
  const uint8_t* table;
  const int32_t* ids;
  float* out;
  int64_t row_bytes, ldo, n, units;   // units: rows times pieces of a row
  int vocab, K;
  float scale;
  int pieces;              // of a row
  bool past, through;      // out passes the caches by, or the L2 only
};

struct PoolArgs {
  int32_t* table;
  int32_t* held;
  int32_t* free;
  int32_t* n_free;
  int64_t stride;
  int pages_per_seq, n_pages, shift;
};

struct ReleaseArgs {
  PoolArgs p;
  const int32_t* keep;
  const int32_t* shared;
  int n_seqs;
};

struct PlanArgs {
  PoolArgs p;
  const int32_t* cached;
  const int32_t* n_new;
  int32_t* start;
  int32_t* len;
  int32_t* row_seq;
  int32_t* row_pos;
  int64_t* row_slot;
  int32_t* missing;
  int n_seqs, n_rows;
  int64_t* off;            // workspace: n_seqs + 1 sums of the pages needed, then {given, free before}
  int32_t* held;           // workspace: pages held before, n_seqs
};

struct LoraArgs {
  const uint8_t* A;
  const uint8_t* B;
  const int32_t* rank;
  const float* scale;
  const float* x;
  const float* base;
  float* out;
  const int32_t* row_seq;
  const int32_t* adapter;
  int64_t stride_a, stride_b, ldx, ldb, ldo, K, M;
  int n, n_seqs, n_adapters, max_rank;
  int splits, steps;       // ranges of K, and chunks of one
  int pieces;              // of M, of a slice
  int leads;               // rows of a block that a workgroup looks for tiles at
  bool past;               // out passes the caches by
  float* part;             // [split][row][max_rank]
};

struct SampleArgs {
  const float* logits;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const int32_t* row_seq;
  const float* u;
  int32_t* tokens;
  float* chosen;
  float* probs;
  int64_t ldl, ldp;
  int vocab, n_rows, n_seqs, chunks;
  bool zeroed;             // probs are no part of logits: written on the way
  bool past;               // probs pass the caches by
  uint8_t* ws;
};

int launch_embed(int type, const EmbedArgs& a, hipStream_t st);
int launch_release(const ReleaseArgs& a, hipStream_t st);
int64_t plan_bytes(int n_seqs);
int launch_plan(const PlanArgs& a, hipStream_t st);
int64_t lora_bytes(int64_t n, int64_t K, int64_t M, int max_rank);
int launch_lora(int type, const LoraArgs& a, hipStream_t st);
int64_t sample_bytes(int n_rows, int vocab, int* chunks);
int launch_sample(const SampleArgs& a, hipStream_t st);

}  // namespace qmv
