// serve_api.hip - the C ABI declared in include/mmvq_serve.h.
//
// Every entry point validates its arguments on the host and enqueues
// nothing when they are invalid; it never synchronizes and never aborts.
#include "call.hpp"
#include "launch.hpp"
#include "serve_args.hpp"

using namespace qmv;

namespace {

constexpr int kMaxSeqs = 1 << 20, kMaxRows = 1 << 20;

// Elements and bytes of a block of a table's type.
int table_block(int type, int* elems, int* bytes) {
  if (type == MMVQ_F32 || type == MMVQ_F16 || type == MMVQ_BF16) {
    *elems = 1;
    *bytes = type == MMVQ_F32 ? 4 : 2;
    return MMVQ_OK;
  }
  if (type == MMVQ_Q8_1) return MMVQ_ERR_TYPE;   // of activations only
  return mmvq_type_info(type, elems, bytes);
}

int check_pool(const mmvq_kv_pool* pool, int n_seqs, PoolArgs* out) {
  if (!pool) return MMVQ_ERR_NULL;
  if (n_seqs < 0 || n_seqs > kMaxSeqs || pool->n_pages < 1 || pool->page_size < 16 || pool->page_size > MMVQ_KV_MAX_PAGE ||
      (pool->page_size & (pool->page_size - 1)) || pool->pages_per_seq < 1 || pool->pages_per_seq > (1 << 26) ||
      pool->table_stride < pool->pages_per_seq || pool->table_stride > kMaxElems)
    return MMVQ_ERR_SHAPE;
  if (!pool->n_free || !pool->free_pages || (n_seqs > 0 && (!pool->page_table || !pool->pages_held))) return MMVQ_ERR_NULL;
  if (!aligned(pool->n_free, 4) || !aligned(pool->free_pages, 4) || !aligned(pool->page_table, 4) || !aligned(pool->pages_held, 4))
    return MMVQ_ERR_ALIGN;
  *out = PoolArgs{pool->page_table, pool->pages_held, pool->free_pages, pool->n_free, pool->table_stride, pool->pages_per_seq,
                  pool->n_pages, __builtin_ctz(static_cast<unsigned>(pool->page_size))};
  return MMVQ_OK;
}

int check_lora(const mmvq_lora_set* s, int64_t n) {
  if (!s) return MMVQ_ERR_NULL;
  if (s->type != MMVQ_F16 && s->type != MMVQ_BF16 && s->type != MMVQ_F32) return MMVQ_ERR_TYPE;
  if (n < 0 || n > kMaxRows || s->K < 8 || s->K > (1 << 20) || s->K % 8 || s->max_rank < 8 || s->max_rank > 256 || s->max_rank % 8 ||
      s->M < 1 || s->M > kMaxRow || s->n_adapters < 1 || s->n_adapters > (1 << 20))
    return MMVQ_ERR_SHAPE;
  if (s->stride_a < s->max_rank * s->K || s->stride_a > kMaxElems || s->stride_a % 8 || s->stride_b < s->M * s->max_rank ||
      s->stride_b > kMaxElems || s->stride_b % 8)
    return MMVQ_ERR_SHAPE;
  return MMVQ_OK;
}

}  // namespace

extern "C" {

int mmvq_embed(const void* table, int type, int64_t vocab, int64_t K, const int32_t* ids, int64_t n, float scale, float* out,
               int64_t ldo, void* stream) {
  if (n != 0 && (!table || !ids || !out)) return MMVQ_ERR_NULL;
  int elems = 0, bytes = 0;
  const int rc = table_block(type, &elems, &bytes);
  if (rc) return rc;
  if (K < 1 || K > kMaxRow || K % elems || vocab < 1 || vocab > 0x7fffffff || n < 0 || n > kMaxElems / K || ldo < K || ldo > kMaxElems)
    return MMVQ_ERR_SHAPE;
  if (!aligned(table, 16) || !aligned(ids, 4) || !aligned(out, 4)) return MMVQ_ERR_ALIGN;
  if (n == 0) return MMVQ_OK;
  EmbedArgs a{};
  a.table = static_cast<const uint8_t*>(table);
  a.ids = ids;
  a.out = out;
  a.row_bytes = K / elems * bytes;
  a.ldo = ldo;
  a.n = n;
  a.vocab = static_cast<int>(vocab);
  a.K = static_cast<int>(K);
  a.scale = scale;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const OnStreamDevice on(st);
  return launch_embed(type, a, st);
}

int mmvq_kv_release(const mmvq_kv_pool* pool, int n_seqs, const int32_t* keep, const int32_t* shared, void* stream) {
  ReleaseArgs a{};
  const int rc = check_pool(pool, n_seqs, &a.p);
  if (rc) return rc;
  if (n_seqs > 0 && !keep) return MMVQ_ERR_NULL;
  if (!aligned(keep, 4) || !aligned(shared, 4)) return MMVQ_ERR_ALIGN;
  if (n_seqs == 0) return MMVQ_OK;
  a.keep = keep;
  a.shared = shared;
  a.n_seqs = n_seqs;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const OnStreamDevice on(st);
  return launch_release(a, st);
}

int mmvq_kv_plan_workspace(int n_seqs, int64_t* bytes) {
  if (!bytes) return MMVQ_ERR_NULL;
  if (n_seqs < 0 || n_seqs > kMaxSeqs) return MMVQ_ERR_SHAPE;
  *bytes = plan_bytes(n_seqs);
  return MMVQ_OK;
}

int mmvq_kv_plan(const mmvq_kv_pool* pool, const int32_t* cached, const int32_t* n_new, int n_seqs, int n_rows, int32_t* token_start,
                 int32_t* seq_len, int32_t* row_seq, int32_t* row_pos, int64_t* row_slot, int32_t* n_missing, void* workspace,
                 int64_t workspace_bytes, void* stream) {
  PlanArgs a{};
  const int rc = check_pool(pool, n_seqs, &a.p);
  if (rc) return rc;
  if (!token_start || !workspace || (n_seqs > 0 && (!cached || !n_new || !seq_len))) return MMVQ_ERR_NULL;
  if (n_rows < 0 || n_rows > kMaxRows || workspace_bytes < plan_bytes(n_seqs)) return MMVQ_ERR_SHAPE;
  if (!aligned(cached, 4) || !aligned(n_new, 4) || !aligned(token_start, 4) || !aligned(seq_len, 4) || !aligned(row_seq, 4) ||
      !aligned(row_pos, 4) || !aligned(row_slot, 8) || !aligned(n_missing, 4) || !aligned(workspace, 16))
    return MMVQ_ERR_ALIGN;
  a.cached = cached;
  a.n_new = n_new;
  a.start = token_start;
  a.len = seq_len;
  a.row_seq = row_seq;
  a.row_pos = row_pos;
  a.row_slot = row_slot;
  a.missing = n_missing;
  a.n_seqs = n_seqs;
  a.n_rows = n_rows;
  a.off = static_cast<int64_t*>(workspace);
  a.held = reinterpret_cast<int32_t*>(a.off + n_seqs + 3);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const OnStreamDevice on(st);
  return launch_plan(a, st);
}

int mmvq_lora_workspace(const mmvq_lora_set* set, int64_t n, int64_t* bytes) {
  if (!bytes) return MMVQ_ERR_NULL;
  const int rc = check_lora(set, n);
  if (rc) return rc;
  *bytes = lora_bytes(n, set->K, set->M, set->max_rank);
  return MMVQ_OK;
}

int mmvq_lora(const mmvq_lora_set* set, const float* x, int64_t ldx, int64_t n, const int32_t* row_seq, const int32_t* adapter,
              int n_seqs, const float* base, int64_t ldb, float* out, int64_t ldo, void* workspace, int64_t workspace_bytes,
              void* stream) {
  const int rc = check_lora(set, n);
  if (rc) return rc;
  if (n != 0 && (!set->A || !set->B || !x || !base || !out || !workspace || (n_seqs > 0 && !adapter))) return MMVQ_ERR_NULL;
  if (ldx < set->K || ldx > kMaxElems || ldb < set->M || ldb > kMaxElems || ldo < set->M || ldo > kMaxElems || n_seqs < 0 ||
      (!row_seq && n_seqs < n) || (base == out && base && ldb != ldo) ||
      workspace_bytes < lora_bytes(n, set->K, set->M, set->max_rank))
    return MMVQ_ERR_SHAPE;
  if (!aligned(set->A, 16) || !aligned(set->B, 16) || !aligned(set->rank, 4) || !aligned(set->scale, 4) || !aligned(x, 4) ||
      !aligned(row_seq, 4) || !aligned(adapter, 4) || !aligned(base, 4) || !aligned(out, 4) || !aligned(workspace, 16))
    return MMVQ_ERR_ALIGN;
  if (n == 0) return MMVQ_OK;
  LoraArgs a{};
  a.A = static_cast<const uint8_t*>(set->A);
  a.B = static_cast<const uint8_t*>(set->B);
  a.rank = set->rank;
  a.scale = set->scale;
  a.x = x;
  a.base = base;
  a.out = out;
  a.row_seq = row_seq;
  a.adapter = adapter;
  a.stride_a = set->stride_a;
  a.stride_b = set->stride_b;
  a.ldx = ldx;
  a.ldb = ldb;
  a.ldo = ldo;
  a.K = set->K;
  a.M = set->M;
  a.n = static_cast<int>(n);
  a.n_seqs = n_seqs;
  a.n_adapters = set->n_adapters;
  a.max_rank = set->max_rank;
  a.part = static_cast<float*>(workspace);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const OnStreamDevice on(st);
  return launch_lora(set->type, a, st);
}

int mmvq_sample_workspace(int n_rows, int vocab, int64_t* bytes) {
  if (!bytes) return MMVQ_ERR_NULL;
  if (n_rows < 0 || n_rows > kMaxRows || vocab < 1 || vocab > kMaxRow) return MMVQ_ERR_SHAPE;
  *bytes = sample_bytes(n_rows, vocab, nullptr);
  return MMVQ_OK;
}

int mmvq_sample(const float* logits, int64_t ldl, int vocab, int n_rows, const mmvq_sampling* params, const int32_t* row_seq,
                int n_seqs, const float* u, int32_t* tokens, float* chosen, float* probs, int64_t ldp, void* workspace,
                int64_t workspace_bytes, void* stream) {
  if (n_rows != 0 && (!logits || !workspace || (!tokens && !chosen && !probs) || ((tokens || chosen) && !u))) return MMVQ_ERR_NULL;
  int64_t need = 0;
  const int rc = mmvq_sample_workspace(n_rows, vocab, &need);
  if (rc) return rc;
  if (ldl < vocab || ldl > kMaxElems || (probs && (ldp < vocab || ldp > kMaxElems)) || (probs == logits && probs && ldp != ldl) ||
      n_seqs < 0 || (!row_seq && n_seqs < n_rows) || workspace_bytes < need)
    return MMVQ_ERR_SHAPE;
  SampleArgs a{};
  if (params) {
    a.temperature = params->temperature;
    a.top_k = params->top_k;
    a.top_p = params->top_p;
    a.min_p = params->min_p;
  }
  if (!aligned(logits, 4) || !aligned(a.temperature, 4) || !aligned(a.top_k, 4) || !aligned(a.top_p, 4) || !aligned(a.min_p, 4) ||
      !aligned(row_seq, 4) || !aligned(u, 4) || !aligned(tokens, 4) || !aligned(chosen, 4) || !aligned(probs, 4) ||
      !aligned(workspace, 16))
    return MMVQ_ERR_ALIGN;
  if (n_rows == 0) return MMVQ_OK;
  a.logits = logits;
  a.row_seq = row_seq;
  a.u = u;
  a.tokens = tokens;
  a.chosen = chosen;
  a.probs = probs;
  a.ldl = ldl;
  a.ldp = ldp;
  a.vocab = vocab;
  a.n_rows = n_rows;
  a.n_seqs = n_seqs;
  a.zeroed = probs && probs != logits;
  sample_bytes(n_rows, vocab, &a.chunks);
  a.ws = static_cast<uint8_t*>(workspace);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const OnStreamDevice on(st);
  return launch_sample(a, st);
}

}  // extern "C"
