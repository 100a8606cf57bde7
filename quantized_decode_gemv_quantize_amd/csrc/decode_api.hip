// decode_api.hip - the C ABI declared in include/mmvq_decode.h.
//
// Every entry point validates its arguments on the host and enqueues
// nothing when they are invalid; it never synchronizes and never aborts.
#include <math.h>

#include "call.hpp"
#include "decode_args.hpp"
#include "launch.hpp"

using namespace qmv;

namespace {

int kv_kind(int type) {
  return type == MMVQ_F16 ? kKvF16 : type == MMVQ_Q8_0 ? kKvQ8 : type == MMVQ_Q4_0 ? kKvQ4 : -1;
}

int check_pages(int type, int page_size, int n_kv_heads, int head_dim) {
  if (kv_kind(type) < 0) return MMVQ_ERR_TYPE;
  if (page_size < 16 || page_size > MMVQ_KV_MAX_PAGE || (page_size & (page_size - 1))) return MMVQ_ERR_SHAPE;
  if (n_kv_heads < 1 || n_kv_heads > 1024) return MMVQ_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 96 && head_dim != 128 && head_dim != 256) return MMVQ_ERR_SHAPE;
  return MMVQ_OK;
}

// Host-visible geometry of a cache and a batch.
int check_shapes(const mmvq_kv_cache* c, const mmvq_kv_batch* b) {
  if (!c || !b) return MMVQ_ERR_NULL;
  const int rc = check_pages(c->type, c->page_size, c->n_kv_heads, c->head_dim);
  if (rc) return rc;
  if (c->n_pages < 1) return MMVQ_ERR_SHAPE;
  if (b->n_seqs < 0 || b->n_seqs > (1 << 20) || b->n_tokens < 0 || b->n_tokens > (1 << 20)) return MMVQ_ERR_SHAPE;
  if (b->max_new < 1 || b->max_new > (1 << 20) || b->max_len < 1 || b->max_len > (1 << 30)) return MMVQ_ERR_SHAPE;
  if (b->pages_per_seq < 1 || b->pages_per_seq > (1 << 26) || b->table_stride < b->pages_per_seq) return MMVQ_ERR_SHAPE;
  return MMVQ_OK;
}

// Nothing to do: buffers that have no element then may have no address.
bool empty(const mmvq_kv_batch* b) { return b->n_seqs == 0 || b->n_tokens == 0; }

int check_kv(const mmvq_kv_cache* c, const mmvq_kv_batch* b, BatchArgs* out) {
  const int rc = check_shapes(c, b);
  if (rc) return rc;
  if (!c->k || !c->v || !b->token_start || (b->n_seqs > 0 && (!b->seq_len || !b->page_table))) return MMVQ_ERR_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return MMVQ_ERR_ALIGN;
  if (!aligned(b->token_start, 4) || !aligned(b->seq_len, 4) || !aligned(b->page_table, 4)) return MMVQ_ERR_ALIGN;
  *out = BatchArgs{b->token_start, b->seq_len, b->page_table, b->table_stride, b->n_seqs, b->n_tokens,
                   b->pages_per_seq, c->n_pages, __builtin_ctz(static_cast<unsigned>(c->page_size)), c->n_kv_heads};
  return MMVQ_OK;
}

int kv_io(const mmvq_kv_cache* c, const mmvq_kv_batch* b, float* k, int64_t ldk, float* v, int64_t ldv, bool write,
          void* stream) {
  KvIoArgs a{};
  const int rc = check_kv(c, b, &a.b);
  if (rc) return rc;
  if (!empty(b) && (write ? !k || !v : !k && !v)) return MMVQ_ERR_NULL;
  const int64_t width = static_cast<int64_t>(c->n_kv_heads) * c->head_dim;
  if (((k || write) && (ldk < width || ldk > kMaxElems)) || ((v || write) && (ldv < width || ldv > kMaxElems)))
    return MMVQ_ERR_SHAPE;
  if (!aligned(k, 4) || !aligned(v, 4)) return MMVQ_ERR_ALIGN;
  if (empty(b)) return MMVQ_OK;
  a.cache[0] = static_cast<uint8_t*>(c->k);
  a.cache[1] = static_cast<uint8_t*>(c->v);
  a.act[0] = k;
  a.act[1] = v;
  a.ld[0] = ldk;
  a.ld[1] = ldv;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const OnStreamDevice on(st);
  return write ? launch_kv_write(kv_kind(c->type), c->head_dim / 32, a, b->max_new, st)
               : launch_kv_read(kv_kind(c->type), c->head_dim / 32, a, b->max_new, st);
}

int check_attn(const mmvq_kv_cache* c, const mmvq_kv_batch* b, int n_heads) {
  const int rc = check_shapes(c, b);
  if (rc) return rc;
  if (n_heads < 1 || n_heads > 65535 || n_heads % c->n_kv_heads) return MMVQ_ERR_SHAPE;
  if (static_cast<int64_t>(b->n_tokens) * n_heads > (1 << 30)) return MMVQ_ERR_SHAPE;
  return MMVQ_OK;
}

AttnShape shape_of(const mmvq_kv_cache* c, const mmvq_kv_batch* b, int n_heads, int window) {
  const int most = b->max_new < b->n_tokens ? b->max_new : b->n_tokens;
  return attn_shape(c->head_dim / 32, b->n_seqs, c->n_kv_heads, n_heads / c->n_kv_heads, most,
                    b->max_len, window);
}

int64_t attn_bytes(const mmvq_kv_cache* c, const mmvq_kv_batch* b, int n_heads, int splits) {
  if (splits == 1) return 0;
  return static_cast<int64_t>(b->n_tokens) * n_heads * splits * (c->head_dim * 4 + 8);
}

}  // namespace

extern "C" {

int mmvq_add_rms_norm(const float* x, int64_t K, int64_t n, int64_t ldx, const float* residual, int64_t ldr,
                      const float* weight, float eps, float* sum_out, int64_t lds, float* y, int64_t ldy, void* y_q,
                      void* stream) {
  if (n != 0 && (!x || (!y && !y_q))) return MMVQ_ERR_NULL;
  if (K < 1 || K > kMaxRow || n < 0 || n > kMaxElems / K || (y_q && K % 32)) return MMVQ_ERR_SHAPE;
  if (ldx < K || ldx > kMaxElems || (residual && (ldr < K || ldr > kMaxElems)) ||
      (sum_out && (lds < K || lds > kMaxElems)) || (y && (ldy < K || ldy > kMaxElems)))
    return MMVQ_ERR_SHAPE;
  if (!aligned(x, 4) || !aligned(residual, 4) || !aligned(weight, 4) || !aligned(sum_out, 4) || !aligned(y, 4) ||
      !aligned(y_q, 16))
    return MMVQ_ERR_ALIGN;
  if (n == 0) return MMVQ_OK;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const OnStreamDevice on(st);
  return launch_norm(NormArgs{x, residual, weight, sum_out, y, static_cast<uint8_t*>(y_q), ldx, ldr, lds, ldy, n,
                              static_cast<int>(K), static_cast<double>(eps), 1.0 / static_cast<double>(K)},
                     st);
}

int mmvq_dequantize_q8_1(const void* y_q, int64_t K, int64_t n, float* x, int64_t ldx, void* stream) {
  if (n != 0 && (!y_q || !x)) return MMVQ_ERR_NULL;
  if (K < 1 || K > kMaxRow || K % 32 || n < 0 || n > kMaxElems / K || ldx < K || ldx > kMaxElems) return MMVQ_ERR_SHAPE;
  if (!aligned(y_q, 16) || !aligned(x, 4)) return MMVQ_ERR_ALIGN;
  if (n == 0) return MMVQ_OK;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const OnStreamDevice on(st);
  return launch_dequantize_q8_1(static_cast<const uint8_t*>(y_q), K, n, x, ldx, st);
}

int mmvq_kv_page_bytes(int type, int page_size, int n_kv_heads, int head_dim, int64_t* bytes) {
  if (!bytes) return MMVQ_ERR_NULL;
  const int rc = check_pages(type, page_size, n_kv_heads, head_dim);
  if (rc) return rc;
  *bytes = static_cast<int64_t>(n_kv_heads) * (page_size / 16) * kv_unit_bytes(kv_kind(type), head_dim / 32);
  return MMVQ_OK;
}

int mmvq_kv_write(const mmvq_kv_cache* cache, const mmvq_kv_batch* batch, const float* k, int64_t ldk, const float* v,
                  int64_t ldv, void* stream) {
  return kv_io(cache, batch, const_cast<float*>(k), ldk, const_cast<float*>(v), ldv, true, stream);
}

int mmvq_kv_read(const mmvq_kv_cache* cache, const mmvq_kv_batch* batch, float* k, int64_t ldk, float* v, int64_t ldv,
                 void* stream) {
  return kv_io(cache, batch, k, ldk, v, ldv, false, stream);
}

int mmvq_attn_workspace(const mmvq_kv_cache* cache, const mmvq_kv_batch* batch, int n_heads, int64_t* bytes) {
  if (!bytes) return MMVQ_ERR_NULL;
  const int rc = check_attn(cache, batch, n_heads);
  if (rc) return rc;
  // without a window the keys are most, and so are the ranges they are cut into
  *bytes = empty(batch)
               ? 0 : attn_bytes(cache, batch, n_heads, shape_of(cache, batch, n_heads, 0).splits);
  return MMVQ_OK;
}

int mmvq_attn(const mmvq_kv_cache* cache, const mmvq_kv_batch* batch, const float* q, int64_t ldq, int n_heads,
              float scale, int window, const float* sinks, float* out, int64_t ldo, void* workspace,
              int64_t workspace_bytes, void* stream) {
  AttnArgs a{};
  int rc = check_attn(cache, batch, n_heads);
  if (rc) return rc;
  rc = check_kv(cache, batch, &a.b);
  if (rc) return rc;
  if (!empty(batch) && (!q || !out)) return MMVQ_ERR_NULL;
  const int64_t width = static_cast<int64_t>(n_heads) * cache->head_dim;
  if (ldq < width || ldq > kMaxElems || ldo < width || ldo > kMaxElems || window < 0) return MMVQ_ERR_SHAPE;
  if (!aligned(q, 4) || !aligned(out, 4) || !aligned(sinks, 4) || !aligned(workspace, 16)) return MMVQ_ERR_ALIGN;
  if (empty(batch)) return MMVQ_OK;
  const AttnShape s = shape_of(cache, batch, n_heads, window);
  const int64_t need = attn_bytes(cache, batch, n_heads, s.splits);
  if (need > 0 && !workspace) return MMVQ_ERR_NULL;
  if (workspace_bytes < need) return MMVQ_ERR_SHAPE;
  a.k = static_cast<const uint8_t*>(cache->k);
  a.v = static_cast<const uint8_t*>(cache->v);
  a.q = q;
  a.out = out;
  a.sinks = sinks;
  a.ldq = ldq;
  a.ldo = ldo;
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * M_LOG2E);
  a.window = window < (1 << 30) ? window : 0;   // positions are below 2^30: it hides nothing
  a.n_heads = n_heads;
  a.group = FastDiv(static_cast<uint32_t>(n_heads / cache->n_kv_heads));
  a.heads = FastDiv(static_cast<uint32_t>(cache->n_kv_heads));
  a.head_dim = cache->head_dim;
  a.tiles = FastDiv(static_cast<uint32_t>(s.tiles));
  a.splits = FastDiv(static_cast<uint32_t>(s.splits));
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + static_cast<int64_t>(batch->n_tokens) * n_heads * s.splits * cache->head_dim);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const OnStreamDevice on(st);
  const int kind = kv_kind(cache->type), nb = cache->head_dim / 32;
  rc = kind == kKvF16  ? launch_attn_f16(nb, s, a, st)
       : kind == kKvQ8 ? launch_attn_q8_0(nb, s, a, st)
                       : launch_attn_q4_0(nb, s, a, st);
  if (rc || s.splits == 1) return rc;
  return launch_attn_join(a, kind == kKvF16, st);
}

int mmvq_verify_workspace(int n_seqs, int n_rows, int vocab, int64_t* bytes) {
  if (!bytes) return MMVQ_ERR_NULL;
  if (n_seqs < 0 || n_seqs > (1 << 20) || n_rows < 0 || n_rows > (1 << 20) || vocab < 1 || vocab > kMaxRow)
    return MMVQ_ERR_SHAPE;
  *bytes = verify_bytes(n_seqs, n_rows, vocab, nullptr);
  return MMVQ_OK;
}

int mmvq_verify_draft(const float* target, int64_t ldt, int vocab, int kind, const float* temperature,
                      const int32_t* draft_tokens, const float* draft_probs, int64_t ldd, const int32_t* row_start,
                      int n_seqs, int n_rows, const float* u_accept, const float* u_sample, int32_t* n_accepted,
                      int32_t* tokens, int max_out, void* workspace, int64_t workspace_bytes, void* stream) {
  if ((n_seqs != 0 && (!row_start || !u_sample || !n_accepted || !tokens || !workspace)) ||
      (n_seqs != 0 && n_rows != 0 && (!target || !draft_tokens || !u_accept)))
    return MMVQ_ERR_NULL;
  if (kind != MMVQ_TARGET_LOGITS && kind != MMVQ_TARGET_WEIGHTS) return MMVQ_ERR_TYPE;
  int64_t need = 0;
  const int rc = mmvq_verify_workspace(n_seqs, n_rows, vocab, &need);
  if (rc) return rc;
  if (ldt < vocab || ldt > kMaxElems || (draft_probs && (ldd < vocab || ldd > kMaxElems)) || max_out < 1 ||
      workspace_bytes < need)
    return MMVQ_ERR_SHAPE;
  if (!aligned(target, 4) || !aligned(temperature, 4) || !aligned(draft_tokens, 4) || !aligned(draft_probs, 4) ||
      !aligned(row_start, 4) || !aligned(u_accept, 4) || !aligned(u_sample, 4) || !aligned(n_accepted, 4) ||
      !aligned(tokens, 4) || !aligned(workspace, 16))
    return MMVQ_ERR_ALIGN;
  if (n_seqs == 0) return MMVQ_OK;
  VerifyArgs a{};
  a.target = target;
  a.temperature = kind == MMVQ_TARGET_LOGITS ? temperature : nullptr;
  a.draft_probs = draft_probs;
  a.u_accept = u_accept;
  a.u_sample = u_sample;
  a.draft_tokens = draft_tokens;
  a.row_start = row_start;
  a.n_accepted = n_accepted;
  a.tokens = tokens;
  a.ldt = ldt;
  a.ldd = ldd;
  a.vocab = vocab;
  a.kind = kind;
  a.n_seqs = n_seqs;
  a.n_rows = n_rows;
  a.max_out = max_out;
  verify_bytes(n_seqs, n_rows, vocab, &a.chunks);
  a.ws = static_cast<uint8_t*>(workspace);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const OnStreamDevice on(st);
  return launch_verify(a, st);
}

}  // extern "C"
