// kv_api.cu -- the extern "C" entry points of the INT8 paged KV cache
// (declared and documented in include/w8a8.h): host-side argument checks and
// the dispatch to the kernels. No entry point allocates device memory.
#include <cmath>

#include "kernels.h"

namespace w8a8 {

namespace {

constexpr int64_t kMaxLen = int64_t(1) << 30;     // positions and packed rows stay far inside int32
constexpr int32_t kMaxGroup = 128;                // query heads of a kv head
constexpr int64_t kMaxBatch = 65535;
constexpr float kMaxSoftcap = 4096.0f;

bool aligned(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

w8a8_status from_cuda(cudaError_t e) { return e == cudaSuccess ? W8A8_OK : W8A8_ERR_CUDA; }

w8a8_status check_cache(const w8a8_kv_cache *c, KvCache *out) {
  if (!c) return W8A8_ERR_INVALID_ARG;
  if (c->num_pages < 0 || c->num_pages > INT32_MAX || c->kv_heads <= 0 || c->kv_heads > 65535)
    return W8A8_ERR_INVALID_ARG;
  int shift;
  switch (c->page_size) {
    case 16: shift = 4; break;
    case 32: shift = 5; break;
    case 64: shift = 6; break;
    case 128: shift = 7; break;
    default: return W8A8_ERR_UNSUPPORTED_SHAPE;
  }
  if (c->head_dim != 64 && c->head_dim != 96 && c->head_dim != 128) return W8A8_ERR_UNSUPPORTED_SHAPE;
  if (c->num_pages > 0 && (!c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale)) return W8A8_ERR_INVALID_ARG;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return W8A8_ERR_MISALIGNED;
  out->k = c->k_codes;
  out->v = c->v_codes;
  out->ks = c->k_scale;
  out->vs = c->v_scale;
  out->pages = c->num_pages;
  out->heads = c->kv_heads;
  out->page = c->page_size;
  out->page_shift = shift;
  out->d = c->head_dim;
  return W8A8_OK;
}

w8a8_status check_table(const int32_t *table, int64_t ld, int64_t batch, int64_t max_pages, int32_t page) {
  if (batch < 0 || batch > kMaxBatch || max_pages < 0 || ld < max_pages || (batch > 0 && max_pages > 0 && !table))
    return W8A8_ERR_INVALID_ARG;
  if (!aligned(table, 4)) return W8A8_ERR_MISALIGNED;
  if (max_pages > kMaxLen / page) return W8A8_ERR_UNSUPPORTED_SHAPE;
  return W8A8_OK;
}

w8a8_status check_batch(const w8a8_kv_batch *b, int64_t tokens, const KvCache &c, KvSeqs *out) {
  if (!b || tokens < 0) return W8A8_ERR_INVALID_ARG;
  if (tokens > kMaxLen) return W8A8_ERR_UNSUPPORTED_SHAPE;
  if (w8a8_status s = check_table(b->page_table, b->page_table_ld, b->batch, b->max_pages, c.page)) return s;
  if (b->max_q_len < 0 || b->max_kv_len < 0 || b->max_kv_len > static_cast<int64_t>(b->max_pages) * c.page)
    return W8A8_ERR_INVALID_ARG;
  if (b->batch > 0 && (!b->seq_start || !b->kv_len)) return W8A8_ERR_INVALID_ARG;
  if (!aligned(b->seq_start, 4) || !aligned(b->kv_len, 4)) return W8A8_ERR_MISALIGNED;
  out->table = b->page_table;
  out->table_ld = b->page_table_ld;
  out->seq_start = b->seq_start;
  out->kv_len = b->kv_len;
  out->batch = b->batch;
  out->max_pages = b->max_pages;
  out->max_q = static_cast<int32_t>(b->max_q_len < tokens ? b->max_q_len : tokens);
  out->max_kv = b->max_kv_len;
  out->tokens = tokens;
  return W8A8_OK;
}

w8a8_status check_rows(const void *p, int64_t token_stride, int64_t head_stride, KvRows *out) {
  if (!p || token_stride < 0 || head_stride < 0) return W8A8_ERR_INVALID_ARG;
  if (!aligned(p, 16) || token_stride % 8 != 0 || head_stride % 8 != 0) return W8A8_ERR_MISALIGNED;
  out->p = static_cast<const uint16_t *>(p);
  out->token_stride = token_stride;
  out->head_stride = head_stride;
  return W8A8_OK;
}

// Which kernel a call takes, by the query rows of a kv head (new tokens x
// group): the one for few rows reads the codes of a context once for each 16 of
// them; the other expands the context to bf16 once and costs nearly the same
// for any number up to 256. Few : other, us a call, head dim 128, contexts of
// 200, 1024, 4096, 16384:
//   16 sequences x 8 kv heads, 32 rows 25 36 72 217 : 23 44 131 495
//                              48 rows 29 44 99 320 : 24 44 132 494
//                              64 rows 35 55 129 429 : 24 45 132 496
//   8 sequences x 8 kv heads,  64 rows 24 34 69 216 : 22 32 88 289
//   1 sequence x 32 kv heads,  64 rows 10 16 41 114 : 21 30 48 162
//   1 sequence x 8 kv heads,   64 rows 9 16 22 40 : 17 28 26 46
// so up to kFewRows always, and up to twice as many where (sequence, kv head)
// pairs are few or contexts long.
constexpr int64_t kFewRows = 32, kFewPairs = 64, kFewLong = 4096;

bool few_rows(const KvAttnArgs &a) {
  const int64_t rows = static_cast<int64_t>(a.s.max_q) * a.group;
  if (rows <= kFewRows) return true;
  return rows <= 2 * kFewRows && (static_cast<int64_t>(a.s.batch) * a.c.heads <= kFewPairs || a.s.max_kv >= kFewLong);
}

// Cache, batch and heads of an attention call (what its workspace depends on).
w8a8_status check_attention_shape(const w8a8_kv_cache *cache, const w8a8_kv_batch *batch, int64_t tokens,
                                  int32_t q_heads, KvAttnArgs *a) {
  if (w8a8_status s = check_cache(cache, &a->c)) return s;
  if (w8a8_status s = check_batch(batch, tokens, a->c, &a->s)) return s;
  if (q_heads <= 0) return W8A8_ERR_INVALID_ARG;
  if (q_heads % a->c.heads != 0 || q_heads / a->c.heads > kMaxGroup) return W8A8_ERR_UNSUPPORTED_SHAPE;
  a->q_heads = q_heads;
  a->group = q_heads / a->c.heads;
  if (few_rows(*a) ? !kv_decode_fits(*a) : !kv_prefill_fits(*a)) return W8A8_ERR_UNSUPPORTED_SHAPE;
  return W8A8_OK;
}

size_t workspace_bytes_of(const KvAttnArgs &a, int sms) {
  return few_rows(a) ? kv_decode_workspace_bytes(a, sms) : kv_prefill_workspace_bytes(a, sms);
}

w8a8_status run_attention(const w8a8_kv_cache *cache, const w8a8_kv_batch *batch, int64_t tokens, const void *q,
                          int64_t q_token_stride, int64_t q_head_stride, int32_t q_heads, const w8a8_kv_scores *scores,
                          void *out, const float *r_out, const int32_t *z_out, void *workspace, size_t workspace_bytes,
                          void *stream) {
  KvAttnArgs a;
  if (w8a8_status s = check_attention_shape(cache, batch, tokens, q_heads, &a)) return s;
  // (the capped form c - 2 c / (1 + 2^x) of c tanh in fp32 is off by c 2^-22 or so: kMaxSoftcap keeps that below 2^-10)
  if (!scores || !std::isfinite(scores->scale) || !(scores->softcap >= 0.0f && scores->softcap <= kMaxSoftcap) ||
      scores->window < 0 || (scores->softcap > 0.0f && !std::isfinite(scores->scale / scores->softcap)))
    return W8A8_ERR_INVALID_ARG;
  if (!aligned(scores->slopes, 4) || !aligned(scores->prefix_len, 4)) return W8A8_ERR_MISALIGNED;
  if (tokens == 0 || a.s.batch == 0 || a.s.max_q == 0) return W8A8_OK;
  if (w8a8_status s = check_rows(q, q_token_stride, q_head_stride, &a.q)) return s;
  if ((tokens > 1 && q_token_stride == 0) || (q_heads > 1 && q_head_stride == 0)) return W8A8_ERR_INVALID_ARG;
  if (!out) return W8A8_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(workspace, 16)) return W8A8_ERR_MISALIGNED;
  a.scale = scores->scale;
  a.softcap = scores->softcap;
  a.slopes = scores->slopes;
  a.window = scores->window < a.s.max_kv ? scores->window : 0;  // a window of all positions is none
  a.prefix = scores->prefix_len;
  a.out = out;
  a.r_out = r_out;
  a.z_out = z_out;
  int sms = 0;
  if (w8a8_status s = current_device_info(&sms, &a.status)) return s;
  const size_t need = workspace_bytes_of(a, sms);
  if (need > 0 && (!workspace || workspace_bytes < need)) return W8A8_ERR_WORKSPACE;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return from_cuda(few_rows(a) ? launch_kv_decode(a, workspace, sms, st) : launch_kv_prefill(a, workspace, sms, st));
}

}  // namespace

}  // namespace w8a8

using namespace w8a8;

extern "C" {

w8a8_status w8a8_kv_append(const w8a8_kv_cache *cache, const w8a8_kv_batch *batch, int64_t tokens, const void *k,
                           int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
                           int64_t v_head_stride, const float *cos, const float *sin, int64_t rope_len,
                           int32_t rot_dim, int32_t interleaved, const void *q, int64_t q_token_stride,
                           int64_t q_head_stride, int32_t q_heads, void *q_out, void *stream) {
  KvAppendArgs a;
  if (w8a8_status s = check_cache(cache, &a.c)) return s;
  if (w8a8_status s = check_batch(batch, tokens, a.c, &a.s)) return s;
  if ((cos == nullptr) != (sin == nullptr) || (q == nullptr) != (q_out == nullptr)) return W8A8_ERR_INVALID_ARG;
  if (cos) {
    if (rope_len < 0) return W8A8_ERR_INVALID_ARG;
    if (rot_dim < 16 || rot_dim > a.c.d || rot_dim % 16 != 0) return W8A8_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(cos, 16) || !aligned(sin, 16)) return W8A8_ERR_MISALIGNED;
  }
  if (q && (q_heads <= 0 || q_heads > 65535)) return W8A8_ERR_INVALID_ARG;
  if (tokens == 0 || a.s.batch == 0 || a.s.max_q == 0) return W8A8_OK;
  if (w8a8_status s = check_rows(k, k_token_stride, k_head_stride, &a.k)) return s;
  if (w8a8_status s = check_rows(v, v_token_stride, v_head_stride, &a.v)) return s;
  if (q) {
    if (w8a8_status s = check_rows(q, q_token_stride, q_head_stride, &a.q)) return s;
    if (!aligned(q_out, 16)) return W8A8_ERR_MISALIGNED;
    a.q_heads = q_heads;
    a.q_out = static_cast<uint16_t *>(q_out);
  }
  a.cos = cos;
  a.sin = sin;
  a.rot = cos ? rot_dim : 0;
  a.interleaved = interleaved != 0;
  if (!kv_append_fits(a)) return W8A8_ERR_UNSUPPORTED_SHAPE;
  a.len_limit = cos && rope_len < a.s.max_kv ? static_cast<int32_t>(rope_len) : a.s.max_kv;
  int sms = 0;
  if (w8a8_status s = current_device_info(&sms, &a.status)) return s;
  return from_cuda(launch_kv_append(a, static_cast<cudaStream_t>(stream)));
}

w8a8_status w8a8_kv_gather(const w8a8_kv_cache *cache, const int32_t *page_table, int64_t page_table_ld, int32_t batch,
                           int32_t max_pages, const int32_t *first_pos, const int32_t *row_start, int64_t rows,
                           void *k_out, void *v_out, w8a8_dtype out_dtype, void *stream) {
  KvGatherArgs a;
  if (w8a8_status s = check_cache(cache, &a.c)) return s;
  if (w8a8_status s = check_table(page_table, page_table_ld, batch, max_pages, a.c.page)) return s;
  if (out_dtype != W8A8_BF16 && out_dtype != W8A8_FP32) return W8A8_ERR_UNSUPPORTED_DTYPE;
  if (rows < 0) return W8A8_ERR_INVALID_ARG;
  if (rows > kMaxLen) return W8A8_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0 || batch == 0) return W8A8_OK;
  if (!first_pos || !row_start || (!k_out && !v_out)) return W8A8_ERR_INVALID_ARG;
  if (!aligned(first_pos, 4) || !aligned(row_start, 4) || !aligned(k_out, 16) || !aligned(v_out, 16))
    return W8A8_ERR_MISALIGNED;
  a.table = page_table;
  a.table_ld = page_table_ld;
  a.batch = batch;
  a.max_pages = max_pages;
  a.first_pos = first_pos;
  a.row_start = row_start;
  a.rows = rows;
  a.k_out = k_out;
  a.v_out = v_out;
  if (!kv_gather_fits(a)) return W8A8_ERR_UNSUPPORTED_SHAPE;
  int sms = 0;
  if (w8a8_status s = current_device_info(&sms, &a.status)) return s;
  return from_cuda(launch_kv_gather(a, out_dtype == W8A8_BF16, static_cast<cudaStream_t>(stream)));
}

w8a8_status w8a8_kv_attention(const w8a8_kv_cache *cache, const w8a8_kv_batch *batch, int64_t tokens, const void *q,
                              int64_t q_token_stride, int64_t q_head_stride, int32_t q_heads,
                              const w8a8_kv_scores *scores, void *out, void *workspace, size_t workspace_bytes,
                              void *stream) {
  return run_attention(cache, batch, tokens, q, q_token_stride, q_head_stride, q_heads, scores, out, nullptr, nullptr,
                       workspace, workspace_bytes, stream);
}

w8a8_status w8a8_kv_attention_requant(const w8a8_kv_cache *cache, const w8a8_kv_batch *batch, int64_t tokens,
                                      const void *q, int64_t q_token_stride, int64_t q_head_stride, int32_t q_heads,
                                      const w8a8_kv_scores *scores, const float *r_out, const int32_t *Z_out,
                                      int8_t *codes_out, void *workspace, size_t workspace_bytes, void *stream) {
  if (!r_out || !Z_out) return W8A8_ERR_INVALID_ARG;
  if (!aligned(r_out, 4) || !aligned(Z_out, 4)) return W8A8_ERR_MISALIGNED;
  return run_attention(cache, batch, tokens, q, q_token_stride, q_head_stride, q_heads, scores, codes_out, r_out,
                       Z_out, workspace, workspace_bytes, stream);
}

size_t w8a8_kv_attention_workspace_size(const w8a8_kv_cache *cache, const w8a8_kv_batch *batch, int64_t tokens,
                                        int32_t q_heads) {
  KvAttnArgs a;
  if (check_attention_shape(cache, batch, tokens, q_heads, &a) != W8A8_OK) return 0;
  if (tokens == 0 || a.s.batch == 0 || a.s.max_q == 0) return 0;
  int sms = 0;
  if (current_device_info(&sms, &a.status) != W8A8_OK) return 0;
  return workspace_bytes_of(a, sms);
}

}  // extern "C"
