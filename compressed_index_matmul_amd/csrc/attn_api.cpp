// C ABI of the attention entry points: argument validation (host only, before
// any HIP call), dispatch to the kernel launchers, status mapping.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "vqmm_internal.h"

namespace vqmm {

namespace {

constexpr int64_t kMaxInt = ((int64_t)1 << 31) - 1;

bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

bool valid_head_dim(int d) { return d == 64 || d == 128 || d == 256; }

int map_hip(hipError_t e) { return e == hipSuccess ? VQ_OK : VQ_ERR_HIP; }

// Rows of heads; `rows` == 0 lets the pointer be NULL.
int check_heads(const attn_heads *h, int64_t rows) {
  if (!h) return VQ_ERR_NULL;
  if (rows > 0 && !h->data) return VQ_ERR_NULL;
  if (misaligned(h->data, 16)) return VQ_ERR_ALIGN;
  if (h->token_stride < 8 || h->head_stride < 8 || (h->token_stride & 7) || (h->head_stride & 7)) return VQ_ERR_SHAPE;
  if (h->token_stride >= ((int64_t)1 << 22) || h->head_stride >= ((int64_t)1 << 40)) return VQ_ERR_SHAPE;
  return VQ_OK;
}

int check_batch(const attn_batch *b, AttnView *a, bool pointers = true) {
  if (!b) return VQ_ERR_NULL;
  if (b->dtype != VQ_BF16 && b->dtype != VQ_F16) return VQ_ERR_DTYPE;
  if (b->n_q_heads < 1 || b->n_kv_heads < 1 || b->n_q_heads % b->n_kv_heads != 0) return VQ_ERR_SHAPE;
  if (b->n_q_heads > 65535) return VQ_ERR_SHAPE;
  if (b->n_seqs < 0 || b->total_q < 0 || b->total_k < 0 || b->reserved != 0) return VQ_ERR_SHAPE;
  if (b->causal != 0 && b->causal != 1) return VQ_ERR_VALUE;
  if (!std::isfinite(b->scale) || b->scale <= 0.0f) return VQ_ERR_VALUE;
  if (!valid_head_dim(b->head_dim)) return VQ_ERR_UNSUPPORTED;
  if (pointers) {
    if (!b->cu_q || !b->cu_k) return VQ_ERR_NULL;
    if (misaligned(b->cu_q, 4) || misaligned(b->cu_k, 4)) return VQ_ERR_ALIGN;
  }
  *a = AttnView{};
  a->hq = b->n_q_heads;
  a->hkv = b->n_kv_heads;
  a->d = b->head_dim;
  a->nseq = b->n_seqs;
  a->tq = b->total_q;
  a->tk = b->total_k;
  a->causal = b->causal == 1;
  a->f16 = b->dtype == VQ_F16;
  a->scale = b->scale;
  a->cu_q = b->cu_q;
  a->cu_k = b->cu_k;
  return VQ_OK;
}

// One workgroup a tile of 128 queries (or keys) of each sequence and head.
bool grid_fits(int64_t total, int64_t nseq, int64_t heads) { return (total / 128 + nseq) * heads <= kMaxBlocks; }

int check_cache(const kv4_cache *c, KvView *v, bool pointers) {
  if (!c) return VQ_ERR_NULL;
  if (c->n_pages < 1 || c->n_kv_heads < 1 || c->n_kv_heads > 65535) return VQ_ERR_SHAPE;
  if (c->page_size < 32 || c->page_size > 1024 || c->page_size % 32 != 0) return VQ_ERR_SHAPE;
  if (!valid_head_dim(c->head_dim)) return VQ_ERR_UNSUPPORTED;
  if (pointers) {
    if (!c->codes || !c->scales || !c->weights || !c->pos) return VQ_ERR_NULL;
    if (misaligned(c->codes, 16) || misaligned(c->scales, 16) || misaligned(c->weights, 16) || misaligned(c->pos, 16))
      return VQ_ERR_ALIGN;
  }
  *v = KvView{};
  v->np = c->n_pages;
  v->ps = c->page_size;
  v->hkv = c->n_kv_heads;
  v->d = c->head_dim;
  v->codes = c->codes;
  v->scales = c->scales;
  v->weights = c->weights;
  v->pos = c->pos;
  return VQ_OK;
}

int check_seqs(const kv4_seqs *s, KvView *v, bool need_lens) {
  if (!s) return VQ_ERR_NULL;
  if (s->n_seqs < 0 || s->max_pages < 1 || (int64_t)s->max_pages * v->ps > kMaxInt) return VQ_ERR_SHAPE;
  if (s->n_seqs > 0 && (!s->block_table || (need_lens && !s->lens))) return VQ_ERR_NULL;
  if (misaligned(s->block_table, 4) || misaligned(s->lens, 4)) return VQ_ERR_ALIGN;
  v->nseq = s->n_seqs;
  v->mp = s->max_pages;
  v->table = s->block_table;
  v->lens = s->lens;
  return VQ_OK;
}

int check_rows(const KvView &v, int32_t total, const int32_t *cu) {
  if (total < 0) return VQ_ERR_SHAPE;
  if (!cu) return VQ_ERR_NULL;
  if (misaligned(cu, 4)) return VQ_ERR_ALIGN;
  // four slots and eight channels a thread, 256 threads a workgroup
  const int64_t per = ((int64_t)2 * v.hkv * (v.d / 8) + 255) / 256;
  if (((int64_t)total / 4 + 2 * (int64_t)v.nseq) * per > kMaxBlocks) return VQ_ERR_SHAPE;
  return VQ_OK;
}

// The sizes kv4_attend accepts (everything but pointers).
int check_attend_sizes(const KvView &v, int n_q_heads, int max_len, bool weigh) {
  if (n_q_heads < 1 || n_q_heads > 65535 || n_q_heads % v.hkv != 0 || max_len < 0) return VQ_ERR_SHAPE;
  const int64_t group = n_q_heads / v.hkv;
  const int64_t rows = v.hkv * ((group + 15) / 16);  // of a sequence
  // of the join's part for the weights, whose lengths are bounded by the pool too
  const int64_t chunks = weigh ? (std::min<int64_t>(max_len, (int64_t)v.np * v.ps) + 1023) / 1024 : 0;
  if (chunks * v.nseq * v.hkv + (int64_t)v.nseq * n_q_heads > kMaxBlocks) return VQ_ERR_SHAPE;
  if (v.nseq * rows > ((int64_t)1 << 22) || ((int64_t)max_len / 32 + 1) * rows > kMaxInt) return VQ_ERR_SHAPE;
  return VQ_OK;
}

int check_evict_sizes(const KvView &v, int keep, int recent, int max_len) {
  if (keep < 1 || max_len < 0) return VQ_ERR_SHAPE;
  if ((int64_t)v.nseq * v.hkv >= ((int64_t)1 << 22)) return VQ_ERR_SHAPE;  // workgroups of up to 1024 threads
  if (recent < 0 || recent > keep) return VQ_ERR_VALUE;
  return VQ_OK;
}

}  // namespace

}  // namespace vqmm

using namespace vqmm;

extern "C" {

int attn_prompt(const attn_batch *b, const attn_heads *q, const attn_heads *k, const attn_heads *v, void *out,
                float *lse, void *workspace, size_t ws_bytes, void *stream) {
  AttnView a;
  int st = check_batch(b, &a);
  if (st != VQ_OK) return st;
  if ((st = check_heads(q, a.tq)) != VQ_OK || (st = check_heads(k, a.tk)) != VQ_OK || (st = check_heads(v, a.tk)) != VQ_OK)
    return st;
  if ((a.tq > 0 && !out) || (ws_bytes > 0 && !workspace)) return VQ_ERR_NULL;
  if (misaligned(out, 16) || misaligned(lse, 4) || misaligned(workspace, 16)) return VQ_ERR_ALIGN;
  if (!grid_fits(a.tq, a.nseq, a.hq)) return VQ_ERR_SHAPE;
  const PromptPlan p = attn_prompt_plan(a);
  if (ws_bytes < p.bytes) return VQ_ERR_WORKSPACE;
  a.q = static_cast<const uint16_t *>(q->data);
  a.k = static_cast<const uint16_t *>(k->data);
  a.v = static_cast<const uint16_t *>(v->data);
  a.q_ts = q->token_stride, a.q_hs = q->head_stride;
  a.k_ts = k->token_stride, a.k_hs = k->head_stride;
  a.v_ts = v->token_stride, a.v_hs = v->head_stride;
  if (a.tq == 0 || a.nseq == 0) return VQ_OK;
  return map_hip(launch_attn_prompt(a, p, static_cast<uint16_t *>(out), lse, workspace, reinterpret_cast<hipStream_t>(stream)));
}

size_t attn_prompt_workspace_size(const attn_batch *b) {
  AttnView a;
  if (check_batch(b, &a, false) != VQ_OK || !grid_fits(a.tq, a.nseq, a.hq)) return 0;
  return attn_prompt_plan(a).bytes;
}

int attn_prompt_weights(const attn_batch *b, const attn_heads *q, const attn_heads *k, const float *lse, int32_t last,
                        int32_t accumulate, float *weights, void *workspace, size_t ws_bytes, void *stream) {
  AttnView a;
  int st = check_batch(b, &a);
  if (st != VQ_OK) return st;
  if ((st = check_heads(q, a.tq)) != VQ_OK || (st = check_heads(k, a.tk)) != VQ_OK) return st;
  if ((a.tq > 0 && !lse) || (a.tk > 0 && !weights) || (ws_bytes > 0 && !workspace)) return VQ_ERR_NULL;
  if (misaligned(lse, 4) || misaligned(weights, 4) || misaligned(workspace, 16)) return VQ_ERR_ALIGN;
  if (last < 0) return VQ_ERR_SHAPE;
  if (accumulate != 0 && accumulate != 1) return VQ_ERR_VALUE;
  if (!grid_fits(a.tk, a.nseq, a.hkv)) return VQ_ERR_SHAPE;
  const PromptPlan p = attn_weights_plan(a, last);
  if (ws_bytes < p.bytes) return VQ_ERR_WORKSPACE;
  a.q = static_cast<const uint16_t *>(q->data);
  a.k = static_cast<const uint16_t *>(k->data);
  a.q_ts = q->token_stride, a.q_hs = q->head_stride;
  a.k_ts = k->token_stride, a.k_hs = k->head_stride;
  if (a.tk == 0 || a.nseq == 0) return VQ_OK;
  return map_hip(launch_attn_weights(a, p, lse, last, accumulate == 1, weights, workspace, reinterpret_cast<hipStream_t>(stream)));
}

size_t attn_prompt_weights_workspace_size(const attn_batch *b, int32_t last) {
  AttnView a;
  if (check_batch(b, &a, false) != VQ_OK || last < 0 || !grid_fits(a.tk, a.nseq, a.hkv)) return 0;
  return attn_weights_plan(a, last).bytes;
}

int kv4_append(const kv4_cache *c, const kv4_seqs *s, const attn_heads *k, const attn_heads *v, int32_t dtype,
               int32_t total, const int32_t *cu, const int32_t *pos, const float *weights, void *stream) {
  KvView w;
  int st = check_cache(c, &w, true);
  if (st != VQ_OK || (st = check_seqs(s, &w, false)) != VQ_OK) return st;
  if (dtype != VQ_F32 && dtype != VQ_BF16 && dtype != VQ_F16) return VQ_ERR_DTYPE;
  if ((st = check_rows(w, total, cu)) != VQ_OK) return st;
  if ((st = check_heads(k, total)) != VQ_OK || (st = check_heads(v, total)) != VQ_OK) return st;
  if (misaligned(pos, 4) || misaligned(weights, 4)) return VQ_ERR_ALIGN;
  if (total == 0 || w.nseq == 0) return VQ_OK;
  return map_hip(launch_kv4_append(w, k->data, v->data, k->token_stride, k->head_stride, v->token_stride, v->head_stride,
                                   dtype, total, cu, pos, weights, reinterpret_cast<hipStream_t>(stream)));
}

int kv4_read(const kv4_cache *c, const kv4_seqs *s, const int32_t *cu, int32_t total, int32_t dtype, void *k_out,
             void *v_out, void *stream) {
  KvView w;
  int st = check_cache(c, &w, true);
  if (st != VQ_OK || (st = check_seqs(s, &w, false)) != VQ_OK) return st;
  if (dtype != VQ_F32 && dtype != VQ_BF16 && dtype != VQ_F16) return VQ_ERR_DTYPE;
  if ((st = check_rows(w, total, cu)) != VQ_OK) return st;
  if (total > 0 && (!k_out || !v_out)) return VQ_ERR_NULL;
  if (misaligned(k_out, 16) || misaligned(v_out, 16)) return VQ_ERR_ALIGN;
  if (total == 0 || w.nseq == 0) return VQ_OK;
  return map_hip(launch_kv4_read(w, cu, total, dtype, k_out, v_out, reinterpret_cast<hipStream_t>(stream)));
}

size_t kv4_attend_workspace_size(const kv4_cache *c, int32_t n_seqs, int32_t n_q_heads, int32_t max_len,
                                 int32_t add_weights) {
  KvView w;
  if (check_cache(c, &w, false) != VQ_OK || n_seqs < 1) return 0;
  w.nseq = n_seqs;
  w.mp = (int)(kMaxInt / w.ps);
  if (check_attend_sizes(w, n_q_heads, max_len, add_weights != 0) != VQ_OK) return 0;
  return kv4_attend_plan(w, n_q_heads, max_len, add_weights != 0).bytes;
}

int kv4_attend(const kv4_cache *c, const kv4_seqs *s, const attn_heads *q, int32_t dtype, int32_t n_q_heads,
               float scale, int32_t max_len, int32_t add_weights, void *out, float *lse, void *workspace,
               size_t ws_bytes, void *stream) {
  KvView w;
  int st = check_cache(c, &w, true);
  if (st != VQ_OK || (st = check_seqs(s, &w, true)) != VQ_OK) return st;
  if (dtype != VQ_BF16 && dtype != VQ_F16) return VQ_ERR_DTYPE;
  if ((st = check_attend_sizes(w, n_q_heads, max_len, add_weights != 0)) != VQ_OK) return st;
  if ((st = check_heads(q, w.nseq)) != VQ_OK) return st;
  if (!std::isfinite(scale) || scale <= 0.0f || (add_weights != 0 && add_weights != 1)) return VQ_ERR_VALUE;
  if (w.nseq == 0) return VQ_OK;
  if (!out || (ws_bytes > 0 && !workspace)) return VQ_ERR_NULL;
  if (misaligned(out, 16) || misaligned(lse, 4) || misaligned(workspace, 16)) return VQ_ERR_ALIGN;
  // the sizing call knows no block table: the same plan, from max_len alone
  KvView sized = w;
  sized.mp = (int)(kMaxInt / w.ps);
  AttendPlan p = kv4_attend_plan(sized, n_q_heads, max_len, add_weights == 1);
  if (ws_bytes < p.bytes) return VQ_ERR_WORKSPACE;
  p.len_cap = (int)std::min<int64_t>(p.len_cap, (int64_t)w.mp * w.ps);
  return map_hip(launch_kv4_attend(w, p, q->data, q->token_stride, q->head_stride, dtype == VQ_F16, n_q_heads, scale,
                                   add_weights == 1, out, lse, workspace, reinterpret_cast<hipStream_t>(stream)));
}

size_t kv4_evict_workspace_size(const kv4_cache *c, int32_t n_seqs, int32_t keep, int32_t max_len) {
  KvView w;
  if (check_cache(c, &w, false) != VQ_OK || n_seqs < 1) return 0;
  w.nseq = n_seqs;
  w.mp = (int)(kMaxInt / w.ps);
  if (check_evict_sizes(w, keep, 0, max_len) != VQ_OK) return 0;
  return kv4_evict_plan(w, keep, max_len).bytes;
}

int kv4_evict(const kv4_cache *c, const kv4_seqs *s, const int32_t *next_pos, int32_t keep, int32_t recent,
              int32_t max_len, void *workspace, size_t ws_bytes, void *stream) {
  KvView w;
  int st = check_cache(c, &w, true);
  if (st != VQ_OK || (st = check_seqs(s, &w, true)) != VQ_OK) return st;
  if ((st = check_evict_sizes(w, keep, recent, max_len)) != VQ_OK) return st;
  if (w.nseq == 0) return VQ_OK;
  if (!next_pos || (ws_bytes > 0 && !workspace)) return VQ_ERR_NULL;
  if (misaligned(next_pos, 4) || misaligned(workspace, 16)) return VQ_ERR_ALIGN;
  KvView sized = w;
  sized.mp = (int)(kMaxInt / w.ps);
  EvictPlan p = kv4_evict_plan(sized, keep, max_len);
  if (ws_bytes < p.bytes) return VQ_ERR_WORKSPACE;
  p.len_cap = (int)std::min<int64_t>(p.len_cap, (int64_t)w.mp * w.ps);
  if (p.max_moves == 0) return VQ_OK;  // no sequence can be longer than keep
  return map_hip(launch_kv4_evict(w, p, next_pos, keep, recent, workspace, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
