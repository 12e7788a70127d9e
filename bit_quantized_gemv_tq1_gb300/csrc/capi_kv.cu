// capi_kv.cu -- the extern "C" entry points of the paged key/value cache's
// operators (declared in include/tq1.h): host-side argument checks and
// launches.
#include <cmath>

#include "../../include/tq1.h"
#include "kv_internal.h"
#include "tq1_internal.h"

using namespace tq1;

namespace {

constexpr int64_t kMaxSeqCount = 8192;
constexpr int64_t kMaxTableWidth = int64_t{1} << 20;  // pages of one sequence
constexpr int64_t kMaxPoolPages = int64_t{1} << 22;

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }
bool pow2(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }
cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

// Checks and translates the cache and the batch of a call over t tokens.
int get_cache(const tq1_kv_cache* c, KvCache* out) {
  if (!c) return TQ1_ERR_NULL;
  if (c->n_pages < 0 || c->n_kv <= 0 || c->page_size <= 0 || c->head_dim <= 0 || c->head_dim % 8 != 0 ||
      c->page_stride < 0 || c->head_stride < 0 || c->slot_stride < c->head_dim)
    return TQ1_ERR_SHAPE;
  if (!c->k || !c->v) return TQ1_ERR_NULL;
  if (off16(c->k) || off16(c->v) || c->page_stride % 8 != 0 || c->head_stride % 8 != 0 || c->slot_stride % 8 != 0)
    return TQ1_ERR_ALIGN;
  if (c->dtype != TQ1_F16 && c->dtype != TQ1_BF16) return TQ1_ERR_UNSUPPORTED;
  if (!pow2(c->page_size) || c->page_size < 16 || c->page_size > 256 || c->head_dim > 256 || c->n_kv > 4096 ||
      c->n_pages > kMaxPoolPages * 8)
    return TQ1_ERR_UNSUPPORTED;
  out->k = static_cast<uint16_t*>(c->k);
  out->v = static_cast<uint16_t*>(c->v);
  out->page_stride = c->page_stride;
  out->head_stride = c->head_stride;
  out->slot_stride = c->slot_stride;
  out->n_pages = static_cast<int>(c->n_pages);
  out->n_kv = static_cast<int>(c->n_kv);
  out->page_size = static_cast<int>(c->page_size);
  out->page_shift = 0;
  while ((1 << out->page_shift) < out->page_size) ++out->page_shift;
  out->d = static_cast<int>(c->head_dim);
  out->dtype = c->dtype;
  return TQ1_OK;
}

int get_batch(const tq1_kv_batch* b, int64_t page_size, int64_t t, KvBatch* out) {
  if (!b) return TQ1_ERR_NULL;
  if (b->n_seqs <= 0 || b->max_pages <= 0 || t < 0) return TQ1_ERR_SHAPE;
  if (!b->page_table || !b->q_start || !b->kv_len) return TQ1_ERR_NULL;
  if (off4(b->page_table) || off4(b->q_start) || off4(b->kv_len)) return TQ1_ERR_ALIGN;
  if (b->n_seqs > kMaxSeqCount || b->max_pages > kMaxTableWidth || t > (int64_t{1} << 24)) return TQ1_ERR_UNSUPPORTED;
  out->table = b->page_table;
  out->q_start = b->q_start;
  out->kv_len = b->kv_len;
  out->n_seqs = static_cast<int>(b->n_seqs);
  out->max_pages = static_cast<int>(b->max_pages);
  out->t = static_cast<int>(t);
  out->max_len = static_cast<int>(b->max_pages * page_size);
  return TQ1_OK;
}

int get_pool(const tq1_page_pool* p, PagePool* out) {
  if (!p) return TQ1_ERR_NULL;
  if (p->n_pools < 0 || p->n_pages <= 0 || p->page_bytes <= 0 || p->page_size <= 0 || p->n_seqs <= 0 ||
      p->max_pages <= 0 || p->pool_stride < 0)
    return TQ1_ERR_SHAPE;
  if (p->n_pools > (1 << 16) || p->n_pages > kMaxPoolPages || p->n_seqs > (1 << 20) || p->max_pages > kMaxTableWidth ||
      p->page_size > 256 || p->page_bytes > (int64_t{1} << 30))
    return TQ1_ERR_UNSUPPORTED;
  if (p->pool_stride < p->n_pages * p->page_bytes) return TQ1_ERR_SHAPE;
  if (!p->base || !p->refs || !p->page_table || !p->kv_len) return TQ1_ERR_NULL;
  if (off16(p->base) || off16(p->refs) || off4(p->page_table) || off4(p->kv_len) || p->page_bytes % 16 != 0 ||
      p->pool_stride % 16 != 0)
    return TQ1_ERR_ALIGN;
  out->base = static_cast<uint8_t*>(p->base);
  out->pool_stride = p->pool_stride;
  out->page_bytes = p->page_bytes;
  out->table = p->page_table;
  out->kv_len = p->kv_len;
  out->refs = p->refs;
  out->n_pools = static_cast<int>(p->n_pools);
  out->n_pages = static_cast<int>(p->n_pages);
  out->n_seqs = static_cast<int>(p->n_seqs);
  out->max_pages = static_cast<int>(p->max_pages);
  out->page_size = Divisor(static_cast<int>(p->page_size));
  return TQ1_OK;
}

int check_pages_call(const PagePool& p, int64_t n, const int32_t* a, const int32_t* b, const void* ws, size_t ws_bytes) {
  if (n < 0) return TQ1_ERR_SHAPE;
  if (n == 0) return TQ1_OK;
  if (!a || !b || !ws) return TQ1_ERR_NULL;
  if (off4(a) || off4(b) || off16(ws)) return TQ1_ERR_ALIGN;
  if (n > p.n_seqs) return TQ1_ERR_SHAPE;  // the sequences are distinct
  if (ws_bytes < pages_workspace_bytes(p.n_pages, p.n_seqs)) return TQ1_ERR_WORKSPACE;
  return TQ1_OK;
}

}  // namespace

extern "C" {

int tq1_rope_freqs(float* inv_freq, int64_t rot_dim, double base, double factor, double orig_len, double low,
                   double high, void* stream) {
  if (rot_dim <= 0 || rot_dim % 2 != 0 || !(base > 0) || !(factor > 0) || !std::isfinite(base) ||
      !std::isfinite(factor) || std::isnan(orig_len) || std::isnan(low) || std::isnan(high))
    return TQ1_ERR_SHAPE;
  if (!inv_freq) return TQ1_ERR_NULL;
  if (off4(inv_freq)) return TQ1_ERR_ALIGN;
  if (rot_dim > 256) return TQ1_ERR_UNSUPPORTED;
  if (!status_word()) return TQ1_ERR_CUDA;
  return launch_rope_freqs(inv_freq, static_cast<int>(rot_dim), base, factor, orig_len, low, high, as_stream(stream));
}

int tq1_rope_append(const tq1_kv_cache* cache, const tq1_kv_batch* batch, const void* q, int64_t ldq, const void* k,
                    int64_t ldk, const void* v, int64_t ldv, int in_dtype, void* q_out, int64_t t, int64_t n_q,
                    const float* inv_freq, int64_t rot_dim, int interleaved, float mscale, const int32_t* positions,
                    void* stream) {
  KvCache c;
  KvBatch b;
  int rc = get_cache(cache, &c);
  if (rc != TQ1_OK) return rc;
  rc = get_batch(batch, c.page_size, t, &b);
  if (rc != TQ1_OK) return rc;
  if (n_q > 65536) return TQ1_ERR_UNSUPPORTED;
  if (n_q <= 0 || rot_dim < 0 || rot_dim % 8 != 0 || rot_dim > c.d || ldq < n_q * c.d ||
      ldk < static_cast<int64_t>(c.n_kv) * c.d || ldv < static_cast<int64_t>(c.n_kv) * c.d)
    return TQ1_ERR_SHAPE;
  if (in_dtype != TQ1_F32 && in_dtype != TQ1_F16 && in_dtype != TQ1_BF16) return TQ1_ERR_UNSUPPORTED;
  if (t == 0) return TQ1_OK;
  if (!q || !k || !v || !q_out || (!inv_freq && rot_dim > 0)) return TQ1_ERR_NULL;
  if (off16(q) || off16(k) || off16(v) || off16(q_out) || off4(inv_freq) || off4(positions) || ldq % 4 != 0 ||
      ldk % 4 != 0 || ldv % 4 != 0)
    return TQ1_ERR_ALIGN;
  unsigned* st = status_word();
  if (!st) return TQ1_ERR_CUDA;
  const RopeArgs a = {q,        k,         v,
                      ldq,      ldk,       ldv,
                      static_cast<uint16_t*>(q_out),
                      inv_freq, positions, static_cast<int>(n_q),
                      static_cast<int>(rot_dim), interleaved != 0, in_dtype, mscale};
  return launch_rope_append(c, b, a, st, as_stream(stream));
}

size_t tq1_paged_attn_workspace_size(const tq1_kv_cache* cache, int64_t t, int64_t n_q, int64_t n_seqs) {
  KvCache c;
  if (get_cache(cache, &c) != TQ1_OK || t < 0 || n_q <= 0 || n_q > 65536 || n_seqs <= 0 || t > (int64_t{1} << 24)) return 0;
  if (!status_word()) return 0;
  // One sequence has the widest tiles: what its call needs grows with t and
  // serves t tokens of any number of sequences.
  return attn_workspace_bytes(c, t, n_q, 1);
}

int tq1_paged_attn(const tq1_kv_cache* cache, const tq1_kv_batch* batch, const void* q, int64_t ldq, int64_t t,
                   int64_t n_q, float scale, int causal, int64_t window, void* out, int64_t ldo, int out_f32, void* ws,
                   size_t ws_bytes, void* stream) {
  KvCache c;
  KvBatch b;
  int rc = get_cache(cache, &c);
  if (rc != TQ1_OK) return rc;
  rc = get_batch(batch, c.page_size, t, &b);
  if (rc != TQ1_OK) return rc;
  if (n_q > 65536) return TQ1_ERR_UNSUPPORTED;
  if (n_q <= 0 || n_q % c.n_kv != 0 || window < 0 || !(scale > 0) || !std::isfinite(scale) || ldq < n_q * c.d ||
      ldo < n_q * c.d)
    return TQ1_ERR_SHAPE;
  if ((c.d != 64 && c.d != 128) || n_q / c.n_kv > 128 || t * (n_q / c.n_kv) > (int64_t{1} << 30)) return TQ1_ERR_UNSUPPORTED;
  if (t == 0) return TQ1_OK;
  if (!q || !out || !ws) return TQ1_ERR_NULL;
  if (off16(q) || off16(out) || off16(ws) || ldq % 8 != 0 || ldo % 8 != 0) return TQ1_ERR_ALIGN;
  unsigned* st = status_word();
  if (!st) return TQ1_ERR_CUDA;
  if (ws_bytes < attn_workspace_bytes(c, t, n_q, b.n_seqs)) return TQ1_ERR_WORKSPACE;
  const AttnArgs a = {static_cast<const uint16_t*>(q),
                      out,
                      ldq,
                      ldo,
                      scale,
                      static_cast<int>(n_q),
                      causal != 0,
                      static_cast<int>(window > b.max_len ? 0 : window),
                      out_f32 != 0};
  return launch_attn(c, b, a, ws, st, as_stream(stream));
}

size_t tq1_pages_workspace_size(const tq1_page_pool* pool) {
  PagePool p;
  if (get_pool(pool, &p) != TQ1_OK) return 0;
  return pages_workspace_bytes(p.n_pages, p.n_seqs);
}

int tq1_pages_copy(const tq1_page_pool* pool, const int32_t* src, const int32_t* dst, int64_t n, void* stream) {
  PagePool p;
  const int rc = get_pool(pool, &p);
  if (rc != TQ1_OK) return rc;
  if (n < 0 || n > p.n_pages) return TQ1_ERR_SHAPE;
  if (n == 0 || p.n_pools == 0) return TQ1_OK;
  if (!src || !dst) return TQ1_ERR_NULL;
  if (off4(src) || off4(dst)) return TQ1_ERR_ALIGN;
  unsigned* st = status_word();
  if (!st) return TQ1_ERR_CUDA;
  return launch_pages_copy(p, src, dst, n, st, as_stream(stream));
}

int tq1_pages_resize(const tq1_page_pool* pool, const int32_t* seqs, const int32_t* new_len, int64_t n, void* ws,
                     size_t ws_bytes, void* stream) {
  PagePool p;
  int rc = get_pool(pool, &p);
  if (rc != TQ1_OK) return rc;
  rc = check_pages_call(p, n, seqs, new_len, ws, ws_bytes);
  if (rc != TQ1_OK || n == 0) return rc;
  unsigned* st = status_word();
  if (!st) return TQ1_ERR_CUDA;
  return launch_pages_resize(p, seqs, new_len, static_cast<int>(n), ws, st, as_stream(stream));
}

int tq1_pages_fork(const tq1_page_pool* pool, const int32_t* parents, const int32_t* children, int64_t n, void* ws,
                   size_t ws_bytes, void* stream) {
  PagePool p;
  int rc = get_pool(pool, &p);
  if (rc != TQ1_OK) return rc;
  rc = check_pages_call(p, n, parents, children, ws, ws_bytes);
  if (rc != TQ1_OK || n == 0) return rc;
  unsigned* st = status_word();
  if (!st) return TQ1_ERR_CUDA;
  return launch_pages_fork(p, parents, children, static_cast<int>(n), ws, st, as_stream(stream));
}

int tq1_pages_compact(const tq1_page_pool* pool, void* ws, size_t ws_bytes, void* stream) {
  PagePool p;
  const int rc = get_pool(pool, &p);
  if (rc != TQ1_OK) return rc;
  if (!ws) return TQ1_ERR_NULL;
  if (off16(ws)) return TQ1_ERR_ALIGN;
  if (ws_bytes < pages_workspace_bytes(p.n_pages, p.n_seqs)) return TQ1_ERR_WORKSPACE;
  unsigned* st = status_word();
  if (!st) return TQ1_ERR_CUDA;
  return launch_pages_compact(p, ws, st, as_stream(stream));
}

}  // extern "C"
