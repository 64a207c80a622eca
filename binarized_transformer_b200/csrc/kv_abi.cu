// kv_abi.cu -- the extern "C" entry points on the paged key-value cache
// (declared in include/bwta.h): argument validation on the host, then launches
// on the caller's stream. Nothing here allocates memory.
#include <cmath>

#include "kv.cuh"

using namespace bwta;

namespace {

constexpr int64_t I32_MAX = 0x7fffffff;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? BWTA_OK : BWTA_ERR_CUDA; }

int check_cache(const bwta_kv_cache *c) {
  if (!c) return BWTA_ERR_INVALID_ARG;
  if (c->type != BWTA_KV_F16 && c->type != BWTA_KV_E4M3) return BWTA_ERR_INVALID_ARG;
  if (c->num_pages < 0 || c->n_kv_heads < 1 || c->head_dim < 1 || c->page_size < 1)
    return BWTA_ERR_INVALID_ARG;
  if (c->num_pages > I32_MAX || c->n_kv_heads > 65535) return BWTA_ERR_UNSUPPORTED;
  if (c->head_dim % 8 != 0 || c->head_dim > KV_MAX_D) return BWTA_ERR_UNSUPPORTED;
  if (c->page_size % 16 != 0 || c->page_size > 65536) return BWTA_ERR_UNSUPPORTED;
  const int64_t rows = c->n_kv_heads * c->page_size, elt = c->type == BWTA_KV_E4M3 ? 1 : 2;
  if (c->page_stride < rows * c->head_dim) return BWTA_ERR_INVALID_ARG;
  // the byte offset of any page stays far inside 64 bits
  if (c->page_stride > (int64_t)1 << 40) return BWTA_ERR_UNSUPPORTED;
  if (c->num_pages > 0 && (!c->k || !c->v)) return BWTA_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v) || c->page_stride * elt % 16 != 0)
    return BWTA_ERR_ALIGNMENT;
  if (c->type == BWTA_KV_E4M3) {
    if (c->num_pages > 0 && (!c->k_scale || !c->v_scale)) return BWTA_ERR_INVALID_ARG;
    if (c->scale_stride < rows) return BWTA_ERR_INVALID_ARG;
    if (c->scale_stride > (int64_t)1 << 40) return BWTA_ERR_UNSUPPORTED;
    if (!aligned16(c->k_scale) || !aligned16(c->v_scale) || c->scale_stride % 4 != 0)
      return BWTA_ERR_ALIGNMENT;
  }
  return BWTA_OK;
}

int check_table(const bwta_kv_table *t) {
  if (!t) return BWTA_ERR_INVALID_ARG;
  if (t->n_slots < 0 || t->max_pages < 0 || t->ld < t->max_pages) return BWTA_ERR_INVALID_ARG;
  if (t->n_slots > I32_MAX || t->max_pages > I32_MAX) return BWTA_ERR_UNSUPPORTED;
  if (t->n_slots > 0 && !t->kv_len) return BWTA_ERR_INVALID_ARG;
  if (t->n_slots > 0 && t->max_pages > 0 && !t->pages) return BWTA_ERR_INVALID_ARG;
  return BWTA_OK;
}

KvView view_of(const bwta_kv_cache *c) {
  KvView v = {};
  v.k = static_cast<const uint8_t *>(c->k);
  v.v = static_cast<const uint8_t *>(c->v);
  v.ks = c->k_scale;
  v.vs = c->v_scale;
  v.page_stride = c->page_stride;
  v.scale_stride = c->type == BWTA_KV_E4M3 ? c->scale_stride : 0;
  v.num_pages = (int32_t)c->num_pages;
  v.ps = (int32_t)c->page_size;
  v.H = (int32_t)c->n_kv_heads;
  v.D = (int32_t)c->head_dim;
  return v;
}

KvRows rows_of(const bwta_kv_table *t, const int32_t *slots) {
  KvRows r = {};
  r.pages = t->pages;
  r.len = t->kv_len;
  r.slots = slots;
  r.ld = t->ld;
  r.max_pages = (int32_t)t->max_pages;
  r.n_slots = (int32_t)t->n_slots;
  return r;
}

// The sequences of a call: n_seq of them, total_q rows.
int check_seqs(const bwta_kv_table *t, const int32_t *slots, int64_t n_seq, const int32_t *cu_q,
               int64_t total_q) {
  if (n_seq < 0 || total_q < 0) return BWTA_ERR_INVALID_ARG;
  if (!slots && n_seq > t->n_slots) return BWTA_ERR_INVALID_ARG;
  if (!cu_q && total_q != n_seq) return BWTA_ERR_INVALID_ARG;
  if (n_seq > I32_MAX || total_q > I32_MAX) return BWTA_ERR_UNSUPPORTED;
  return BWTA_OK;
}

int attn_args(const bwta_kv_cache *cache, const bwta_kv_table *table, const int32_t *slots,
              int64_t n_seq, const int32_t *cu_q, int64_t total_q, const uint16_t *q, int64_t ldq,
              int64_t n_heads, float scale, int64_t window, int64_t sinks, uint16_t *out,
              int64_t ldo, int32_t *d_status, AttnArgs &a) {
  if (int r = check_cache(cache)) return r;
  if (int r = check_table(table)) return r;
  if (int r = check_seqs(table, slots, n_seq, cu_q, total_q)) return r;
  if (n_heads < 1 || n_heads % cache->n_kv_heads != 0) return BWTA_ERR_INVALID_ARG;
  if (n_heads > 65535) return BWTA_ERR_UNSUPPORTED;
  // positions and tiles are counted in 32 bits
  if (table->max_pages * cache->page_size > I32_MAX - 65536) return BWTA_ERR_UNSUPPORTED;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return BWTA_ERR_INVALID_ARG;
  if (window < 0 || sinks < 0 || (window == 0 && sinks != 0)) return BWTA_ERR_INVALID_ARG;
  const int64_t width = n_heads * cache->head_dim;
  if (ldq < width || ldo < width) return BWTA_ERR_INVALID_ARG;
  if (total_q > 0 && (!q || !out)) return BWTA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || ldq % 8 != 0 || ldo % 8 != 0) return BWTA_ERR_ALIGNMENT;
  a.c = view_of(cache);
  a.r = rows_of(table, slots);
  a.cu_q = cu_q;
  a.n_seq = n_seq;
  a.total_q = total_q;
  a.q = q;
  a.ldq = ldq;
  a.n_heads = (int32_t)n_heads;
  a.scale = scale;
  // past every length both mean "all of them"
  a.window = window < I32_MAX ? window : 0;
  a.sinks = sinks < I32_MAX ? sinks : I32_MAX;
  a.out = out;
  a.ldo = ldo;
  a.d_status = d_status;
  return BWTA_OK;
}

KvTableView table_view(const bwta_kv_table *t) {
  KvTableView v = {};
  v.pages = t->pages;
  v.len = t->kv_len;
  v.ref = t->refcount;
  v.ld = t->ld;
  v.max_pages = (int32_t)t->max_pages;
  v.n_slots = (int32_t)t->n_slots;
  return v;
}

int check_pool(const bwta_kv_table *t, int64_t num_pages, int64_t page_size) {
  if (int r = check_table(t)) return r;
  if (num_pages < 0 || page_size < 1) return BWTA_ERR_INVALID_ARG;
  if (num_pages > BWTA_KV_MAX_POOL || page_size % 16 != 0 || page_size > 65536)
    return BWTA_ERR_UNSUPPORTED;
  if (num_pages > 0 && !t->refcount) return BWTA_ERR_INVALID_ARG;
  return BWTA_OK;
}

// The layers of a page call and their common geometry.
int check_layers(const bwta_kv_cache *src, const bwta_kv_cache *dst, int64_t n_layers, KvLayers &l,
                 KvGeometry &g) {
  if (n_layers < 1 || !src || !dst) return BWTA_ERR_INVALID_ARG;
  if (n_layers > BWTA_KV_MAX_LAYERS) return BWTA_ERR_UNSUPPORTED;
  auto same = [](const bwta_kv_cache &a, const bwta_kv_cache &b, bool pool) {
    return a.type == b.type && a.page_size == b.page_size && a.n_kv_heads == b.n_kv_heads &&
           a.head_dim == b.head_dim &&
           (!pool || (a.num_pages == b.num_pages && a.page_stride == b.page_stride &&
                      (a.type == BWTA_KV_F16 || a.scale_stride == b.scale_stride)));
  };
  for (int64_t i = 0; i < n_layers; ++i) {
    if (int r = check_cache(src + i)) return r;
    if (int r = check_cache(dst + i)) return r;
    if (!same(src[i], src[0], true) || !same(dst[i], dst[0], true) || !same(src[i], dst[i], false))
      return BWTA_ERR_INVALID_ARG;
    l.src[i] = {static_cast<uint8_t *>(src[i].k), static_cast<uint8_t *>(src[i].v), src[i].k_scale,
                src[i].v_scale};
    l.dst[i] = {static_cast<uint8_t *>(dst[i].k), static_cast<uint8_t *>(dst[i].v), dst[i].k_scale,
                dst[i].v_scale};
  }
  if (src->num_pages > BWTA_KV_MAX_POOL || dst->num_pages > BWTA_KV_MAX_POOL)
    return BWTA_ERR_UNSUPPORTED;
  const bool e4m3 = src->type == BWTA_KV_E4M3;
  const int64_t rows = src->n_kv_heads * src->page_size, elt = e4m3 ? 1 : 2;
  g = {};
  g.kv_bytes = rows * src->head_dim * elt;
  g.src_kv_stride = src->page_stride * elt;
  g.dst_kv_stride = dst->page_stride * elt;
  g.sc_bytes = e4m3 ? rows * 4 : 0;
  g.src_sc_stride = e4m3 ? src->scale_stride * 4 : 0;
  g.dst_sc_stride = e4m3 ? dst->scale_stride * 4 : 0;
  g.n_layers = (int32_t)n_layers;
  g.src_pages = (int32_t)src->num_pages;
  g.dst_pages = (int32_t)dst->num_pages;
  g.page_size = (int32_t)src->page_size;
  return BWTA_OK;
}

int check_workspace(const void *ws, int64_t have, int64_t want) {
  if (have < want || (want > 0 && !ws)) return BWTA_ERR_INVALID_ARG;
  return aligned16(ws) ? BWTA_OK : BWTA_ERR_ALIGNMENT;
}

}  // namespace

extern "C" {

int bwta_kv_append(const bwta_kv_cache *cache, const bwta_kv_table *table, const int32_t *slots,
                   int64_t n_seq, const int32_t *cu_q, int64_t total_q, const void *k, int64_t ldk,
                   const void *v, int64_t ldv, int row_type, int32_t *d_status,
                   bwta_stream_t stream) {
  if (int r = check_cache(cache)) return r;
  if (int r = check_table(table)) return r;
  if (int r = check_seqs(table, slots, n_seq, cu_q, total_q)) return r;
  if (row_type != BWTA_ROWS_F16 && row_type != BWTA_ROWS_F32) return BWTA_ERR_INVALID_ARG;
  const int64_t width = cache->n_kv_heads * cache->head_dim;
  if (ldk < width || ldv < width) return BWTA_ERR_INVALID_ARG;
  if (total_q > 0 && (!k || !v)) return BWTA_ERR_INVALID_ARG;
  const int64_t per = row_type == BWTA_ROWS_F32 ? 4 : 8;
  if (!aligned16(k) || !aligned16(v) || ldk % per != 0 || ldv % per != 0) return BWTA_ERR_ALIGNMENT;
  if (total_q == 0 || n_seq == 0) return BWTA_OK;
  KvAppendArgs a = {};
  a.c = view_of(cache);
  a.r = rows_of(table, slots);
  a.cu_q = cu_q;
  a.n_seq = n_seq;
  a.total_q = total_q;
  a.k = k;
  a.v = v;
  a.ldk = ldk;
  a.ldv = ldv;
  a.f32 = row_type == BWTA_ROWS_F32;
  a.e4m3 = cache->type == BWTA_KV_E4M3;
  a.d_status = d_status;
  return cuda_status(launch_kv_append(a, (cudaStream_t)stream));
}

int64_t bwta_attn_decode_workspace(int64_t n_heads, int64_t n_kv_heads, int64_t head_dim) {
  if (n_heads < 1 || n_kv_heads < 1 || head_dim < 1) return 0;
  return attn_decode_ws(n_heads, n_kv_heads, head_dim);
}

int bwta_attn_decode_paged(const bwta_kv_cache *cache, const bwta_kv_table *table,
                           const int32_t *slots, int64_t n_seq, const uint16_t *q, int64_t ldq,
                           int64_t n_heads, float softmax_scale, int64_t window, int64_t sinks,
                           uint16_t *out, int64_t ldo, void *workspace, int64_t workspace_bytes,
                           int32_t *d_status, bwta_stream_t stream) {
  AttnArgs a = {};
  if (int r = attn_args(cache, table, slots, n_seq, nullptr, n_seq, q, ldq, n_heads, softmax_scale,
                        window, sinks, out, ldo, d_status, a))
    return r;
  if (int r = check_workspace(workspace, workspace_bytes,
                              bwta_attn_decode_workspace(n_heads, cache->n_kv_heads, cache->head_dim)))
    return r;
  if (n_seq == 0) return BWTA_OK;
  if (n_seq * ((n_heads + 7) / 8) > I32_MAX) return BWTA_ERR_UNSUPPORTED;
  return cuda_status(launch_attn_decode(a, cache->type == BWTA_KV_E4M3, static_cast<float *>(workspace),
                                        (cudaStream_t)stream));
}

int bwta_attn_prompt_paged(const bwta_kv_cache *cache, const bwta_kv_table *table,
                           const int32_t *slots, int64_t n_seq, const int32_t *cu_q,
                           int64_t total_q, const uint16_t *q, int64_t ldq, int64_t n_heads,
                           float softmax_scale, int64_t window, int64_t sinks, uint16_t *out,
                           int64_t ldo, int32_t *d_status, bwta_stream_t stream) {
  if (!cu_q) return BWTA_ERR_INVALID_ARG;
  AttnArgs a = {};
  if (int r = attn_args(cache, table, slots, n_seq, cu_q, total_q, q, ldq, n_heads, softmax_scale,
                        window, sinks, out, ldo, d_status, a))
    return r;
  if (n_heads / cache->n_kv_heads > 128) return BWTA_ERR_UNSUPPORTED;
  if (n_seq == 0 || total_q == 0) return BWTA_OK;
  if (attn_prompt_blocks(n_seq, total_q, n_heads, cache->n_kv_heads) > I32_MAX) return BWTA_ERR_UNSUPPORTED;
  return cuda_status(launch_attn_prompt(a, cache->type == BWTA_KV_E4M3, (cudaStream_t)stream));
}

int bwta_kv_reserve(const bwta_kv_table *table, int64_t num_pages, int64_t page_size,
                    const int32_t *slots, const int32_t *n_new, int64_t n, int32_t *d_status,
                    bwta_stream_t stream) {
  if (int r = check_pool(table, num_pages, page_size)) return r;
  if (n < 0 || (n > 0 && (!slots || !n_new))) return BWTA_ERR_INVALID_ARG;
  if (n > BWTA_KV_MAX_LIST) return BWTA_ERR_UNSUPPORTED;
  if (n == 0) return BWTA_OK;
  return cuda_status(launch_kv_reserve(table_view(table), (int32_t)num_pages, (int32_t)page_size,
                                       slots, n_new, (int32_t)n, d_status, (cudaStream_t)stream));
}

int bwta_kv_free(const bwta_kv_table *table, int64_t num_pages, int64_t page_size,
                 const int32_t *slots, int64_t n, int32_t *d_status, bwta_stream_t stream) {
  if (int r = check_pool(table, num_pages, page_size)) return r;
  if (n < 0 || (n > 0 && !slots)) return BWTA_ERR_INVALID_ARG;
  if (n > I32_MAX) return BWTA_ERR_UNSUPPORTED;
  if (n == 0) return BWTA_OK;
  return cuda_status(launch_kv_free(table_view(table), (int32_t)num_pages, (int32_t)page_size,
                                    slots, n, d_status, (cudaStream_t)stream));
}

int64_t bwta_kv_pages_workspace(int64_t num_pages, int64_t n) {
  if (num_pages < 0 || n < 0) return 0;
  return 4 * kv_pages_ws_ints(num_pages, n);
}

int bwta_kv_fork(const bwta_kv_cache *caches, int64_t n_layers, const bwta_kv_table *table,
                 const int32_t *src, const int32_t *dst, int64_t n, void *workspace,
                 int64_t workspace_bytes, int32_t *d_status, bwta_stream_t stream) {
  KvLayers l;
  KvGeometry g;
  if (int r = check_layers(caches, caches, n_layers, l, g)) return r;
  if (int r = check_pool(table, caches->num_pages, caches->page_size)) return r;
  if (n < 0 || (n > 0 && (!src || !dst))) return BWTA_ERR_INVALID_ARG;
  if (n > BWTA_KV_MAX_LIST) return BWTA_ERR_UNSUPPORTED;
  if (int r = check_workspace(workspace, workspace_bytes, bwta_kv_pages_workspace(caches->num_pages, n)))
    return r;
  if (n == 0) return BWTA_OK;
  return cuda_status(launch_kv_fork(l, g, table_view(table), src, dst, (int32_t)n,
                                    static_cast<int32_t *>(workspace), d_status, (cudaStream_t)stream));
}

int bwta_kv_compact(const bwta_kv_cache *caches, int64_t n_layers, const bwta_kv_table *table,
                    int32_t *n_used, void *workspace, int64_t workspace_bytes, int32_t *d_status,
                    bwta_stream_t stream) {
  KvLayers l;
  KvGeometry g;
  if (int r = check_layers(caches, caches, n_layers, l, g)) return r;
  if (int r = check_pool(table, caches->num_pages, caches->page_size)) return r;
  if (int r = check_workspace(workspace, workspace_bytes, bwta_kv_pages_workspace(caches->num_pages, 0)))
    return r;
  return cuda_status(launch_kv_compact(l, g, table_view(table), n_used,
                                       static_cast<int32_t *>(workspace), d_status, (cudaStream_t)stream));
}

int bwta_kv_copy_pages(const bwta_kv_cache *src, const bwta_kv_cache *dst, int64_t n_layers,
                       const int32_t *src_pages, const int32_t *dst_pages, int64_t n,
                       void *workspace, int64_t workspace_bytes, int32_t *d_status,
                       bwta_stream_t stream) {
  KvLayers l;
  KvGeometry g;
  if (int r = check_layers(src, dst, n_layers, l, g)) return r;
  if (n < 0 || (n > 0 && (!src_pages || !dst_pages))) return BWTA_ERR_INVALID_ARG;
  if (n > BWTA_KV_MAX_POOL) return BWTA_ERR_UNSUPPORTED;
  if (int r = check_workspace(workspace, workspace_bytes, bwta_kv_pages_workspace(0, n))) return r;
  if (n == 0) return BWTA_OK;
  // One pool in every layer (the list then must not read what it writes), or two that share
  // nothing. Where a pool is empty no copy is made, and its pointers mean nothing.
  bool same = false;
  if (src->num_pages > 0 && dst->num_pages > 0) {
    same = true;
    bool shared = false;
    const bool scales = src->type == BWTA_KV_E4M3;
    for (int64_t i = 0; i < n_layers; ++i) {
      same = same && src[i].k == dst[i].k && src[i].v == dst[i].v &&
             (!scales || (src[i].k_scale == dst[i].k_scale && src[i].v_scale == dst[i].v_scale));
      for (int64_t j = 0; j < n_layers; ++j) {
        const bool kk = src[i].k == dst[j].k, vv = src[i].v == dst[j].v;
        const bool ks = scales && src[i].k_scale == dst[j].k_scale, vs = scales && src[i].v_scale == dst[j].v_scale;
        if (src[i].k == dst[j].v || src[i].v == dst[j].k) return BWTA_ERR_INVALID_ARG;
        if (scales && (src[i].k_scale == dst[j].v_scale || src[i].v_scale == dst[j].k_scale))
          return BWTA_ERR_INVALID_ARG;
        if (i != j && (kk || vv || ks || vs)) return BWTA_ERR_INVALID_ARG;
        // two layers into one target: its pages would hold parts of each
        if (i < j && ((dst[i].k == dst[j].k && src[i].k != src[j].k) || (dst[i].v == dst[j].v && src[i].v != src[j].v)))
          return BWTA_ERR_INVALID_ARG;
        if (scales && i < j &&
            ((dst[i].k_scale == dst[j].k_scale && src[i].k_scale != src[j].k_scale) ||
             (dst[i].v_scale == dst[j].v_scale && src[i].v_scale != src[j].v_scale)))
          return BWTA_ERR_INVALID_ARG;
        shared = shared || kk || vv || ks || vs;
      }
    }
    if (shared && !same) return BWTA_ERR_INVALID_ARG;
    if (same && (src->num_pages != dst->num_pages || src->page_stride != dst->page_stride ||
                 g.src_sc_stride != g.dst_sc_stride))
      return BWTA_ERR_INVALID_ARG;  // two descriptions of one pool
  }
  return cuda_status(launch_kv_copy(l, g, same, src_pages, dst_pages, n,
                                    static_cast<int32_t *>(workspace), d_status, (cudaStream_t)stream));
}

}  // extern "C"
