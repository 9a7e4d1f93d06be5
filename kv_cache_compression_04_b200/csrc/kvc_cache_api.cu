// Host side of the paged 4-bit cache's calls (include/kvc.h): argument checks,
// workspace layouts and launches. Allocates nothing and keeps no state.
#include "kvc_cache.h"

using namespace kvc;

namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

uint32_t block_bytes(const kvc_cache_desc *c) {
  return uint32_t(c->page_tokens) / kTileTok * cache_tile_bytes(c->head_dim, c->group_size);
}

constexpr uint64_t kGolden = 0x9E3779B97F4A7C15ull;
uint64_t effective_seed(const kvc_cache_desc *c) {
  if (c->signs != KVC_SIGNS_PER_VECTOR) return c->sign_seed;
  return c->sign_seed + uint64_t(c->first_layer) * 2u * uint64_t(c->kv_heads) *
                            uint64_t(c->head_dim / 64) * kGolden;
}

// The description without its pool pointer and strides.
kvc_status check_shape(const kvc_cache_desc *c) {
  if (!c || c->layers < 0 || c->kv_heads < 0 || c->num_pages < 0 || c->first_layer < 0 ||
      c->reserved != 0 || c->page_tokens < 1)
    return KVC_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return KVC_ERR_UNSUPPORTED;
  if (c->bits != 4 || (c->group_size != 32 && c->group_size != 64 && c->group_size != 128) ||
      c->group_size > c->head_dim)
    return KVC_ERR_UNSUPPORTED;
  if ((c->quant != KVC_QUANT_ASYM && c->quant != KVC_QUANT_SYM) ||
      (c->signs != KVC_SIGNS_GLOBAL && c->signs != KVC_SIGNS_PER_VECTOR))
    return KVC_ERR_UNSUPPORTED;
  if (c->page_tokens % kTileTok != 0 || c->page_tokens > 65536) return KVC_ERR_UNSUPPORTED;
  // slots are counted in 32 bits, (layer, kv, head) indexes too
  if (c->num_pages >= (int64_t(1) << 31) ||
      uint64_t(c->num_pages) * uint64_t(c->page_tokens) >= (uint64_t(1) << 32) ||
      uint64_t(c->layers) * 2u * uint64_t(c->kv_heads) >= (uint64_t(1) << 24))
    return KVC_ERR_UNSUPPORTED;
  return KVC_OK;
}

kvc_status check_cache(const kvc_cache_desc *c, CachePool &p) {
  const kvc_status st = check_shape(c);
  if (st != KVC_OK) return st;
  if ((c->stride_layer | c->stride_page | c->stride_kv | c->stride_head) % 16 != 0)
    return KVC_ERR_INVALID_ARG;
  if (uint64_t(c->layers) * uint64_t(c->kv_heads) * uint64_t(c->num_pages) > 0 &&
      (!c->pool || !aligned(c->pool, 16)))
    return KVC_ERR_INVALID_ARG;
  p = CachePool{};
  p.pool = static_cast<uint8_t *>(c->pool);
  p.s_l = c->stride_layer;
  p.s_p = c->stride_page;
  p.s_kv = c->stride_kv;
  p.s_h = c->stride_head;
  p.layers = uint32_t(c->layers);
  p.heads = uint32_t(c->kv_heads);
  p.slots = uint32_t(uint64_t(c->num_pages) * uint64_t(c->page_tokens));
  p.num_pages = uint32_t(c->num_pages);
  p.pt = make_fastdiv(uint32_t(c->page_tokens));
  p.vec_signs = c->signs == KVC_SIGNS_PER_VECTOR ? 1u : 0u;
  p.sym = c->quant == KVC_QUANT_SYM ? 1u : 0u;
  p.seed = effective_seed(c);
  uint64_t s = p.seed;
  p.w0 = splitmix64(s);
  p.w1 = splitmix64(s);
  return KVC_OK;
}

bool rows_ok(const void *p, int64_t a, int64_t b, int64_t c) {
  return p && aligned(p, 16) && ((a | b | c) % 8) == 0;
}

kvc_status check_rows(const kvc_cache_desc *cache, const kvc_cache_rows *r, const uint32_t *status,
                      CachePool &p, RowArgs &a, bool &empty) {
  const kvc_status st = check_cache(cache, p);
  if (st != KVC_OK) return st;
  if (!r || r->reserved != 0 || r->tokens < 0 || r->tokens >= (int64_t(1) << 31) ||
      !aligned(status, 4))
    return KVC_ERR_INVALID_ARG;
  if (r->dtype != KVC_BF16 && r->dtype != KVC_FP16) return KVC_ERR_UNSUPPORTED;
  empty = r->tokens == 0 || p.layers == 0 || p.heads == 0;
  if (empty) return KVC_OK;
  if (!rows_ok(r->k, r->k_stride_layer, r->k_stride_token, r->k_stride_head) ||
      !rows_ok(r->v, r->v_stride_layer, r->v_stride_token, r->v_stride_head) || !r->slots ||
      !aligned(r->slots, 8))
    return KVC_ERR_INVALID_ARG;
  a = RowArgs{};
  a.k = static_cast<uint8_t *>(r->k);
  a.v = static_cast<uint8_t *>(r->v);
  a.k_l = r->k_stride_layer * 2;
  a.k_t = r->k_stride_token * 2;
  a.k_h = r->k_stride_head * 2;
  a.v_l = r->v_stride_layer * 2;
  a.v_t = r->v_stride_token * 2;
  a.v_h = r->v_stride_head * 2;
  a.tokens = uint32_t(r->tokens);
  a.slots = r->slots;
  a.one = 1.0f;
  return KVC_OK;
}

// kvc_cache_load's workspace: the status word, then a 16 KB slot per meta
// chunk of the stream.
struct LoadShape {
  uint64_t tokens = 0, vectors = 0, meta_chunks = 0, total = 0;
};
kvc_status load_shape(const kvc_cache_desc *c, const int32_t *seq_lens, int32_t n, LoadShape &s) {
  const kvc_status st = check_shape(c);
  if (st != KVC_OK) return st;
  if (n < 0 || n > KVC_MAX_REQUESTS || (n > 0 && !seq_lens)) return KVC_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i) {
    if (seq_lens[i] < 0) return KVC_ERR_INVALID_ARG;
    s.tokens += uint64_t(seq_lens[i]);
  }
  s.vectors = uint64_t(c->layers) * 2u * uint64_t(c->kv_heads) * s.tokens;
  if (s.tokens >= (uint64_t(1) << 31) || s.vectors >= (uint64_t(1) << 31))
    return KVC_ERR_UNSUPPORTED;
  s.meta_chunks = (s.vectors * uint64_t(c->head_dim / c->group_size) * 4 + kChunk - 1) / kChunk;
  s.total = kWsCtl + s.meta_chunks * kChunk;
  return KVC_OK;
}

// The attention's workspace: prefixes of work and the requests' shapes; with blocks of 128
// rows, their numbers; the transformed queries per unit (layer, kv head, block of rows of
// a request); then one record per unit and per warp or CTA (each cols x (4 +
// head_dim) fp32).
struct AttnWs {
  uint64_t blocks = 0, shapes = 0, frags = 0, queries = 0, rec = 0, total = 0;
};
kvc_status check_attn(const kvc_cache_desc *cache, const kvc_cache_attn *t, CachePool &p, AttnWs &w,
                      bool pool_too) {
  kvc_status st = pool_too ? check_cache(cache, p) : check_shape(cache);
  if (st != KVC_OK) return st;
  if (!t || t->reserved != 0 || t->n_requests < 0 || t->n_requests > KVC_MAX_REQUESTS ||
      t->max_q < 1 || (t->causal != 0 && t->causal != 1) || t->window < 0 ||
      (t->window > 0 && !t->causal) || t->q_tokens < 0 || t->q_tokens > (int64_t(1) << 24) ||
      t->page_table_stride < 0 || t->page_table_pages < 0 ||
      t->page_table_pages >= (int64_t(1) << 31) || t->page_table_stride >= (int64_t(1) << 40))
    return KVC_ERR_INVALID_ARG;
  if ((t->dtype != KVC_BF16 && t->dtype != KVC_FP16) || t->q_per_kv < 1 ||
      t->q_per_kv > KVC_CACHE_MAX_Q_PER_KV)
    return KVC_ERR_UNSUPPORTED;
  if (!t->q_starts && t->q_tokens < t->n_requests) return KVC_ERR_INVALID_ARG;
  const uint64_t heads = uint64_t(cache->kv_heads), qpk = uint64_t(t->q_per_kv);
  const uint64_t rows = uint64_t(t->max_q) * qpk, cols = uint64_t(cache_cols(rows, cache->head_dim));
  const uint64_t reqs = uint64_t(t->n_requests), lh = uint64_t(cache->layers) * heads;
  w.blocks = cols > 16 ? uint64_t(t->q_tokens) * qpk / cols + reqs : reqs * ((rows + cols - 1) / cols);
  const uint64_t units = lh * w.blocks;
  // (query rows of a request, and units, are counted in 32 bits; a CTA has 32 of 128 rows)
  if (units * (cols > 16 ? 4 : 1) >= (uint64_t(1) << 31) - 1 || uint64_t(t->q_tokens) * qpk >= (uint64_t(1) << 31))
    return KVC_ERR_UNSUPPORTED;
  // (the merge has a CTA per row at most)
  if (lh * qpk * uint64_t(t->q_tokens) >= (uint64_t(1) << 31)) return KVC_ERR_UNSUPPORTED;
  w.shapes = round256(8 * ((cols > 16 ? w.blocks : reqs) + 1));
  w.frags = w.shapes + round256(16 * reqs);
  w.queries = w.frags + (cols > 16 ? round256(16 * w.blocks) : 0);
  w.rec = round256(w.queries + units * (cols > 16 ? cache_block_q_bytes(cache->head_dim, cache->group_size)
                                                  : cache_frag_bytes(cache->head_dim, int(cols))));
  w.total = w.rec + (units + (cols > 16 ? kCachePrefillCtas : kCacheWarpsMax)) * cols *
                        (4 + uint64_t(cache->head_dim)) * sizeof(float);
  return KVC_OK;
}

}  // namespace

extern "C" {

size_t kvc_cache_block_bytes(const kvc_cache_desc *cache) {
  return check_shape(cache) == KVC_OK ? block_bytes(cache) : 0;
}

uint64_t kvc_cache_stream_seed(const kvc_cache_desc *cache) {
  return check_shape(cache) == KVC_OK ? effective_seed(cache) : 0;
}

kvc_status kvc_cache_status_clear(uint32_t *status, kvc_stream_t stream) {
  if (!status || !aligned(status, 4)) return KVC_ERR_INVALID_ARG;
  return cudaMemsetAsync(status, 0, 4, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? KVC_OK
             : KVC_ERR_CUDA;
}

kvc_status kvc_cache_write(const kvc_cache_desc *cache, const kvc_cache_rows *rows,
                           uint32_t *status, kvc_stream_t stream) {
  CachePool p;
  RowArgs a;
  bool empty = false;
  const kvc_status st = check_rows(cache, rows, status, p, a, empty);
  if (st != KVC_OK || empty) return st;
  a.status = status;
  const int sms = sm_count();
  if (sms <= 0) return KVC_ERR_CUDA;
  return launch_cache_write(cache->head_dim, cache->group_size, rows->dtype, p, a, sms,
                            reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? KVC_OK
             : KVC_ERR_CUDA;
}

kvc_status kvc_cache_read(const kvc_cache_desc *cache, const kvc_cache_rows *rows,
                          uint32_t *status, kvc_stream_t stream) {
  CachePool p;
  RowArgs a;
  bool empty = false;
  const kvc_status st = check_rows(cache, rows, status, p, a, empty);
  if (st != KVC_OK || empty) return st;
  a.status = status;
  const int sms = sm_count();
  if (sms <= 0) return KVC_ERR_CUDA;
  return launch_cache_read(cache->head_dim, cache->group_size, rows->dtype, p, a, sms,
                           reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? KVC_OK
             : KVC_ERR_CUDA;
}

size_t kvc_cache_load_workspace_bytes(const kvc_cache_desc *cache, const int32_t *seq_lens,
                                      int32_t n_requests) {
  LoadShape s;
  return load_shape(cache, seq_lens, n_requests, s) == KVC_OK ? size_t(s.total) : 0;
}

kvc_status kvc_cache_load_noting(const void *in, size_t in_bytes, const kvc_cache_desc *cache,
                                 const int32_t *seq_lens, int32_t n_requests,
                                 const int64_t *slots, void *workspace, size_t workspace_bytes,
                                 uint32_t *status, kvc_stream_t stream) {
  LoadShape s;
  kvc_status st = load_shape(cache, seq_lens, n_requests, s);
  if (st != KVC_OK) return st;
  CachePool p;
  st = check_cache(cache, p);
  if (st != KVC_OK) return st;
  if (!in || !aligned(in, 16) || !workspace || !aligned(workspace, 16) || !aligned(status, 4) ||
      (s.vectors > 0 && (!slots || !aligned(slots, 8))))
    return KVC_ERR_INVALID_ARG;
  if (workspace_bytes < s.total) return KVC_ERR_CAPACITY;
  const int sms = sm_count();
  if (sms <= 0) return KVC_ERR_CUDA;
  LoadArgs a{};
  a.d.in = static_cast<const uint8_t *>(in);
  a.d.in_bytes = in_bytes;
  a.d.status = static_cast<uint32_t *>(workspace);
  a.d.layers = p.layers;
  a.d.kv_heads = p.heads;
  a.d.head_dim = uint32_t(cache->head_dim);
  a.d.n_req = uint32_t(n_requests);
  a.d.tokens = s.tokens;
  a.d.V = uint32_t(s.vectors);
  a.d.paged_receiver = 1u;
  a.d.tdiv = make_fastdiv(uint32_t(s.tokens ? s.tokens : 1));
  a.d.ws_meta = static_cast<uint8_t *>(workspace) + kWsCtl;
  a.d.ws_meta_chunks = uint32_t(s.meta_chunks);
  a.group = uint32_t(cache->group_size);
  const uint64_t code_chunks = (s.vectors * uint64_t(cache->head_dim / 2) + kChunk - 1) / kChunk;
  a.tokens_at = kHeader + 8 * (code_chunks + s.meta_chunks);
  a.table_fits = a.tokens_at + 4 * uint64_t(n_requests) <= in_bytes ? 1u : 0u;
  for (int32_t i = 0; i < n_requests; ++i) a.lens[i] = uint32_t(seq_lens[i]);
  a.slots = slots;
  a.note = status;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, kWsCtl, cs) != cudaSuccess) return KVC_ERR_CUDA;
  return launch_cache_load(cache->head_dim, cache->group_size, p, a, sms, cs) == cudaSuccess
             ? KVC_OK
             : KVC_ERR_CUDA;
}

kvc_status kvc_cache_load(const void *in, size_t in_bytes, const kvc_cache_desc *cache,
                          const int32_t *seq_lens, int32_t n_requests, const int64_t *slots,
                          void *workspace, size_t workspace_bytes, kvc_stream_t stream) {
  return kvc_cache_load_noting(in, in_bytes, cache, seq_lens, n_requests, slots, workspace,
                               workspace_bytes, nullptr, stream);
}

size_t kvc_cache_attend_workspace_bytes(const kvc_cache_desc *cache, const kvc_cache_attn *attn) {
  CachePool p;
  AttnWs w;
  return check_attn(cache, attn, p, w, false) == KVC_OK ? size_t(w.total) : 0;
}

kvc_status kvc_cache_attend(const kvc_cache_desc *cache, const kvc_cache_attn *t, void *workspace,
                            size_t workspace_bytes, uint32_t *status, kvc_stream_t stream) {
  CachePool p;
  AttnWs w;
  const kvc_status st = check_attn(cache, t, p, w, true);
  if (st != KVC_OK) return st;
  if (!aligned(status, 4)) return KVC_ERR_INVALID_ARG;
  if (p.layers == 0 || p.heads == 0 || t->n_requests == 0 || t->q_tokens == 0) return KVC_OK;
  if (!rows_ok(t->q, t->q_stride_layer, t->q_stride_token, t->q_stride_head) ||
      !rows_ok(t->out, t->out_stride_layer, t->out_stride_token, t->out_stride_head) ||
      !t->seq_lens || !aligned(t->seq_lens, 4) || !aligned(t->q_starts, 4) ||
      !aligned(t->page_table, 4) || (t->page_table_pages > 0 && !t->page_table) ||
      !aligned(t->lse, 4) || !workspace || !aligned(workspace, 16))
    return KVC_ERR_INVALID_ARG;
  if (workspace_bytes < w.total) return KVC_ERR_CAPACITY;
  const int sms = sm_count();
  if (sms <= 0) return KVC_ERR_CUDA;
  CacheAttnArgs a{};
  a.c = p;
  a.n_req = uint32_t(t->n_requests);
  a.qpk = uint32_t(t->q_per_kv);
  a.max_q = uint32_t(t->max_q);
  a.causal = uint32_t(t->causal);
  a.window = uint32_t(t->window);
  a.scale = float(double(t->scale) * 1.4426950408889634 / double(cache->head_dim));
  a.q_tokens = uint32_t(t->q_tokens);
  a.q_starts = t->q_starts;
  a.seq_lens = t->seq_lens;
  a.page_table = t->page_table;
  a.pt_stride = t->page_table_stride;
  const uint64_t reach = uint64_t(t->page_table_pages) * p.pt.d;
  a.max_len = uint32_t(reach < 0x7FFFFFFFull ? reach : 0x7FFFFFFFull);
  a.max_blocks = uint32_t(w.blocks);
  a.row_blocks = uint32_t(w.blocks / uint64_t(t->n_requests));
  a.tpp = make_fastdiv(p.pt.d / kTileTok);
  a.q = static_cast<const uint8_t *>(t->q);
  a.q_l = t->q_stride_layer * 2;
  a.q_t = t->q_stride_token * 2;
  a.q_h = t->q_stride_head * 2;
  a.out = static_cast<uint8_t *>(t->out);
  a.o_l = t->out_stride_layer * 2;
  a.o_t = t->out_stride_token * 2;
  a.o_h = t->out_stride_head * 2;
  a.lse = t->lse;
  a.status = status;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  a.wpre = reinterpret_cast<uint64_t *>(ws);
  a.shapes = reinterpret_cast<uint4 *>(ws + w.shapes);
  a.blk = reinterpret_cast<uint4 *>(ws + w.frags);
  a.qws = ws + w.queries;
  a.rec = reinterpret_cast<float *>(ws + w.rec);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const int g = cache->group_size;
  cudaError_t e;
  if (uint64_t(t->max_q) * uint64_t(t->q_per_kv) > cache_few_rows(cache->head_dim))
    e = cache->head_dim == 128 ? launch_cache_prefill_d128(g, t->dtype, a, sms, cs)
                               : launch_cache_prefill_d64(g, t->dtype, a, sms, cs);
  else
    e = cache->head_dim == 128 ? launch_cache_attend_d128(g, t->dtype, a, sms, cs)
                               : launch_cache_attend_d64(g, t->dtype, a, sms, cs);
  return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA;
}

}  // extern "C"
