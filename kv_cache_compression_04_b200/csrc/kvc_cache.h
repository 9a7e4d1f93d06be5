// Shared by the host side and the kernels of the paged 4-bit cache
// (kvc_cache_* in include/kvc.h).
#pragma once

#include "kvc_internal.h"

namespace kvc {

constexpr int kTileTok = 16;  // tokens per tile of a block

KVC_HD constexpr uint32_t cache_code_bytes(int d) { return uint32_t(d) / 2; }
KVC_HD constexpr uint32_t cache_tile_bytes(int d, int g) {
  return kTileTok * (cache_code_bytes(d) + uint32_t(d / g) * 4);
}

// The pool as the kernels see it. `seed` is the state whose diagonal 0 is that
// of (layer 0 of the description, keys, head 0); w0 and w1 are the global
// diagonal's sign words.
struct CachePool {
  uint8_t *pool;
  int64_t s_l, s_p, s_kv, s_h;  // bytes
  uint32_t layers, heads;
  uint32_t slots;     // num_pages * page_tokens (below 2^32)
  uint32_t num_pages;
  FastDiv pt;         // page_tokens
  uint32_t vec_signs, sym;
  uint64_t seed, w0, w1;
};

// New or stored rows (kvc_cache_rows), strides in bytes.
struct RowArgs {
  uint8_t *k, *v;
  int64_t k_l, k_t, k_h, v_l, v_t, v_h;
  uint32_t tokens;
  const int64_t *slots;
  uint32_t *status;  // may be null
  float one;         // 1.0: the quantiser's integer rounding multiplies by it
};

// kvc_cache_load: the stream, checked against the pool's description.
struct LoadArgs {
  DecArgs d;  // header fields, status and the expanded meta chunks
  uint32_t group;
  uint32_t table_fits;    // 1: in_bytes reach past the token table
  uint64_t tokens_at;     // of the token table, for the chunks that the caller's numbers give
  uint32_t *note;         // the caller's status word, beside the workspace's; may be null
  const int64_t *slots;
  uint32_t lens[KVC_MAX_REQUESTS];
};

// kvc_cache_attend. Strides in bytes.
struct CacheAttnArgs {
  CachePool c;
  uint32_t n_req, qpk, max_q, causal, window;
  float scale;              // the call's scale x log2(e) / head_dim
  uint32_t q_tokens;
  const int32_t *q_starts;  // null: one query per request
  const int32_t *seq_lens;
  const int32_t *page_table;
  int64_t pt_stride;
  uint32_t max_len;         // tokens a row of the page table can name
  uint32_t max_blocks;      // blocks of 128 query rows of all requests, at most
  uint32_t row_blocks;      // blocks of up to 16 query rows of a request, at most
  FastDiv tpp;              // tiles per page
  const uint8_t *q;
  int64_t q_l, q_t, q_h;
  uint8_t *out;
  int64_t o_l, o_t, o_h;
  float *lse;
  uint32_t *status;
  // workspace: per request prefixes of work and shapes (queries, first row, keys),
  // queries per unit (fragments, or blocks of 128 rows), records per unit and warp
  uint64_t *wpre;  // per request, or per block of 128 rows
  uint4 *shapes;
  uint4 *blk;      // blocks of 128 rows: request, first row, first key tile, tiles
  uint8_t *qws;
  float *rec;
};

// Query rows of one unit of the attention: a request's (queries x query heads per kv
// head) rounded up to 4, 8 or 16; blocks of 16 (warp products) for a few more, of 128
// (tcgen05) above. A block of 16 reads the keys once more, one of 128 rows takes as long
// for 20 as for 128. 16 requests x 8 heads, blocks of 16 against of 128, in us, 32 / 48 / 64
// rows: 4096 keys 78 / 104 / 128 against 84 / 89 / 93 (d 128), 47 / 66 / 81 against 67 / 70 /
// 71 (d 64); 1024 keys 33 / 44 / 50 against 41 / 45 / 46, 25 / 32 / 35 against 35 / 38 / 39.
inline uint64_t cache_few_rows(int d) { return d == 128 ? 32 : 48; }
inline int cache_cols(uint64_t rows, int d) {
  return rows <= 4 ? 4 : rows <= 8 ? 8 : rows <= cache_few_rows(d) ? 16 : 128;
}
// A unit's query fragments in the workspace, bytes: 16-bit hi and lo parts, then
// factors and sums.
inline uint64_t cache_frag_bytes(int d, int cols) {
  if (cols > 16) return 0;
  return uint64_t(cols == 4 ? 1 : cols / 8) * uint64_t(d / 16) * 32 * (cols == 4 ? 8 : 16) + 512;
}
// A block of 128 rows' queries in the workspace, bytes: both parts as shared memory holds
// them, factors and sums.
inline uint64_t cache_block_q_bytes(int d, int g) { return 128 * (4 * uint64_t(d) + 4 * uint64_t(1 + d / g)); }
// Warps of an attention launch at most (the workspace holds a record for each
// beside one per unit): 16 for each of 160 SMs.
constexpr uint32_t kCacheWarpsMax = 2560;
// CTAs of a launch for blocks of 128 rows at most: one for each of 160 SMs.
constexpr uint32_t kCachePrefillCtas = 160;

cudaError_t launch_cache_write(int d, int g, int dtype, const CachePool &c, const RowArgs &r,
                               int sms, cudaStream_t st);
cudaError_t launch_cache_read(int d, int g, int dtype, const CachePool &c, const RowArgs &r,
                              int sms, cudaStream_t st);
// Many rows: blocks of 32 tokens of one (layer, kv, head) each.
#define KVC_DECLARE_BLOCKS(K, D)                                                        \
  cudaError_t launch_cache_##K##_blocks_d##D(int g, int dtype, const CachePool &c,      \
                                             const RowArgs &r, uint32_t blocks, int sms, \
                                             cudaStream_t st);
KVC_DECLARE_BLOCKS(write, 128)
KVC_DECLARE_BLOCKS(write, 64)
KVC_DECLARE_BLOCKS(read, 128)
KVC_DECLARE_BLOCKS(read, 64)
#undef KVC_DECLARE_BLOCKS
cudaError_t launch_cache_load(int d, int g, const CachePool &c, const LoadArgs &l, int sms,
                              cudaStream_t st);
cudaError_t launch_cache_attend_d128(int g, int dtype, const CacheAttnArgs &a, int sms,
                                     cudaStream_t st);
cudaError_t launch_cache_prefill_d128(int g, int dtype, const CacheAttnArgs &a, int sms,
                                      cudaStream_t st);
cudaError_t launch_cache_prefill_d64(int g, int dtype, const CacheAttnArgs &a, int sms,
                                     cudaStream_t st);
cudaError_t launch_cache_attend_d64(int g, int dtype, const CacheAttnArgs &a, int sms,
                                    cudaStream_t st);

}  // namespace kvc
