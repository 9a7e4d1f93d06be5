// Shared by the two forms of the paged cache's row kernels: four lanes per vector
// (kvc_cache_rows.cu) and one lane per vector (kvc_cache_blocks.cuh).
#pragma once

#include "kvc_cache.h"
#include "kvc_launch.cuh"

namespace kvc {

__device__ __forceinline__ void note(uint32_t *status, uint32_t code) {
  if (status) set_status(status, code);
}

// The row of a slot in (layer, kv, head)'s blocks: its codes, and its meta.
template <int D, int G>
struct Place {
  uint8_t *codes, *meta;
  __device__ __forceinline__ Place(const CachePool &c, uint32_t slot, uint32_t l, uint32_t kv,
                                   uint32_t h) {
    const uint32_t page = fdiv(c.pt, slot), in = slot - page * c.pt.d;
    const uint32_t tile = in / kTileTok, lane = in % kTileTok;
    uint8_t *t = c.pool + int64_t(l) * c.s_l + int64_t(page) * c.s_p + int64_t(kv) * c.s_kv +
                 int64_t(h) * c.s_h + uint64_t(tile) * cache_tile_bytes(D, G);
    codes = t + lane * cache_code_bytes(D);
    meta = t + kTileTok * cache_code_bytes(D) + lane * (D / G * 4);
  }
};

// The words 4 b + p (one per 32-channel block b) to piece p of a stored row, or from it.
template <int D>
__device__ __forceinline__ void put_words(uint8_t *codes, uint32_t p, uint32_t kv,
                                          const uint32_t (&w)[D / 32]) {
  if constexpr (D == 128) {
    uint4 v = make_uint4(w[0], w[1], w[2], w[3]);
    if (kv)
      v = make_uint4(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410),
                     __byte_perm(w[0], w[1], 0x7632), __byte_perm(w[2], w[3], 0x7632));
    *reinterpret_cast<uint4 *>(codes + 16 * p) = v;
  } else {
    uint2 v = make_uint2(w[0], w[1]);
    if (kv) v = make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[0], w[1], 0x7632));
    *reinterpret_cast<uint2 *>(codes + 8 * p) = v;
  }
}
template <int D>
__device__ __forceinline__ void get_words(const uint8_t *codes, uint32_t p, uint32_t kv,
                                          uint32_t (&w)[D / 32]) {
  if constexpr (D == 128) {
    const uint4 v = *reinterpret_cast<const uint4 *>(codes + 16 * p);
    w[0] = kv ? __byte_perm(v.x, v.z, 0x5410) : v.x;
    w[1] = kv ? __byte_perm(v.x, v.z, 0x7632) : v.y;
    w[2] = kv ? __byte_perm(v.y, v.w, 0x5410) : v.z;
    w[3] = kv ? __byte_perm(v.y, v.w, 0x7632) : v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2 *>(codes + 8 * p);
    w[0] = kv ? __byte_perm(v.x, v.y, 0x5410) : v.x;
    w[1] = kv ? __byte_perm(v.x, v.y, 0x7632) : v.y;
  }
}

// The token's slot; none (0xFFFFFFFF, never a slot number) if it is skipped.
__device__ __forceinline__ uint32_t slot_of(const RowArgs &r, const CachePool &c, uint32_t t) {
  if (t >= r.tokens) return ~0u;
  const int64_t s = __ldg(reinterpret_cast<const long long *>(r.slots) + t);
  if (s < 0) return ~0u;
  if (s >= int64_t(c.slots)) {
    note(r.status, KVC_ERR_CORRUPT);
    return ~0u;
  }
  return uint32_t(s);
}

// The meta words of a row (a vector with an error: NaN).
template <int NG>
__device__ __forceinline__ void put_meta(uint8_t *p, const uint32_t (&m)[NG], bool bad) {
  constexpr uint32_t n = 0x7FFF7FFFu;
  if constexpr (NG == 1) *reinterpret_cast<uint32_t *>(p) = bad ? n : m[0];
  else if constexpr (NG == 2) *reinterpret_cast<uint2 *>(p) = make_uint2(bad ? n : m[0], bad ? n : m[1]);
  else
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(bad ? n : m[0], bad ? n : m[1], bad ? n : m[2], bad ? n : m[3]);
}

}  // namespace kvc
