// Attention over the paged 4-bit cache.
//
// A stored vector is x = S H y / d, y = 8 (z + n s) with its codes n (integers
// 0..15), fp16 zero z and scale s per group, S the sign diagonal and H the
// Walsh-Hadamard matrix (symmetric). With qt = (scale log2 e / d) H S q the
// score in base 2 is
//   8 sum over groups [ s (qt . n) + z sum(qt) ]
// and the weighted values are S H / d of
//   sum_t p_t y_t = 8 [ sum_t (p_t s_t) n_t + sum_t p_t z_t ] per group,
// so both products contract integer codes, exact in fp16, with one fp32
// operand that is split in fp16 parts; the transform is applied once per query
// and once per output row.
//
// Products (mma m16n8k16, fp16 in, fp32 sums; fragment maps in
// kvc_attend_mma.cuh). Codes are the 16-row operand: tokens in the score
// product, channels in the value product. The operand is n - 8, with z + 8 s in
// the place of z: centred, because what rounding is left in the other operand
// is multiplied by the codes' mean and lands in one channel after the inverse
// transform (measured with n itself: 2e-3 there, 1e-4 elsewhere). Two codes
// take one three-input logic op (their bits into the mantissas of 1024 + n, or
// of 64 + n for the nibble above) and one fp16 subtraction on the other pipe.
// (The bits alone, as the subnormals n 2^-24, save the subtraction but the
// products then keep only about 18 bits.) The columns are the unit's query rows, in blocks of four:
// column 2i + 0 / 1 of a score product is row i's fp16 hi / lo part (hi + lo
// holds 22 bits), so that a lane's two accumulators are the two parts of one
// row's score. Up to 4 rows the value product has the weights' hi and lo parts in
// its columns too; with more, its eight columns are eight rows and the weights
// are rounded to fp16 once (2^-12 relative at most, independent per key: no more
// than rounding the output to fp16).
//
// Work. A unit is (layer, request, kv head, block of query rows); its keys are
// chunks of 32 tokens (two tiles). All units' chunks in a row, each unit with
// kCaLead chunks' worth of fixed work before them, are cut in equal shares, one
// per CTA, from the lengths on the device: ragged batches and single long
// requests balance alike, and a captured call follows its lengths. A CTA's part of
// a unit is a segment. One warp asks for the chunks (bulk copies into a ring,
// ahead into the next segments); the others take them in turn, each with its own
// running maximum and sums, no barrier inside a segment; the segment's record (m,
// l, o per row) goes to the workspace. The second kernel merges each row's records
// and applies S H / d.
#pragma once

#include "kvc_attend_mma.cuh"
#include "kvc_cache.h"
#include "kvc_launch.cuh"

namespace kvc {

constexpr int kChunkTok = 2 * kTileTok;
constexpr uint32_t kCaLead = 6;      // a segment's fixed work, in chunks
constexpr uint32_t kCaMinShare = 8;  // chunks (and fixed work) per CTA at least

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Transposes an 8 x 8 matrix of 16-bit values held as a fragment.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Bounded wait for the phase with the given parity; false if it gave up, at once
// when another wait of the CTA has (*dead).
__device__ __forceinline__ bool ring_wait(uint64_t *bar, uint32_t parity,
                                          const volatile uint32_t *dead) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t i = 1; i < kWaitIters; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 15u) == 0 && (*dead || globaltimer() - t0 > kWaitNs)) return false;
  }
  return false;
}
// n - 8 of the codes in bits 0..3 (kHigh: 4..7) of both halves, as fp16 pairs.
template <bool kHigh>
__device__ __forceinline__ uint32_t centred(uint32_t x) {
  uint32_t t, d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;"
      : "=r"(t)
      : "r"(x), "n"(kHigh ? 0x00F000F0 : 0x000F000F), "n"(kHigh ? 0x54005400 : 0x64006400));
  asm("sub.f16x2 %0, %1, %2;" : "=r"(d) : "r"(t), "r"(kHigh ? 0x54805480u : 0x64086408u));
  return d;
}
__device__ __forceinline__ float half_lo(uint32_t m) {
  return __half2float(__ushort_as_half(uint16_t(m)));
}
__device__ __forceinline__ float half_hi(uint32_t m) {
  return __half2float(__ushort_as_half(uint16_t(m >> 16)));
}
// A meta word's z + 8 s.
__device__ __forceinline__ float zero8(uint32_t m) { return fmaf(8.f, half_lo(m), half_hi(m)); }

// A request as the host's limits and its device numbers give it: queries,
// their first row, keys, first chunk that some query sees, chunks. A request out of
// range has no queries and ok = 0.
struct ReqShape {
  uint32_t ok, nq, q0, len, chunk0, chunks;
};
__device__ __forceinline__ ReqShape request_shape(const CacheAttnArgs &a, uint32_t r) {
  ReqShape s{};
  const int64_t q0 = a.q_starts ? int64_t(__ldg(a.q_starts + r)) : int64_t(r);
  const int64_t q1 = a.q_starts ? int64_t(__ldg(a.q_starts + r + 1)) : int64_t(r) + 1;
  const int64_t len = __ldg(a.seq_lens + r);
  if (q0 < 0 || q1 < q0 || q1 > int64_t(a.q_tokens) || q1 - q0 > int64_t(a.max_q) || len < 0 ||
      len > int64_t(a.max_len))
    return s;
  s.ok = 1;
  s.nq = uint32_t(q1 - q0);
  s.q0 = uint32_t(q0);
  s.len = uint32_t(len);
  if (s.nq == 0 || len == 0) return s;
  const int64_t lo = a.window ? len - int64_t(s.nq) - int64_t(a.window) + 1 : 0;
  s.chunk0 = lo > 0 ? uint32_t(lo) / kChunkTok : 0;
  s.chunks = (s.len + kChunkTok - 1) / kChunkTok - s.chunk0;
  return s;
}
// Keys [lo, hi) that query i of a request sees.
__device__ __forceinline__ void key_range(const CacheAttnArgs &a, const ReqShape &s, uint32_t i,
                                          int32_t &lo, int32_t &hi) {
  const int64_t end = a.causal ? int64_t(s.len) - int64_t(s.nq) + int64_t(i) + 1 : int64_t(s.len);
  const int64_t beg = a.window ? end - int64_t(a.window) : 0;
  hi = int32_t(end > 0 ? end : 0);
  lo = int32_t(beg > 0 ? beg : 0);
}

// A unit's work: its chunks, and kCaLead before them. A request's units have the
// same; one without chunks has no work.
__device__ __forceinline__ uint32_t unit_work(const ReqShape &s) {
  return s.chunks ? s.chunks + kCaLead : 0;
}
// CTA b takes the work [b * share, (b + 1) * share) of all units' in a row.
__device__ __forceinline__ uint64_t work_per_cta(uint64_t total, uint32_t grid) {
  const uint64_t s = (total + grid - 1) / grid;
  return s < kCaMinShare ? kCaMinShare : s;
}
// a / b, in 32 bits where they suffice (most calls).
__device__ __forceinline__ uint64_t div64(uint64_t a, uint64_t b) {
  return ((a | b) >> 32) == 0 ? uint64_t(uint32_t(a) / uint32_t(b)) : a / b;
}

template <int D, int G, int NB>
struct CaCfg {
  static constexpr int NG = D / G;
  static constexpr int COLS = 4 * NB;
  static constexpr int W = D / 32;                  // a lane's code words of a key row
  static constexpr int KB = D / 16, MT = D / 16;    // products per tile and column block
  static constexpr int JB = NB == 1 ? 1 : NB / 2;   // column blocks of the value product
  // Warps that take chunks, and CTAs per SM. With the asking warp 16 warps per SM
  // (128 registers each), 12 (168) where a lane's state is that of 16 rows.
  static constexpr int CW = NB <= 2 ? 7 : 11;
  static constexpr int CTAS = NB <= 2 ? 2 : 1;
  static constexpr int THREADS = (CW + 1) * 32;
  static constexpr int MC = COLS < 8 || G < 64 ? 4 : 8;  // rows merged at a time
  static constexpr uint32_t TB = cache_tile_bytes(D, G), CB = cache_code_bytes(D);
  static constexpr uint32_t STAGE = 4 * TB;         // key tiles, value tiles
  // Chunks in flight per CTA: two for each warp that takes them. Position p of the
  // ring belongs to warp p % CW, and NS is a multiple of CW, so the warp that waits
  // for a stage's next phase is the one that has released the phase before (a
  // parity wait says nothing of a barrier that is two phases behind).
  static constexpr int NS = 2 * CW;
  // shared memory
  static constexpr size_t ring = 0;
  static constexpr size_t qf = ring + size_t(NS) * STAGE;
  static constexpr size_t part = qf + size_t(NB) * KB * 32 * 8;
  static constexpr size_t ml = part + size_t(CW) * MC * D * 4;
  static constexpr size_t qs = ml + size_t(CW) * COLS * 8;
  static constexpr size_t fcol = qs + size_t(COLS) * NG * 4;
  static constexpr size_t lim = fcol + size_t(COLS) * 4;
  static constexpr size_t full = lim + size_t(COLS) * 8;
  static constexpr size_t empty = full + size_t(NS) * 8;
  static constexpr size_t have = empty + size_t(NS) * 8;
  static constexpr size_t red = have + size_t(NS) * 4 + 8;
  static constexpr size_t wpre = (red + size_t(CW + 1) * 16 + 7) / 8 * 8;
  static constexpr size_t bytes(uint32_t n_req) {
    return wpre + 8 * (size_t(n_req) + 1) + 4 * (size_t(n_req) + 2);
  }
  static_assert(full % 8 == 0 && red % 8 == 0 && qf % 16 == 0 && part % 16 == 0, "alignment");
};

// Exclusive prefixes over the requests: work (per layer and head) and blocks of
// query rows. Every thread of the CTA calls it.
template <int COLS, int THREADS>
__device__ __forceinline__ void request_prefixes(const CacheAttnArgs &a, uint64_t *wpre,
                                                 uint32_t *cpre, uint64_t *red) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t n = a.n_req, per = (n + THREADS - 1) / THREADS;
  const uint32_t r0 = uint32_t(tid) * per, r1 = min(n, r0 + per);
  uint64_t w = 0, c = 0;
  for (uint32_t r = r0; r < r1; ++r) {
    const ReqShape s = request_shape(a, r);
    if (!s.ok && blockIdx.x == 0 && a.status) set_status(a.status, KVC_ERR_CORRUPT);
    const uint32_t ct = (s.nq * a.qpk + COLS - 1) / COLS;
    wpre[r] = w;  // within the thread's range; its base is added below
    cpre[r] = uint32_t(c);
    w += uint64_t(unit_work(s)) * ct;
    c += ct;
  }
  uint64_t wi = w, ci = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t x = __shfl_up_sync(0xFFFFFFFFu, wi, o), y = __shfl_up_sync(0xFFFFFFFFu, ci, o);
    if (lane >= o) wi += x, ci += y;
  }
  if (lane == 31) red[2 * warp] = wi, red[2 * warp + 1] = ci;
  __syncthreads();
  uint64_t wb = wi - w, cb = ci - c;
  for (int k = 0; k < warp; ++k) wb += red[2 * k], cb += red[2 * k + 1];
  for (uint32_t r = r0; r < r1; ++r) wpre[r] += wb, cpre[r] += uint32_t(cb);
  if (tid == THREADS - 1) wpre[n] = wb + w, cpre[n] = uint32_t(cb + c);
  __syncthreads();
}

// A CTA's part of a unit.
struct Segment {
  uint32_t l, r, h, c0, nc;      // layer, request, kv head; the unit's query rows
  uint32_t first, chunks;        // the segment's chunks
  uint64_t unit;
  int32_t any_lo, any_hi, all_lo, all_hi;  // keys that some row sees, that every row sees
  ReqShape rs;
};
// The segment at f, the place of the next one (as f). chunks may be 0: the share
// ends inside a unit's fixed work.
template <int COLS>
__device__ __forceinline__ Segment segment_at(const CacheAttnArgs &a, const uint64_t *wpre,
                                              const uint32_t *cpre, uint64_t per_layer,
                                              uint64_t f_end, uint64_t &f) {
  const uint32_t n = a.n_req, H = a.c.heads;
  Segment s;
  s.l = a.c.layers == 1 ? 0 : uint32_t(div64(f, per_layer));
  const uint64_t in_l = f - uint64_t(s.l) * per_layer;
  uint32_t lo = 0, hi = n - 1;  // largest r with wpre[r] * H <= in_l
  while (lo < hi) {
    const uint32_t mid = (lo + hi + 1) >> 1;
    if (wpre[mid] * H <= in_l) lo = mid;
    else hi = mid - 1;
  }
  s.r = lo;
  s.rs = request_shape(a, lo);
  const uint32_t rows = s.rs.nq * a.qpk, cts = (rows + COLS - 1) / COLS, work = unit_work(s.rs);
  const uint64_t in_r = in_l - wpre[lo] * H;
  const uint32_t unit_r = uint32_t(div64(in_r, work));  // h * cts + block
  s.h = unit_r / cts;
  s.c0 = (unit_r - s.h * cts) * COLS;
  s.nc = min(uint32_t(COLS), rows - s.c0);
  s.unit = uint64_t(s.l) * H * cpre[n] + uint64_t(H) * cpre[lo] + unit_r;
  const uint32_t at = uint32_t(in_r - uint64_t(unit_r) * work);
  const uint32_t end = uint32_t(min(uint64_t(work), at + (f_end - f)));
  const uint32_t c_at = at > kCaLead ? at - kCaLead : 0, c_end = end > kCaLead ? end - kCaLead : 0;
  s.first = s.rs.chunk0 + c_at;
  s.chunks = c_end - c_at;
  f += end - at;
  // rows are ordered by query
  key_range(a, s.rs, s.c0 / a.qpk, s.any_lo, s.all_hi);
  key_range(a, s.rs, (s.c0 + s.nc - 1) / a.qpk, s.all_lo, s.any_hi);
  return s;
}

template <int N>  // 1, 2 or 4 words at p (aligned to them)
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  }
}

template <int D, int G, int NB>
__global__ void __launch_bounds__(CaCfg<D, G, NB>::THREADS, CaCfg<D, G, NB>::CTAS)
    cache_attend_kernel(const __grid_constant__ CacheAttnArgs a, const int dtype) {
  using C = CaCfg<D, G, NB>;
  constexpr int NG = C::NG, COLS = C::COLS, CW = C::CW, NS = C::NS;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint2 *qf = reinterpret_cast<uint2 *>(smem + C::qf);
  float *part = reinterpret_cast<float *>(smem + C::part);
  float2 *ml = reinterpret_cast<float2 *>(smem + C::ml);
  float *qs = reinterpret_cast<float *>(smem + C::qs);
  float *fcol = reinterpret_cast<float *>(smem + C::fcol);
  int2 *lim = reinterpret_cast<int2 *>(smem + C::lim);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::full);
  uint64_t *empty = reinterpret_cast<uint64_t *>(smem + C::empty);
  uint32_t *have = reinterpret_cast<uint32_t *>(smem + C::have);  // bit x: tile x was asked for
  volatile uint32_t *dead = have + NS;  // a wait ran out: no more is waited for
  uint64_t *red = reinterpret_cast<uint64_t *>(smem + C::red);
  uint64_t *wpre = reinterpret_cast<uint64_t *>(smem + C::wpre);
  uint32_t *cpre = reinterpret_cast<uint32_t *>(wpre + a.n_req + 1);
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    mbar_fence_init();
    *dead = 0;
  }
  request_prefixes<COLS, C::THREADS>(a, wpre, cpre, red);
  const uint32_t n = a.n_req, H = a.c.heads;
  // Requests that name rows of q twice could name more blocks than the
  // workspace has records for: none is served then (the combining kernel sees
  // the mark).
  const bool over = cpre[n] > a.max_blocks;
  if (blockIdx.x == 0) {
    for (uint32_t r = tid; r <= n; r += C::THREADS) {
      a.wpre[r] = wpre[r];
      a.cpre[r] = over ? ~0u : cpre[r];
    }
    if (over && tid == 0 && a.status) set_status(a.status, KVC_ERR_CORRUPT);
  }
  if (over) return;
  const uint64_t per_layer = wpre[n] * H, total = per_layer * a.c.layers;
  const uint64_t share = work_per_cta(total, gridDim.x);
  const uint64_t f_end = min(total, (uint64_t(blockIdx.x) + 1) * share);
  uint64_t f = uint64_t(blockIdx.x) * share;
  uint32_t pos = 0;  // ring position of the segment's first chunk

  if (warp == CW) {
    // ---- the asking warp. Every chunk takes a ring position. Four chunks at a
    // time, a lane per tile of keys or values: one lane alone, a copy after the
    // other, took 1270 cycles a chunk where the warps need one every 400. The pages
    // of the next four are looked up meanwhile.
    const uint32_t sub = lane >> 2, x = (lane >> 1) & 1, kv = lane & 1;
    uint32_t armed = 0;  // positions asked for
    while (f < f_end) {
      const Segment s = segment_at<COLS>(a, wpre, cpre, per_layer, f_end, f);
      const uint8_t *base = a.c.pool + int64_t(s.l) * a.c.s_l + int64_t(s.h) * a.c.s_h + kv * a.c.s_kv;
      const int32_t *table = a.page_table + int64_t(s.r) * a.pt_stride;
      const uint32_t last = (s.rs.len - 1) / kTileTok;  // the request's last tile
      // the page of this lane's tile of chunk i, -1: no row sees the tile
      auto page_of = [&](uint32_t i) -> int32_t {
        const uint32_t tile = 2 * (s.first + i) + x;
        const int32_t t0 = int32_t(tile * kTileTok);
        if (lane >= 16 || i >= s.chunks || tile > last || t0 >= s.any_hi || t0 + kTileTok <= s.any_lo)
          return -1;
        const int32_t pg = __ldg(table + fdiv(a.tpp, tile));
        return pg >= 0 && uint32_t(pg) < a.c.num_pages ? pg : -2;  // -2: outside the pool
      };
      int32_t next = page_of(sub);
      for (uint32_t i0 = 0; i0 < s.chunks; i0 += 4) {
        const int32_t pg = next;
        const uint32_t i = i0 + sub;
        next = page_of(i + 4);
        if (pg == -2 && a.status) set_status(a.status, KVC_ERR_CORRUPT);
        const uint32_t tile = 2 * (s.first + i) + x;
        const uint32_t in_page = tile - fdiv(a.tpp, tile) * a.tpp.d;
        const int64_t off = int64_t(pg) * a.c.s_p + int64_t(in_page) * C::TB;
        const bool mine = lane < 16 && i < s.chunks;
        const uint32_t at = pos + i, st = at % NS;
        bool ok = true;
        if (mine) {
          ok = ring_wait(empty + st, ((at / NS) & 1u) ^ 1u, dead);
          if (!ok) {
            *dead = 1;
            if (a.status) set_status(a.status, KVC_ERR_TIMEOUT);
          }
        }
        if (!__all_sync(0xFFFFFFFFu, ok && !*dead)) break;  // nothing more is asked for
        armed = pos + min(i0 + 4, s.chunks);
        const bool use = mine && pg >= 0;
        const uint32_t uses = __ballot_sync(0xFFFFFFFFu, use) >> (4 * sub);  // bits 0, 2: tiles 0, 1
        // both tiles next to one another: one copy for the two
        const int64_t other = __shfl_xor_sync(0xFFFFFFFFu, off, 2);
        const bool both = (uses & 5u) == 5u && (x ? off - other : other - off) == int64_t(C::TB);
        if (mine && (lane & 3) == 0) {
          have[st] = (uses & 1u) | ((uses >> 1) & 2u);
          mbar_arrive_expect_tx(full + st, uint32_t(__popc(uses & 15u)) * C::TB);
        }
        __syncwarp();
        if (use && !(both && x))
          bulk_g2s(smem + C::ring + size_t(st) * C::STAGE + (2 * kv + x) * C::TB, base + off,
                   both ? 2 * C::TB : C::TB, full + st);
      }
      pos += s.chunks;
    }
    // after a wait that ran out, the copies in flight arrive before the CTA ends
    if (lane == 0 && *dead) {
      const uint32_t none = 0;
      for (uint32_t i = armed < NS ? 0 : armed - NS; i < armed; ++i)
        ring_wait(full + i % NS, (i / NS) & 1u, &none);
    }
    return;
  }

  const int gq = lane >> 2, tq = lane & 3;
  while (f < f_end) {
    const Segment s = segment_at<COLS>(a, wpre, cpre, per_layer, f_end, f);
    if (s.chunks == 0) continue;

    // ---- the unit's query rows: qt, its fp16 parts as fragments, group sums
    for (int col = warp; col < COLS; col += CW) {
      const bool live = uint32_t(col) < s.nc;
      const uint32_t row = s.c0 + (live ? col : 0), qi = row / a.qpk;
      const uint8_t *src = a.q + int64_t(s.l) * a.q_l + int64_t(s.rs.q0 + qi) * a.q_t +
                           int64_t(s.h * a.qpk + (row - qi * a.qpk)) * a.q_h;
      uint16_t in[C::W];
#pragma unroll
      for (int c = 0; c < C::W; ++c)
        in[c] = live ? __ldg(reinterpret_cast<const uint16_t *>(src) + lane + 32 * c) : uint16_t(0);
      uint64_t w0 = a.c.w0, w1 = a.c.w1;
      if (a.c.vec_signs) {
        uint64_t st = a.c.seed + (uint64_t(s.l) * 2 * H + s.h) * uint64_t(D / 64) * 0x9E3779B97F4A7C15ull;
        w0 = splitmix64(st);
        if constexpr (D == 128) w1 = splitmix64(st);
      }
      float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < C::W; ++c) {
        const float x = dtype == KVC_BF16 ? __uint_as_float(uint32_t(in[c]) << 16)
                                          : __half2float(__ushort_as_half(in[c]));
        const uint32_t sg = uint32_t((c < 2 ? w0 : w1) >> (32 * (c & 1) + lane)) & 1u;
        y[c] = __uint_as_float(__float_as_uint(x) ^ (sg << 31));
      }
      // strides 1 .. 16 across lanes, 32 and 64 in registers
#pragma unroll
      for (int st = 1; st < 32; st <<= 1)
#pragma unroll
        for (int c = 0; c < C::W; ++c) {
          const float o = __shfl_xor_sync(0xFFFFFFFFu, y[c], st);
          y[c] = (lane & st) ? o - y[c] : y[c] + o;
        }
#pragma unroll
      for (int st = 1; st < C::W; st <<= 1)
#pragma unroll
        for (int c = 0; c < C::W; ++c)
          if ((c & st) == 0) {
            const float u = y[c], v = y[c + st];
            y[c] = u + v;
            y[c + st] = u - v;
          }
      float mx = 0.f, gs[NG];
#pragma unroll
      for (int gg = 0; gg < NG; ++gg) gs[gg] = 0.f;
#pragma unroll
      for (int c = 0; c < C::W; ++c) {
        y[c] *= a.scale;
        mx = fmaxf(mx, fabsf(y[c]));
        gs[c * 32 / G] += y[c];
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) gs[gg] += __shfl_xor_sync(0xFFFFFFFFu, gs[gg], o);
      }
      // es = 2^(14 - e), mx in [2^(e - 1), 2^e): the hi parts reach up to 2^14
      const int e = int((__float_as_uint(mx) >> 23) & 255u) - 126;
      const bool fine = mx > 0.f && isfinite(mx) && e > -100;
      const float es = fine ? __uint_as_float(uint32_t(127 + 14 - e) << 23) : 1.f;
      if (lane == 0) {
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) qs[col * NG + gg] = gs[gg] * es;
        fcol[col] = 8.f / es;
        int32_t b = 0, t = 0;
        if (live) key_range(a, s.rs, qi, b, t);
        lim[col] = make_int2(b, t);
      }
      // channel 32 c + lane: nibble lane % 8 of word c of lane lane / 8's chunk
      const int nib = lane & 7, reg = nib & 1, half = nib >> 2;
#pragma unroll
      for (int c = 0; c < C::W; ++c) {
        const int kb = 2 * c + ((nib >> 1) & 1);
        float vh, vl;
        split_f16(y[c] * es, vh, vl);
        uint16_t *dst = reinterpret_cast<uint16_t *>(
            qf + ((col >> 2) * C::KB + kb) * 32 + (2 * (col & 3)) * 4 + (lane >> 3));
        dst[reg * 2 + half] = __half_as_ushort(__float2half_rn(vh));
        dst[4 * 4 + reg * 2 + half] = __half_as_ushort(__float2half_rn(vl));  // the next column
      }
    }
    named_bar_sync(1, CW * 32);

    // ---- running state of this lane's rows (row 4 j + tq of block j). Scores
    // are kept as s / fc (raw); m, in base 2, follows only jumps of more than 2^8
    // (weights reach 2^8; sums in fp32 lose nothing by it).
    float m[NB], thr[NB], ls[NB], z[NB][NG], oacc[C::MT][C::JB][4];
    float fc[NB], qsum[NB][NG];
    uint2 qr[NB <= 2 ? NB : 1][NB <= 2 ? C::KB : 1];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      m[j] = 0.f;           // (0 while thr is -inf)
      thr[j] = -INFINITY;   // raw score past which m is raised
      ls[j] = 0.f;
      fc[j] = fcol[4 * j + tq];
#pragma unroll
      for (int gg = 0; gg < NG; ++gg) z[j][gg] = 0.f, qsum[j][gg] = qs[(4 * j + tq) * NG + gg];
      if constexpr (NB <= 2) {
#pragma unroll
        for (int kb = 0; kb < C::KB; ++kb) qr[j][kb] = qf[(j * C::KB + kb) * 32 + lane];
      }
    }
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
      for (int j = 0; j < C::JB; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) oacc[mt][j][i] = 0.f;
    float wsc = 1.f;       // power of two: the value product's weights are p s wsc
    float s_most = 0.f;    // scales up to this keep p s wsc below fp16's range

    const uint32_t turn = pos % CW;
    for (uint32_t i = uint32_t(warp) >= turn ? warp - turn : warp + CW - turn; i < s.chunks; i += CW) {
      const uint32_t at = pos + i, st = at % NS;
      const bool here = ring_wait(full + st, (at / NS) & 1u, dead);
      if (!__all_sync(0xFFFFFFFFu, here)) {
        if (lane == 0) {
          *dead = 1;
          if (a.status) set_status(a.status, KVC_ERR_TIMEOUT);
        }
        continue;
      }
      const uint32_t got = have[st];
      if (got != 0) {
        const uint8_t *kt = smem + C::ring + size_t(st) * C::STAGE, *vt = kt + 2 * C::TB;
        const int32_t t0 = int32_t((s.first + i) * kChunkTok);
        // rows gq and gq + 8 of a tile's token operand
        const int tA = gq ^ ((gq >> 1) & 1), tB = tA + 8;
        float sc[2][NB][2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint8_t *k = kt + x * C::TB;
          uint32_t wA[C::W], wB[C::W], mA[NG], mB[NG];
          load_words<C::W>(k + tA * C::CB + 4 * C::W * tq, wA);
          load_words<C::W>(k + tB * C::CB + 4 * C::W * tq, wB);
          load_words<NG>(k + 16 * C::CB + tA * 4 * NG, mA);
          load_words<NG>(k + 16 * C::CB + tB * 4 * NG, mB);
          float acc[NB][NG][4];
#pragma unroll
          for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int gg = 0; gg < NG; ++gg)
#pragma unroll
              for (int q = 0; q < 4; ++q) acc[j][gg][q] = 0.f;
#pragma unroll
          for (int kb = 0; kb < C::KB; ++kb) {
            const uint32_t xa = wA[kb / 2] >> (8 * (kb & 1)), xb = wB[kb / 2] >> (8 * (kb & 1));
            const uint32_t af[4] = {centred<false>(xa), centred<false>(xb), centred<true>(xa),
                                    centred<true>(xb)};
#pragma unroll
            for (int j = 0; j < NB; ++j) {
              uint2 q;
              if constexpr (NB <= 2) q = qr[j][kb];
              else q = qf[(j * C::KB + kb) * 32 + lane];
              mma16816(acc[j][(kb / 2) * 32 / G], af, q.x, q.y);
            }
          }
#pragma unroll
          for (int j = 0; j < NB; ++j) sc[x][j][0] = sc[x][j][1] = 0.f;
#pragma unroll
          for (int gg = 0; gg < NG; ++gg) {
            const float sA = half_lo(mA[gg]), sB = half_lo(mB[gg]);
            const float zA = zero8(mA[gg]), zB = zero8(mB[gg]);
#pragma unroll
            for (int j = 0; j < NB; ++j) {
              sc[x][j][0] = fmaf(sA, acc[j][gg][0] + acc[j][gg][1], fmaf(zA, qsum[j][gg], sc[x][j][0]));
              sc[x][j][1] = fmaf(sB, acc[j][gg][2] + acc[j][gg][3], fmaf(zB, qsum[j][gg], sc[x][j][1]));
            }
          }
        }
        // the values' scales and zeros of the same tokens
        uint32_t vA[2][NG], vB[2][NG];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          load_words<NG>(vt + x * C::TB + 16 * C::CB + tA * 4 * NG, vA[x]);
          load_words<NG>(vt + x * C::TB + 16 * C::CB + tB * 4 * NG, vB[x]);
        }
        // no key is hidden from any row
        const bool all = got == 3 && t0 >= s.all_lo && t0 + kChunkTok <= s.all_hi;
        if (!all) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int32_t a0 = t0 + x * kTileTok + tA, b0 = t0 + x * kTileTok + tB;
            const bool there = (got >> x) & 1u;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
              const int2 b = lim[4 * j + tq];
              if (!there || a0 < b.x || a0 >= b.y) sc[x][j][0] = -INFINITY;
              if (!there || b0 < b.x || b0 >= b.y) sc[x][j][1] = -INFINITY;
            }
            // slots that no row sees may hold anything
            const bool inA = there && a0 >= s.any_lo && a0 < s.any_hi;
            const bool inB = there && b0 >= s.any_lo && b0 < s.any_hi;
#pragma unroll
            for (int gg = 0; gg < NG; ++gg) {
              vA[x][gg] = inA ? vA[x][gg] : 0u;
              vB[x][gg] = inB ? vB[x][gg] : 0u;
            }
          }
        }
        // New maximum or scale range?
        float smax = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int gg = 0; gg < NG; ++gg)
            smax = fmaxf(smax, fmaxf(half_lo(vA[x][gg]), half_lo(vB[x][gg])));
        bool raise = smax > s_most;
        float top[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          top[j] = fmaxf(fmaxf(sc[0][j][0], sc[0][j][1]), fmaxf(sc[1][j][0], sc[1][j][1]));
          raise |= top[j] > thr[j];
        }
        if (__any_sync(0xFFFFFFFFu, raise)) {
          float fac[NB];
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            float x = top[j];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
            x *= fc[j];
            fac[j] = 1.f;
            if (thr[j] == -INFINITY) {  // nothing but NaN so far, if anything
              if (x > -INFINITY) m[j] = x, thr[j] = (x + 8.f) / fc[j];
            } else if (x > m[j]) {
              fac[j] = ex2(m[j] - x);
              m[j] = x;
              thr[j] = (x + 8.f) / fc[j];
            }
            ls[j] *= fac[j];
#pragma unroll
            for (int gg = 0; gg < NG; ++gg) z[j][gg] *= fac[j];
          }
          float ratio = 1.f;
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) smax = fmaxf(smax, __shfl_xor_sync(0xFFFFFFFFu, smax, o));
          if (smax > s_most) {  // bring smax * wsc to [32, 64); up to 128 is let pass
            const uint32_t ex = (__float_as_uint(smax) >> 23) & 255u;
            const float ns = __uint_as_float((254u + 5u - ex) << 23);
            ratio = s_most == 0.f ? 1.f : ns / wsc;  // (no scale so far: oacc is 0)
            wsc = ns;
            s_most = 128.f / ns;
          }
#pragma unroll
          for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
            for (int j = 0; j < C::JB; ++j) {
              const float fa = fac[NB == 1 ? 0 : 2 * j] * ratio;
              const float fb = fac[NB == 1 ? 0 : 2 * j + 1] * ratio;
              oacc[mt][j][0] *= fa, oacc[mt][j][1] *= fb;
              oacc[mt][j][2] *= fa, oacc[mt][j][3] *= fb;
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float p[NB][2];
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            p[j][0] = ex2(fmaf(sc[x][j][0], fc[j], -m[j]));
            p[j][1] = ex2(fmaf(sc[x][j][1], fc[j], -m[j]));
            ls[j] += p[j][0] + p[j][1];
          }
          // weights of the value product per group, as its fragments
          uint32_t pf[NG][C::JB][2];
#pragma unroll
          for (int gg = 0; gg < NG; ++gg) {
            const float sA = half_lo(vA[x][gg]) * wsc, sB = half_lo(vB[x][gg]) * wsc;
            const float zA = zero8(vA[x][gg]), zB = zero8(vB[x][gg]);
            float w[NB][2];
#pragma unroll
            for (int j = 0; j < NB; ++j) {
              w[j][0] = p[j][0] * sA;
              w[j][1] = p[j][1] * sB;
              if (all) {
                z[j][gg] = fmaf(p[j][0], zA, fmaf(p[j][1], zB, z[j][gg]));
              } else {  // a hidden key weighs nothing, whatever its slot holds
                if (p[j][0] == 0.f) w[j][0] = 0.f;
                else z[j][gg] = fmaf(p[j][0], zA, z[j][gg]);
                if (p[j][1] == 0.f) w[j][1] = 0.f;
                else z[j][gg] = fmaf(p[j][1], zB, z[j][gg]);
              }
            }
#pragma unroll
            for (int j = 0; j < C::JB; ++j)
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                if constexpr (NB == 1) {
                  float vh, vl;
                  split_f16(w[0][q], vh, vl);
                  pf[gg][0][q] = movmatrix(f16x2(vh, vl));
                } else {
                  pf[gg][j][q] = movmatrix(f16x2(w[2 * j][q], w[2 * j + 1][q]));
                }
              }
          }
          // tokens of slots 2 tq, 2 tq + 1 of the two halves of the tile
          const int ta = 2 * tq + (tq & 1), tb = ta ^ 1;
          const uint8_t *src = vt + x * C::TB + gq * (D / 16);
          uint32_t v0[C::W / 2], v1[C::W / 2], v2[C::W / 2], v3[C::W / 2];
          load_words<C::W / 2>(src + ta * C::CB, v0);
          load_words<C::W / 2>(src + tb * C::CB, v1);
          load_words<C::W / 2>(src + (ta + 8) * C::CB, v2);
          load_words<C::W / 2>(src + (tb + 8) * C::CB, v3);
#pragma unroll
          for (int q = 0; q < C::W / 2; ++q)
#pragma unroll
            for (int b = 0; b < 2; ++b) {  // 32-channel block 2 q + b
              const uint32_t u = __byte_perm(v0[q], v1[q], b ? 0x7632 : 0x5410);
              const uint32_t v = __byte_perm(v2[q], v3[q], b ? 0x7632 : 0x5410);
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint32_t af[4] = {centred<false>(u >> (8 * y)), centred<true>(u >> (8 * y)),
                                        centred<false>(v >> (8 * y)), centred<true>(v >> (8 * y))};
                const int blk = 2 * q + b, mt = 2 * blk + y;
#pragma unroll
                for (int j = 0; j < C::JB; ++j)
                  mma16816(oacc[mt][j], af, pf[blk * 32 / G][j][0], pf[blk * 32 / G][j][1]);
              }
            }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (lane == 0) mbar_arrive(empty + st);
    }
    pos += s.chunks;

    // ---- the warps' results, merged into the segment's record
#pragma unroll
    for (int j = 0; j < NB; ++j) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        ls[j] += __shfl_xor_sync(0xFFFFFFFFu, ls[j], o);
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) z[j][gg] += __shfl_xor_sync(0xFFFFFFFFu, z[j][gg], o);
      }
      if (gq == 0)
        ml[warp * COLS + 4 * j + tq] = make_float2(thr[j] == -INFINITY ? -INFINITY : m[j], ls[j]);
    }
    const float up = 8.f / wsc;
    float *rec = a.rec + (s.unit + blockIdx.x) * uint64_t(COLS * (4 + D));
#pragma unroll
    for (int c0 = 0; c0 < COLS; c0 += C::MC) {
      if (c0) named_bar_sync(1, CW * 32);  // the rows before are read
#pragma unroll
      for (int mt = 0; mt < C::MT; ++mt) {
        const int ch = 32 * (mt / 2) + 4 * gq + 2 * (mt % 2), gg = (mt / 2) * 32 / G;
#pragma unroll
        for (int j = c0 / 4; j < (c0 + C::MC) / 4; ++j) {
          float even, odd;
          if constexpr (NB == 1) {
            even = oacc[mt][0][0] + oacc[mt][0][1];
            odd = oacc[mt][0][2] + oacc[mt][0][3];
          } else {
            even = oacc[mt][j / 2][j % 2];
            odd = oacc[mt][j / 2][2 + j % 2];
          }
          *reinterpret_cast<float2 *>(part + (size_t(warp) * C::MC + 4 * j - c0 + tq) * D + ch) =
              make_float2(fmaf(even, up, 8.f * z[j][gg]), fmaf(odd, up, 8.f * z[j][gg]));
        }
      }
      named_bar_sync(1, CW * 32);
      const uint32_t rows = s.nc > uint32_t(c0) ? min(s.nc - c0, uint32_t(C::MC)) : 0;
      for (uint32_t i = tid; i < rows * D; i += CW * 32) {
        const uint32_t col = i / D, ch = i % D;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < CW; ++w) M = fmaxf(M, ml[w * COLS + c0 + col].x);
        float x = 0.f, L = 0.f;
#pragma unroll
        for (int w = 0; w < CW; ++w) {
          const float2 v = ml[w * COLS + c0 + col];
          if (v.x == -INFINITY && v.y == 0.f) continue;  // this warp saw none of the row's keys
          const float k = v.x == -INFINITY ? 1.f : ex2(v.x - M);
          x = fmaf(k, part[(size_t(w) * C::MC + col) * D + ch], x);
          L = fmaf(k, v.y, L);
        }
        rec[(c0 + col) * (4 + D) + 4 + ch] = x;
        if (ch == 0) *reinterpret_cast<float2 *>(rec + (c0 + col) * (4 + D)) = make_float2(M, L);
      }
    }
    named_bar_sync(1, CW * 32);  // the shared arrays are free for the next segment
  }
}

// A row's records in turn, or split between WPR warps (few units, many records
// each): their merge, then S H / d.
template <int D, int COLS, int DT, int WPR>
__global__ void __launch_bounds__(WPR == 1 ? 128 : WPR * 32)
    cache_combine_kernel(const __grid_constant__ CacheAttnArgs a, const uint32_t grid) {
  constexpr int W = D / 32;
  __shared__ float part[WPR == 1 ? 1 : WPR][WPR == 1 ? 1 : D];
  __shared__ float2 ml[WPR];
  grid_dependency_wait();  // the records and the prefixes
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, H = a.c.heads, Hq = H * a.qpk;
  const uint64_t i = WPR == 1 ? uint64_t(blockIdx.x) * 4 + warp : uint64_t(blockIdx.x);
  if (i >= uint64_t(a.c.layers) * a.q_tokens * Hq) return;
  const uint32_t n = a.n_req, blocks = a.cpre[n];
  const uint64_t work = a.wpre[n];
  const uint64_t lt = div64(i, Hq);
  const uint32_t j = uint32_t(i - lt * Hq), l = uint32_t(div64(lt, a.q_tokens));
  const uint32_t tok = uint32_t(lt - uint64_t(l) * a.q_tokens);
  uint32_t r = tok;
  if (a.q_starts) {  // largest r with q_starts[r] <= tok
    uint32_t lo = 0, hi = n;
    while (lo < hi) {
      const uint32_t mid = (lo + hi + 1) >> 1;
      if (__ldg(a.q_starts + mid) <= int32_t(tok)) lo = mid;
      else hi = mid - 1;
    }
    r = lo;
  }
  if (r >= n || blocks == ~0u) return;
  const ReqShape rs = request_shape(a, r);
  if (!rs.ok || tok < rs.q0 || tok - rs.q0 >= rs.nq) return;  // a row that no request names
  const uint32_t h = j / a.qpk, row = (tok - rs.q0) * a.qpk + (j - h * a.qpk);
  float y[4] = {0.f, 0.f, 0.f, 0.f}, M = -INFINITY, L = 0.f;
  if (rs.chunks) {
    const uint32_t cts = (rs.nq * a.qpk + COLS - 1) / COLS, ct = row / COLS;
    const uint64_t per_layer = work * H;
    const uint64_t share = work_per_cta(per_layer * a.c.layers, grid);
    const uint64_t unit_r = uint64_t(h) * cts + ct;
    const uint64_t unit = uint64_t(l) * H * blocks + uint64_t(H) * a.cpre[r] + unit_r;
    const uint64_t f0 = uint64_t(l) * per_layer + a.wpre[r] * H + unit_r * unit_work(rs) + kCaLead;
    const uint32_t b0 = uint32_t(div64(f0, share));
    const uint32_t nrec = uint32_t(div64(f0 + rs.chunks - 1, share)) - b0 + 1;
    constexpr uint32_t kStep = COLS * (4 + D);
    const float *p0 = a.rec + (unit + b0) * uint64_t(kStep) + (row - ct * COLS) * (4 + D);
    for (uint32_t b = lane; b < nrec; b += 32) M = fmaxf(M, p0[uint64_t(b) * kStep]);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
#pragma unroll 4
    for (uint32_t b = WPR == 1 ? 0 : warp; b < nrec; b += WPR) {
      const float *p = p0 + uint64_t(b) * kStep;
      const float2 v = *reinterpret_cast<const float2 *>(p);
      const bool none = v.x == -INFINITY && v.y == 0.f;  // no key of this row in the segment
      const float k = none ? 0.f : v.x == -INFINITY ? 1.f : ex2(v.x - M);
      L = fmaf(k, v.y, L);
#pragma unroll
      for (int c = 0; c < W; ++c) {
        const float x = p[4 + lane + 32 * c];
        y[c] = none ? y[c] : fmaf(k, x, y[c]);
      }
    }
  }
  if constexpr (WPR > 1) {  // in the warps' order
#pragma unroll
    for (int c = 0; c < W; ++c) part[warp][lane + 32 * c] = y[c];
    if (lane == 0) ml[warp] = make_float2(M, L);
    __syncthreads();
    if (warp) return;
    L = 0.f;
#pragma unroll
    for (int c = 0; c < W; ++c) y[c] = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      L += ml[w].y;
#pragma unroll
      for (int c = 0; c < W; ++c) y[c] += part[w][lane + 32 * c];
    }
  }
  const bool empty = M == -INFINITY && L == 0.f;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1)
#pragma unroll
    for (int c = 0; c < W; ++c) {
      const float o = __shfl_xor_sync(0xFFFFFFFFu, y[c], s);
      y[c] = (lane & s) ? o - y[c] : y[c] + o;
    }
#pragma unroll
  for (int s = 1; s < W; s <<= 1)
#pragma unroll
    for (int c = 0; c < W; ++c)
      if ((c & s) == 0) {
        const float u = y[c], v = y[c + s];
        y[c] = u + v;
        y[c + s] = u - v;
      }
  uint64_t w0 = a.c.w0, w1 = a.c.w1;
  if (a.c.vec_signs) {  // the values' diagonal
    uint64_t st = a.c.seed + ((uint64_t(l) * 2 + 1) * H + h) * uint64_t(D / 64) * 0x9E3779B97F4A7C15ull;
    w0 = splitmix64(st);
    if constexpr (D == 128) w1 = splitmix64(st);
  }
  const float f = empty ? 0.f : 1.f / (L * float(D));
  uint16_t *out = reinterpret_cast<uint16_t *>(a.out + int64_t(l) * a.o_l + int64_t(tok) * a.o_t +
                                               int64_t(j) * a.o_h);
#pragma unroll
  for (int c = 0; c < W; ++c) {
    const uint32_t sg = uint32_t((c < 2 ? w0 : w1) >> (32 * (c & 1) + lane)) & 1u;
    const float x = empty ? 0.f : __uint_as_float(__float_as_uint(y[c] * f) ^ (sg << 31));
    out[lane + 32 * c] = DT == KVC_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x))
                                        : __half_as_ushort(__float2half_rn(x));
  }
  if (a.lse && lane == 0)
    a.lse[lt * Hq + j] = empty ? -INFINITY : fmaf(M, 0.693147180559945f, logf(L));
}

template <int D, int G, int NB>
cudaError_t cache_attend_t(int dtype, const CacheAttnArgs &a, int sms, cudaStream_t st) {
  using C = CaCfg<D, G, NB>;
  auto k = cache_attend_kernel<D, G, NB>;
  struct Tag {};
  cudaError_t e = prepare<Tag>(k, C::bytes(KVC_MAX_REQUESTS));
  if (e != cudaSuccess) return e;
  static_assert(C::CTAS * (C::bytes(KVC_MAX_REQUESTS) + 1024) <= 227 * 1024, "CTAs per SM");
  const uint32_t want = uint32_t(sms) * C::CTAS;
  const uint32_t grid = want < kCacheGridMax ? want : kCacheGridMax;
  k<<<grid, C::THREADS, C::bytes(a.n_req), st>>>(a, dtype);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // one warp per row where units are as many as CTAs (a row then has one or two
  // records), eight where a unit is spread over many CTAs
  const uint64_t rows = uint64_t(a.c.layers) * a.q_tokens * a.c.heads * a.qpk;
  const bool wide = uint64_t(a.c.layers) * a.n_req * a.c.heads * 4 < grid;
  const uint64_t cg = wide ? rows : (rows + 3) / 4;
  if (cg >= (uint64_t(1) << 31)) return cudaErrorInvalidValue;
  auto ck = dtype == KVC_BF16 ? (wide ? cache_combine_kernel<D, C::COLS, KVC_BF16, 8>
                                      : cache_combine_kernel<D, C::COLS, KVC_BF16, 1>)
                              : (wide ? cache_combine_kernel<D, C::COLS, KVC_FP16, 8>
                                      : cache_combine_kernel<D, C::COLS, KVC_FP16, 1>);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(cg));
  cfg.blockDim = dim3(wide ? 256 : 128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ck, a, grid);
}

template <int D, int G>
cudaError_t cache_attend_g(int dtype, const CacheAttnArgs &a, int sms, cudaStream_t st) {
  switch (cache_cols(uint64_t(a.max_q) * a.qpk)) {
    case 4: return cache_attend_t<D, G, 1>(dtype, a, sms, st);
    case 8: return cache_attend_t<D, G, 2>(dtype, a, sms, st);
    default: return cache_attend_t<D, G, 4>(dtype, a, sms, st);
  }
}

}  // namespace kvc
