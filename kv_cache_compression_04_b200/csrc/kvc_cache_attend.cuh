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
// tiles of 16 tokens. All units' tiles in a row are cut in equal shares, one per
// CTA, from the lengths on the device: ragged batches and single long requests
// balance alike, and a captured call follows its lengths. A CTA's part of a unit
// is a segment; its four warps take the segment's tiles in turn, each with its
// own ring of bulk copies (no block barrier inside a segment), its own running
// maximum and sums, and the segment's record (m, l, o per row) goes to the
// workspace. The second kernel merges each row's records and applies S H / d.
#pragma once

#include "kvc_attend_mma.cuh"
#include "kvc_cache.h"
#include "kvc_launch.cuh"

namespace kvc {

constexpr int kCaWarps = 4;
constexpr int kCaThreads = kCaWarps * 32;
constexpr int kCaStages = 4;           // tiles in flight per warp
constexpr uint32_t kCaMinShare = 4;    // tiles per CTA at least (one per warp)
constexpr int kCombineWarps = 4;

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
// Bounded wait for the phase with the given parity; false if it gave up.
__device__ __forceinline__ bool ring_wait(uint64_t *bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t i = 1; i < kWaitIters; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0 && globaltimer() - t0 > kWaitNs) return false;
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
// their first row, keys, first tile that some query sees, tiles. A request out of
// range has no queries and ok = 0.
struct ReqShape {
  uint32_t ok, nq, q0, len, tile0, tiles;
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
  s.tile0 = lo > 0 ? uint32_t(lo) / kTileTok : 0;
  s.tiles = (s.len + kTileTok - 1) / kTileTok - s.tile0;
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

// How the tiles are shared out: CTA b takes tiles [b * share, (b + 1) * share)
// of all units' tiles in a row.
__device__ __forceinline__ uint64_t tiles_per_cta(uint64_t total, uint32_t grid) {
  const uint64_t s = (total + grid - 1) / grid;
  return s < kCaMinShare ? kCaMinShare : s;
}

template <int D, int G, int NB>
struct CaCfg {
  static constexpr int NG = D / G;
  static constexpr int COLS = 4 * NB;
  static constexpr int W = D / 32;                  // a lane's code words of a key row
  static constexpr int KB = D / 16, MT = D / 16;    // products per tile and column block
  static constexpr int JB = NB == 1 ? 1 : NB / 2;   // column blocks of the value product
  static constexpr uint32_t TB = cache_tile_bytes(D, G), CB = cache_code_bytes(D);
  // shared memory
  static constexpr size_t ring = 0;
  static constexpr size_t bars = ring + size_t(kCaWarps) * kCaStages * 2 * TB;
  static constexpr size_t qf = bars + size_t(kCaWarps) * kCaStages * 8;
  static constexpr size_t part = qf + size_t(NB) * KB * 32 * 8;
  static constexpr size_t ml = part + size_t(kCaWarps) * COLS * D * 4;
  static constexpr size_t qs = ml + size_t(kCaWarps) * COLS * 8;
  static constexpr size_t fcol = qs + size_t(COLS) * NG * 4;
  static constexpr size_t lim = fcol + size_t(COLS) * 4;
  static constexpr size_t wpre = lim + size_t(COLS) * 8 + 64;
  static constexpr size_t bytes(uint32_t n_req) {
    return wpre + 8 * (size_t(n_req) + 1) + 4 * (size_t(n_req) + 2);
  }
  static_assert(wpre % 8 == 0 && qf % 16 == 0 && part % 16 == 0, "alignment");
};

// Exclusive prefixes over the requests: work (tiles x column blocks, per layer
// and head) and column blocks. Every thread of the CTA calls it.
template <int COLS>
__device__ __forceinline__ void request_prefixes(const CacheAttnArgs &a, uint64_t *wpre,
                                                 uint32_t *cpre, uint64_t *red) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t n = a.n_req, per = (n + kCaThreads - 1) / kCaThreads;
  const uint32_t r0 = uint32_t(tid) * per, r1 = min(n, r0 + per);
  uint64_t w = 0, c = 0;
  for (uint32_t r = r0; r < r1; ++r) {
    const ReqShape s = request_shape(a, r);
    if (!s.ok && blockIdx.x == 0 && a.status) set_status(a.status, KVC_ERR_CORRUPT);
    const uint32_t ct = (s.nq * a.qpk + COLS - 1) / COLS;
    wpre[r] = w;  // within the thread's range; its base is added below
    cpre[r] = uint32_t(c);
    w += uint64_t(s.tiles) * ct;
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
  if (tid == kCaThreads - 1) wpre[n] = wb + w, cpre[n] = uint32_t(cb + c);
  __syncthreads();
}

template <int D, int G, int NB>
__global__ void __launch_bounds__(kCaThreads, NB <= 2 ? 4 : 3)
    cache_attend_kernel(const __grid_constant__ CacheAttnArgs a, const int dtype) {
  using C = CaCfg<D, G, NB>;
  constexpr int NG = C::NG, COLS = C::COLS;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::bars) + warp * kCaStages;
  uint8_t *ring = smem + C::ring + size_t(warp) * kCaStages * 2 * C::TB;
  uint2 *qf = reinterpret_cast<uint2 *>(smem + C::qf);
  float *part = reinterpret_cast<float *>(smem + C::part);
  float2 *ml = reinterpret_cast<float2 *>(smem + C::ml);
  float *qs = reinterpret_cast<float *>(smem + C::qs);
  float *fcol = reinterpret_cast<float *>(smem + C::fcol);
  int2 *lim = reinterpret_cast<int2 *>(smem + C::lim);
  uint64_t *red = reinterpret_cast<uint64_t *>(smem + C::lim + COLS * 8);
  uint64_t *wpre = reinterpret_cast<uint64_t *>(smem + C::wpre);
  uint32_t *cpre = reinterpret_cast<uint32_t *>(wpre + a.n_req + 1);
  if (lane == 0) {
    for (int i = 0; i < kCaStages; ++i) mbar_init(bar + i, 1);
    mbar_fence_init();
  }
  request_prefixes<COLS>(a, wpre, cpre, red);
  const uint32_t n = a.n_req, H = a.c.heads;
  // Requests that name rows of q twice could name more blocks than the
  // workspace has records for: none is served then (the combining kernel sees
  // the mark).
  const bool over = cpre[n] > a.max_blocks;
  if (blockIdx.x == 0) {
    for (uint32_t r = tid; r <= n; r += kCaThreads) {
      a.wpre[r] = wpre[r];
      a.cpre[r] = over ? ~0u : cpre[r];
    }
    if (over && tid == 0 && a.status) set_status(a.status, KVC_ERR_CORRUPT);
  }
  if (over) return;
  const uint64_t per_layer = wpre[n] * H, total = per_layer * a.c.layers;
  const uint64_t share = tiles_per_cta(total, gridDim.x);
  const uint64_t f_end = min(total, (uint64_t(blockIdx.x) + 1) * share);
  uint32_t put = 0, got = 0;  // tiles this warp has asked for and used
  bool dead = false;          // a wait ran out: nothing more is asked for

  for (uint64_t f = uint64_t(blockIdx.x) * share; f < f_end;) {
    // ---- the segment: unit (l, r, h, ct), tiles [first, first + nt)
    const uint32_t l = uint32_t(f / per_layer);
    const uint64_t in_l = f - uint64_t(l) * per_layer;
    uint32_t lo = 0, hi = n - 1;  // largest r with wpre[r] * H <= in_l
    while (lo < hi) {
      const uint32_t mid = (lo + hi + 1) >> 1;
      if (wpre[mid] * H <= in_l) lo = mid;
      else hi = mid - 1;
    }
    const uint32_t r = lo;
    const ReqShape rs = request_shape(a, r);
    const uint32_t rows = rs.nq * a.qpk, cts = (rows + COLS - 1) / COLS;
    const uint64_t in_r = in_l - wpre[r] * H;
    const uint64_t unit_r = in_r / rs.tiles;  // h * cts + ct
    const uint32_t h = uint32_t(unit_r / cts), ct = uint32_t(unit_r - uint64_t(h) * cts);
    const uint32_t skip = uint32_t(in_r - unit_r * rs.tiles);
    const uint32_t nt = uint32_t(min(uint64_t(rs.tiles - skip), f_end - f));
    const uint32_t first = rs.tile0 + skip;
    const uint64_t unit = uint64_t(l) * H * cpre[n] + uint64_t(H) * cpre[r] + unit_r;
    const uint32_t c0 = ct * COLS, nc = min(uint32_t(COLS), rows - c0);  // the unit's query rows
    f += nt;

    // keys that every row sees, and that some row sees (rows are ordered by query)
    int32_t any_lo, any_hi, all_lo, all_hi;
    key_range(a, rs, c0 / a.qpk, any_lo, all_hi);
    key_range(a, rs, (c0 + nc - 1) / a.qpk, all_lo, any_hi);

    // ---- this warp's tiles first + warp, + 4, ...: copies ahead of their use
    const uint32_t mine = nt > uint32_t(warp) ? (nt - warp + kCaWarps - 1) / kCaWarps : 0;
    const uint8_t *kbase = a.c.pool + int64_t(l) * a.c.s_l + int64_t(h) * a.c.s_h;
    uint32_t asked = 0, fifo = 0, ahead = 0;  // fifo: bit i, tile (used + i) was asked for
    int32_t page_l = -1;                      // lane j: page of tile 32 * (asked / 32) + j
    auto ask = [&]() {
      if ((asked & 31u) == 0) {
        const uint32_t i = asked + lane;
        page_l = -1;
        if (i < mine) {
          const uint32_t pi = fdiv(a.tpp, first + warp + kCaWarps * i);
          const int32_t pg = __ldg(a.page_table + int64_t(r) * a.pt_stride + pi);
          if (pg >= 0 && uint32_t(pg) < a.c.num_pages) page_l = pg;
          else if (a.status) set_status(a.status, KVC_ERR_CORRUPT);
        }
      }
      const int32_t pg = __shfl_sync(0xFFFFFFFFu, page_l, asked & 31);
      const uint32_t tile = first + warp + kCaWarps * asked;
      const int32_t t0 = int32_t(tile * kTileTok);
      const bool use = pg >= 0 && t0 < any_hi && t0 + kTileTok > any_lo && !dead;
      if (use) {
        const uint32_t st = put % kCaStages;
        if (lane == 0) {
          const uint32_t in_page = tile - fdiv(a.tpp, tile) * a.tpp.d;
          const uint8_t *src = kbase + int64_t(pg) * a.c.s_p + uint64_t(in_page) * C::TB;
          mbar_arrive_expect_tx(bar + st, 2 * C::TB);
          bulk_g2s(ring + size_t(st) * 2 * C::TB, src, C::TB, bar + st);
          bulk_g2s(ring + size_t(st) * 2 * C::TB + C::TB, src + a.c.s_kv, C::TB, bar + st);
        }
        ++put;
      }
      fifo |= uint32_t(use) << ahead;
      ++ahead;
      ++asked;
    };
    while (asked < mine && ahead < kCaStages) ask();

    // ---- the unit's query rows: qt, its fp16 parts as fragments, group sums
    for (int col = warp; col < COLS; col += kCaWarps) {
      const bool live = uint32_t(col) < nc;
      const uint32_t row = c0 + (live ? col : 0), qi = row / a.qpk;
      const uint8_t *src = a.q + int64_t(l) * a.q_l + int64_t(rs.q0 + qi) * a.q_t +
                           int64_t(h * a.qpk + (row - qi * a.qpk)) * a.q_h;
      uint64_t w0 = a.c.w0, w1 = a.c.w1;
      if (a.c.vec_signs) {
        uint64_t st = a.c.seed + (uint64_t(l) * 2 * H + h) * uint64_t(D / 64) * 0x9E3779B97F4A7C15ull;
        w0 = splitmix64(st);
        if constexpr (D == 128) w1 = splitmix64(st);
      }
      float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < C::W; ++c) {
        const uint16_t b = live ? __ldg(reinterpret_cast<const uint16_t *>(src) + lane + 32 * c)
                                : uint16_t(0);
        const float x = dtype == KVC_BF16 ? __uint_as_float(uint32_t(b) << 16)
                                          : __half2float(__ushort_as_half(b));
        const uint32_t sg = uint32_t((c < 2 ? w0 : w1) >> (32 * (c & 1) + lane)) & 1u;
        y[c] = __uint_as_float(__float_as_uint(x) ^ (sg << 31));
      }
      // strides 1 .. 16 across lanes, 32 and 64 in registers
#pragma unroll
      for (int s = 1; s < 32; s <<= 1)
#pragma unroll
        for (int c = 0; c < C::W; ++c) {
          const float o = __shfl_xor_sync(0xFFFFFFFFu, y[c], s);
          y[c] = (lane & s) ? o - y[c] : y[c] + o;
        }
#pragma unroll
      for (int s = 1; s < C::W; s <<= 1)
#pragma unroll
        for (int c = 0; c < C::W; ++c)
          if ((c & s) == 0) {
            const float u = y[c], v = y[c + s];
            y[c] = u + v;
            y[c + s] = u - v;
          }
      float mx = 0.f;
#pragma unroll
      for (int c = 0; c < C::W; ++c) {
        y[c] *= a.scale;
        mx = fmaxf(mx, fabsf(y[c]));
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
      // es = 2^(14 - e), mx in [2^(e - 1), 2^e): the hi parts reach up to 2^14
      const int e = int((__float_as_uint(mx) >> 23) & 255u) - 126;
      const bool fine = mx > 0.f && isfinite(mx) && e > -100;
      const float es = fine ? __uint_as_float(uint32_t(127 + 14 - e) << 23) : 1.f;
#pragma unroll
      for (int gg = 0; gg < NG; ++gg) {
        float x = 0.f;
#pragma unroll
        for (int c = gg * G / 32; c < (gg + 1) * G / 32; ++c) x += y[c];
#pragma unroll
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
        if (lane == 0) qs[col * NG + gg] = 8.f * x;
      }
      if (lane == 0) {
        fcol[col] = 8.f / es;
        int32_t b = 0, t = 0;
        if (live) key_range(a, rs, qi, b, t);
        lim[col] = make_int2(b, t);
      }
      // channel 32 c + lane: nibble lane % 8 of word c of lane lane / 8's chunk
      const int nib = lane & 7, reg = nib & 1, half = nib >> 2;
#pragma unroll
      for (int c = 0; c < C::W; ++c) {
        const int kb = 2 * c + ((nib >> 1) & 1);
        const float v = y[c] * es;
        float vh, vl;
        split_f16(v, vh, vl);
        uint16_t *dst = reinterpret_cast<uint16_t *>(
            qf + ((col >> 2) * C::KB + kb) * 32 + (2 * (col & 3)) * 4 + (lane >> 3));
        dst[reg * 2 + half] = __half_as_ushort(__float2half_rn(vh));
        dst[4 * 4 + reg * 2 + half] = __half_as_ushort(__float2half_rn(vl));  // the next column
      }
    }
    __syncthreads();

    // ---- running state of this lane's rows (row 4 j + tq of block j)
    float m[NB], ls[NB], z[NB][NG], oacc[C::MT][C::JB][4];
    float fc[NB], qsum[NB][NG];
    uint2 qr[NB <= 2 ? NB : 1][NB <= 2 ? C::KB : 1];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      m[j] = -INFINITY;
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
    float wsc = 1.f;    // power of two: the value product's weights are p s wsc
    bool fresh = true;  // wsc is still to be chosen

    for (uint32_t used = 0; used < mine; ++used) {
      const bool have = fifo & 1u;
      fifo >>= 1;
      --ahead;
      if (have && !dead) {
        const uint32_t st = got % kCaStages;
        if (!ring_wait(bar + st, (got / kCaStages) & 1u)) {
          if (a.status) set_status(a.status, KVC_ERR_TIMEOUT);
          dead = true;
        }
        dead = __any_sync(0xFFFFFFFFu, dead);
      }
      if (have && !dead) {
        const uint8_t *kt = ring + size_t(got % kCaStages) * 2 * C::TB, *vt = kt + C::TB;
        const int32_t t0 = int32_t((first + warp + kCaWarps * used) * kTileTok);
        // rows gq and gq + 8 of the token operand
        const int tA = gq ^ ((gq >> 1) & 1), tB = tA + 8;
        uint32_t wA[C::W], wB[C::W];
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4 *>(kt + tA * C::CB + 16 * tq);
          const uint4 y = *reinterpret_cast<const uint4 *>(kt + tB * C::CB + 16 * tq);
          wA[0] = x.x, wA[1] = x.y, wA[2] = x.z, wA[3] = x.w;
          wB[0] = y.x, wB[1] = y.y, wB[2] = y.z, wB[3] = y.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2 *>(kt + tA * C::CB + 8 * tq);
          const uint2 y = *reinterpret_cast<const uint2 *>(kt + tB * C::CB + 8 * tq);
          wA[0] = x.x, wA[1] = x.y;
          wB[0] = y.x, wB[1] = y.y;
        }
        uint32_t mkA[NG], mkB[NG], mvA[NG], mvB[NG];
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) {
          mkA[gg] = reinterpret_cast<const uint32_t *>(kt + 16 * C::CB)[tA * NG + gg];
          mkB[gg] = reinterpret_cast<const uint32_t *>(kt + 16 * C::CB)[tB * NG + gg];
          mvA[gg] = reinterpret_cast<const uint32_t *>(vt + 16 * C::CB)[tA * NG + gg];
          mvB[gg] = reinterpret_cast<const uint32_t *>(vt + 16 * C::CB)[tB * NG + gg];
        }
        float s[NB][2];
        {
          float acc[NB][NG][4];
#pragma unroll
          for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int gg = 0; gg < NG; ++gg)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[j][gg][i] = 0.f;
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
          for (int j = 0; j < NB; ++j) {
            s[j][0] = s[j][1] = 0.f;
#pragma unroll
            for (int gg = 0; gg < NG; ++gg) {
              const float ca = (acc[j][gg][0] + acc[j][gg][1]) * fc[j];
              const float cb = (acc[j][gg][2] + acc[j][gg][3]) * fc[j];
              s[j][0] = fmaf(half_lo(mkA[gg]), ca, fmaf(zero8(mkA[gg]), qsum[j][gg], s[j][0]));
              s[j][1] = fmaf(half_lo(mkB[gg]), cb, fmaf(zero8(mkB[gg]), qsum[j][gg], s[j][1]));
            }
          }
        }
        const bool full = t0 >= all_lo && t0 + kTileTok <= all_hi;  // no key is hidden
        if (!full) {
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const int2 b = lim[4 * j + tq];
            if (t0 + tA < b.x || t0 + tA >= b.y) s[j][0] = -INFINITY;
            if (t0 + tB < b.x || t0 + tB >= b.y) s[j][1] = -INFINITY;
          }
          // slots that no row sees may hold anything
          const bool inA = t0 + tA >= any_lo && t0 + tA < any_hi;
          const bool inB = t0 + tB >= any_lo && t0 + tB < any_hi;
#pragma unroll
          for (int gg = 0; gg < NG; ++gg) {
            mvA[gg] = inA ? mvA[gg] : 0u;
            mvB[gg] = inB ? mvB[gg] : 0u;
          }
        }
        // New maximum or scale range? m follows only jumps of more than 2^8
        // (weights reach 2^8, sums in fp32 lose nothing by it).
        float smax = 0.f;
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) smax = fmaxf(smax, fmaxf(half_lo(mvA[gg]), half_lo(mvB[gg])));
        bool raise = smax * wsc > 128.f || (fresh && smax > 0.f);
#pragma unroll
        for (int j = 0; j < NB; ++j) raise |= fmaxf(s[j][0], s[j][1]) > m[j] + 8.f;
        if (__any_sync(0xFFFFFFFFu, raise)) {
          float fac[NB];
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            float x = fmaxf(s[j][0], s[j][1]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
            const float mn = fmaxf(m[j], x);
            fac[j] = m[j] == -INFINITY ? (ls[j] == 0.f ? 0.f : 1.f) : ex2(m[j] - mn);
            m[j] = mn;
            ls[j] *= fac[j];
#pragma unroll
            for (int gg = 0; gg < NG; ++gg) z[j][gg] *= fac[j];
          }
          float ratio = 1.f;
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) smax = fmaxf(smax, __shfl_xor_sync(0xFFFFFFFFu, smax, o));
          if (smax * wsc > 128.f || (fresh && smax > 0.f)) {  // bring smax * wsc to [32, 64)
            const uint32_t ex = (__float_as_uint(smax) >> 23) & 255u;
            const float ns = __uint_as_float((254u + 5u - ex) << 23);
            ratio = ns / wsc;
            wsc = ns;
            fresh = false;
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
        float p[NB][2];
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const float mm = m[j] == -INFINITY ? 0.f : m[j];
          p[j][0] = ex2(s[j][0] - mm);
          p[j][1] = ex2(s[j][1] - mm);
          ls[j] += p[j][0] + p[j][1];
        }
        // weights of the value product per group, as its fragments
        uint32_t pf[NG][C::JB][2];
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) {
          const float sA = half_lo(mvA[gg]) * wsc, sB = half_lo(mvB[gg]) * wsc;
          const float zA = zero8(mvA[gg]), zB = zero8(mvB[gg]);
          float w[NB][2];
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            w[j][0] = p[j][0] * sA;
            w[j][1] = p[j][1] * sB;
            float u = p[j][0] * zA, v = p[j][1] * zB;
            if (!full) {  // a hidden key weighs nothing, whatever its slot holds
              if (p[j][0] == 0.f) w[j][0] = u = 0.f;
              if (p[j][1] == 0.f) w[j][1] = v = 0.f;
            }
            z[j][gg] += u + v;
          }
#pragma unroll
          for (int j = 0; j < C::JB; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if constexpr (NB == 1) {
                float vh, vl;
                split_f16(w[0][i], vh, vl);
                pf[gg][0][i] = movmatrix(f16x2(vh, vl));
              } else {
                pf[gg][j][i] = movmatrix(f16x2(w[2 * j][i], w[2 * j + 1][i]));
              }
            }
        }
        // tokens of slots 2 tq, 2 tq + 1 of the two halves of the tile
        const int ta = 2 * tq + (tq & 1), tb = ta ^ 1;
#pragma unroll
        for (int x = 0; x < C::W / 2; ++x) {
          const uint8_t *src = vt + gq * (D / 16) + 4 * x;
          const uint32_t v0 = *reinterpret_cast<const uint32_t *>(src + ta * C::CB);
          const uint32_t v1 = *reinterpret_cast<const uint32_t *>(src + tb * C::CB);
          const uint32_t v2 = *reinterpret_cast<const uint32_t *>(src + (ta + 8) * C::CB);
          const uint32_t v3 = *reinterpret_cast<const uint32_t *>(src + (tb + 8) * C::CB);
#pragma unroll
          for (int b = 0; b < 2; ++b) {  // 32-channel block 2 x + b
            const uint32_t u = __byte_perm(v0, v1, b ? 0x7632 : 0x5410);
            const uint32_t v = __byte_perm(v2, v3, b ? 0x7632 : 0x5410);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t af[4] = {centred<false>(u >> (8 * i)), centred<true>(u >> (8 * i)),
                                      centred<false>(v >> (8 * i)), centred<true>(v >> (8 * i))};
              const int blk = 2 * x + b, mt = 2 * blk + i;
#pragma unroll
              for (int j = 0; j < C::JB; ++j)
                mma16816(oacc[mt][j], af, pf[blk * 32 / G][j][0], pf[blk * 32 / G][j][1]);
            }
          }
        }
        ++got;
        __syncwarp();  // every lane has read the stage before it is filled again
      }
      if (asked < mine) ask();
    }
    if (dead) {  // let the copies in flight arrive before anything ends
      for (; got < put; ++got) ring_wait(bar + got % kCaStages, (got / kCaStages) & 1u);
    }

    // ---- the warps' results, merged into the segment's record
#pragma unroll
    for (int j = 0; j < NB; ++j) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        ls[j] += __shfl_xor_sync(0xFFFFFFFFu, ls[j], o);
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) z[j][gg] += __shfl_xor_sync(0xFFFFFFFFu, z[j][gg], o);
      }
      if (gq == 0) ml[warp * COLS + 4 * j + tq] = make_float2(m[j], ls[j]);
    }
    const float up = 8.f / wsc;
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt) {
      const int ch = 32 * (mt / 2) + 4 * gq + 2 * (mt % 2), gg = (mt / 2) * 32 / G;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        float even, odd;
        if constexpr (NB == 1) {
          even = oacc[mt][0][0] + oacc[mt][0][1];
          odd = oacc[mt][0][2] + oacc[mt][0][3];
        } else {
          even = oacc[mt][j / 2][j % 2];
          odd = oacc[mt][j / 2][2 + j % 2];
        }
        *reinterpret_cast<float2 *>(part + (size_t(warp) * COLS + 4 * j + tq) * D + ch) =
            make_float2(fmaf(even, up, 8.f * z[j][gg]), fmaf(odd, up, 8.f * z[j][gg]));
      }
    }
    __syncthreads();
    float *rec = a.rec + (unit + blockIdx.x) * uint64_t(COLS * (4 + D));
    for (uint32_t i = tid; i < nc * D; i += kCaThreads) {
      const uint32_t col = i / D, ch = i % D;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kCaWarps; ++w) M = fmaxf(M, ml[w * COLS + col].x);
      float x = 0.f, L = 0.f;
#pragma unroll
      for (int w = 0; w < kCaWarps; ++w) {
        const float2 v = ml[w * COLS + col];
        if (v.x == -INFINITY && v.y == 0.f) continue;  // this warp saw none of the row's keys
        const float k = v.x == -INFINITY ? 1.f : ex2(v.x - M);
        x = fmaf(k, part[(size_t(w) * COLS + col) * D + ch], x);
        L = fmaf(k, v.y, L);
      }
      rec[col * (4 + D) + 4 + ch] = x;
      if (ch == 0) *reinterpret_cast<float2 *>(rec + col * (4 + D)) = make_float2(M, L);
    }
    __syncthreads();  // the shared arrays are free for the next segment
  }
}

// One warp per output row: its unit's records merged, then S H / d.
template <int D, int COLS, int DT>
__global__ void __launch_bounds__(kCombineWarps * 32)
    cache_combine_kernel(const __grid_constant__ CacheAttnArgs a, const uint32_t grid) {
  constexpr int W = D / 32;
  grid_dependency_wait();  // the records and the prefixes
  const uint32_t lane = threadIdx.x & 31, H = a.c.heads, Hq = H * a.qpk;
  const uint64_t i = uint64_t(blockIdx.x) * kCombineWarps + (threadIdx.x >> 5);
  if (i >= uint64_t(a.c.layers) * a.q_tokens * Hq) return;
  const uint32_t j = uint32_t(i % Hq), l = uint32_t(i / Hq / a.q_tokens);
  const uint32_t tok = uint32_t(i / Hq - uint64_t(l) * a.q_tokens);
  uint32_t r = tok;
  if (a.q_starts) {  // largest r with q_starts[r] <= tok
    uint32_t lo = 0, hi = a.n_req;
    while (lo < hi) {
      const uint32_t mid = (lo + hi + 1) >> 1;
      if (__ldg(a.q_starts + mid) <= int32_t(tok)) lo = mid;
      else hi = mid - 1;
    }
    r = lo;
  }
  if (r >= a.n_req || a.cpre[a.n_req] == ~0u) return;
  const ReqShape rs = request_shape(a, r);
  if (!rs.ok || tok < rs.q0 || tok - rs.q0 >= rs.nq) return;  // a row that no request names
  const uint32_t n = a.n_req, h = j / a.qpk, row = (tok - rs.q0) * a.qpk + (j - h * a.qpk);
  float y[4] = {0.f, 0.f, 0.f, 0.f}, M = -INFINITY, L = 0.f;
  if (rs.tiles) {
    const uint32_t cts = (rs.nq * a.qpk + COLS - 1) / COLS, ct = row / COLS;
    const uint64_t per_layer = a.wpre[n] * H;
    const uint64_t share = tiles_per_cta(per_layer * a.c.layers, grid);
    const uint64_t unit_r = uint64_t(h) * cts + ct;
    const uint64_t unit = uint64_t(l) * H * a.cpre[n] + uint64_t(H) * a.cpre[r] + unit_r;
    const uint64_t f0 = uint64_t(l) * per_layer + a.wpre[r] * H + unit_r * rs.tiles;
    const uint32_t b0 = uint32_t(f0 / share), b1 = uint32_t((f0 + rs.tiles - 1) / share);
    constexpr uint32_t kStep = COLS * (4 + D);
    const float *p0 = a.rec + (unit + b0) * uint64_t(kStep) + (row - ct * COLS) * (4 + D);
    for (uint32_t b = lane; b <= b1 - b0; b += 32) M = fmaxf(M, p0[uint64_t(b) * kStep]);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
#pragma unroll 4
    for (uint32_t b = 0; b <= b1 - b0; ++b) {
      const float *p = p0 + uint64_t(b) * kStep;
      const float2 v = *reinterpret_cast<const float2 *>(p);
      float k = v.x == -INFINITY ? 1.f : ex2(v.x - M);
      const bool none = v.x == -INFINITY && v.y == 0.f;  // no key of this row in the segment
      if (none) k = 0.f;
      L = fmaf(k, v.y, L);
#pragma unroll
      for (int c = 0; c < W; ++c) y[c] = none ? y[c] : fmaf(k, p[4 + lane + 32 * c], y[c]);
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
    a.lse[(uint64_t(l) * a.q_tokens + tok) * Hq + j] =
        empty ? -INFINITY : fmaf(M, 0.693147180559945f, logf(L));
}

template <int D, int G, int NB>
cudaError_t cache_attend_t(int dtype, const CacheAttnArgs &a, int sms, cudaStream_t st) {
  using C = CaCfg<D, G, NB>;
  auto k = cache_attend_kernel<D, G, NB>;
  struct Tag {};
  const size_t smem = C::bytes(a.n_req), most = C::bytes(KVC_MAX_REQUESTS);
  cudaError_t e = prepare<Tag>(k, most);
  if (e != cudaSuccess) return e;
  // resident CTAs per SM: by registers (launch bounds) and by shared memory
  // (227 KB, 1 KB of them reserved per CTA)
  const uint32_t by_smem = uint32_t((227 * 1024) / (smem + 1024)), by_regs = NB <= 2 ? 4 : 3;
  const uint32_t want = uint32_t(sms) * (by_smem < by_regs ? by_smem : by_regs);
  const uint32_t grid = want < kCacheGridMax ? want : kCacheGridMax;
  k<<<grid, kCaThreads, smem, st>>>(a, dtype);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const uint64_t rows = uint64_t(a.c.layers) * a.q_tokens * a.c.heads * a.qpk;
  const uint64_t cg = (rows + kCombineWarps - 1) / kCombineWarps;
  if (cg >= (uint64_t(1) << 31)) return cudaErrorInvalidValue;
  auto ck = dtype == KVC_BF16 ? cache_combine_kernel<D, C::COLS, KVC_BF16>
                              : cache_combine_kernel<D, C::COLS, KVC_FP16>;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(cg));
  cfg.blockDim = dim3(kCombineWarps * 32);
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
