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
// products then keep only about 18 bits. As e4m3, where they need no conversion
// either, the warp-level product is an emulation: 60% slower in all.) Queries are split
// in fp16 hi + lo (22 bits). The eight columns are eight query rows, the score
// product taking both parts into one sum; the value product's weights are rounded to
// fp16 once (2^-11 relative at most, independent per key, and 2^-26 of the row's largest
// weight for small ones: no more than rounding the output to fp16). Up to 4 rows, columns
// 2 i, 2 i + 1 are row i's two parts in both products.
//
// Few query rows (queries x query heads per kv head) of a request, 16 at a time; many are
// kvc_cache_prefill.cuh's (cache_few_rows).
//
// Work. A unit is (layer, kv head, block of a request's rows); its keys are chunks of 32
// tokens (two tiles). All units' chunks in a row, each unit with
// kCaLead chunks' worth of fixed work before them, are cut in equal shares, one per
// warp, from the lengths on the device: ragged batches and single long requests
// balance alike, and a captured call follows its lengths. A warp's part of a unit is
// a segment. Warps work alone, each with its own ring of two chunks, its own running
// maximum and sums: with a segment per CTA,
// its front (lengths, pages, queries) and the merge of its warps cost 8 us each, 27
// chunks' worth, in which most warps waited. Only where a CTA's whole share lies in
// one unit (long requests) are its warps merged. A segment's record (m, l, o per
// row) goes to the workspace.
// Copies are 16-byte cp.async, five instructions a tile: bulk copies of a tile
// (1088 to 1280 bytes, as 16-token pages allow) took about 70 cycles each of an SM's
// copy engine, four of them a chunk, where 32 tokens should take 200 in all.
//
// Measured: 64 ragged requests up to 8192 keys, 64 / 8 heads, two groups: 89 us for the
// second kernel against 47 for the bytes, at 374 warp instructions per tile and head and
// 2.3 issued per cycle (what bounds it; 2 of 3 are the codes' conversion, addresses and
// softmax). One request of 131072 keys, four groups: 34 us. One of 4096: 9 us of which
// the chunk itself takes 1; the kernels before and after it take 4 and 6.
//
// Three kernels: the first reads the requests' numbers, checks them, and turns each
// unit's queries into fragments; the second attends; the third merges each row's
// records and applies S H / d.
#pragma once

#include "kvc_cache_combine.cuh"

namespace kvc {

constexpr int kChunkTok = 2 * kTileTok;
constexpr uint32_t kCaLead = 2;      // a segment's fixed work, in chunks

// Transposes an 8 x 8 matrix of 16-bit values held as a fragment.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Waits until at most N of this thread's committed copy groups are in flight.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// The chunks of keys that some query of a request sees, from the first one on.
struct KeyChunks {
  uint32_t first, count;
};
__device__ __forceinline__ KeyChunks key_chunks(const CacheAttnArgs &a, const ReqShape &s) {
  if (s.nq == 0 || s.len == 0) return KeyChunks{0, 0};
  const int64_t lo = a.window ? int64_t(s.len) - int64_t(s.nq) - int64_t(a.window) + 1 : 0;
  const uint32_t first = lo > 0 ? uint32_t(lo) / kChunkTok : 0;
  return KeyChunks{first, (s.len + kChunkTok - 1) / kChunkTok - first};
}
// A unit's work: the chunks of its request's keys, and kCaLead before them; none without
// chunks.
__device__ __forceinline__ uint32_t unit_work(const KeyChunks &k) {
  return k.count ? k.count + kCaLead : 0;
}
// A request's blocks of query rows.
template <int COLS>
__device__ __forceinline__ uint32_t row_blocks(const CacheAttnArgs &a, const ReqShape &s) {
  return (s.nq * a.qpk + COLS - 1) / COLS;
}
// Warp g (of all CTAs) takes the work [g * share, (g + 1) * share) of all units'
// in a row.
__device__ __forceinline__ uint64_t work_per_warp(uint64_t total, uint32_t warps) {
  return div64(total + warps - 1, warps);
}
template <int D, int G, int NB>
struct CaCfg {
  static constexpr int NG = D / G;
  static constexpr int COLS = 4 * NB;
  static constexpr int W = D / 32;                  // a lane's code words of a key row
  static constexpr int MT = D / 16;                 // 16-channel rows of the value product
  static constexpr int RB = NB == 1 ? 1 : NB / 2;   // column blocks of either product
  static constexpr int LR = NB == 1 ? 1 : 2;        // rows a lane has per block
  static constexpr int KB = D / 16;                 // 16-channel steps of the score product
  // Warps and CTAs per SM: 12 warps with 168 registers (16 with 128 spilled, and
  // took as long or longer); as one CTA where it merges 16 rows.
  static constexpr int CW = NB <= 2 ? 6 : 12;
  static constexpr int CTAS = NB <= 2 ? 2 : 1;
  static constexpr int THREADS = CW * 32;
  static constexpr uint32_t TB = cache_tile_bytes(D, G), CB = cache_code_bytes(D);
  // A unit's query fragments in the workspace: fragments, each row's factor, its sums
  // per group.
  static constexpr uint32_t QF = uint32_t(RB) * KB * 32 * (NB == 1 ? 8 : 16);
  static constexpr uint32_t QB = QF + 512;
  static constexpr uint32_t STAGE = 4 * TB;         // key tiles, value tiles
  static constexpr int NS = 2;                      // chunks of a warp's ring
  // shared memory
  static constexpr size_t ring = 0;
  static constexpr size_t ml = ring + size_t(CW) * NS * STAGE;
  static constexpr size_t wpre = ml + size_t(CW) * COLS * 8;
  static constexpr size_t bytes(uint32_t n_req) { return wpre + 8 * (size_t(n_req) + 1); }
  // merge of the CTA's warps, in the ring's place, MC rows at a time
  static constexpr int MC = COLS < 8 ? COLS : 8;
  static_assert(size_t(CW) * MC * D * 4 <= ml, "merge buffer");
  static_assert(wpre % 8 == 0 && QF % 16 == 0, "alignment");
};

// First kernel. CTA 0 also copies the requests' shapes and the prefixes of their
// work (per layer and head) to the workspace; the others take a unit each.
constexpr int kCaPrepWarps = 4;
template <int D, int G, int NB>
__global__ void __launch_bounds__(kCaPrepWarps * 32)
    cache_attend_prep_kernel(const __grid_constant__ CacheAttnArgs a, const int dtype) {
  using C = CaCfg<D, G, NB>;
  constexpr int NG = C::NG, COLS = C::COLS, T = kCaPrepWarps * 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t n = a.n_req, H = a.c.heads;
  if (blockIdx.x == 0) {
    __shared__ uint64_t red[kCaPrepWarps];
    const uint32_t per = (n + T - 1) / T, r0 = uint32_t(tid) * per, r1 = min(n, r0 + per);
    uint64_t w = 0;
    bool bad = false;
    for (uint32_t r = r0; r < r1; ++r) {
      bool ok;
      const ReqShape s = read_request(a, r, ok);
      bad |= !ok;
      a.shapes[r] = make_uint4(s.nq, s.q0, s.len, 0);
      w += uint64_t(unit_work(key_chunks(a, s))) * row_blocks<COLS>(a, s);
    }
    if (bad && a.status) set_status(a.status, KVC_ERR_CORRUPT);
    uint64_t wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t x = __shfl_up_sync(0xFFFFFFFFu, wi, o);
      if (lane >= o) wi += x;
    }
    if (lane == 31) red[warp] = wi;
    __syncthreads();
    uint64_t base = wi - w;
    for (int k = 0; k < warp; ++k) base += red[k];
    for (uint32_t r = r0; r < r1; ++r) {
      a.wpre[r] = base;
      const uint4 v = a.shapes[r];
      const ReqShape s{v.x, v.y, v.z};
      base += uint64_t(unit_work(key_chunks(a, s))) * row_blocks<COLS>(a, s);
    }
    if (tid == T - 1) a.wpre[n] = base;
    return;
  }
  const uint32_t unit = blockIdx.x - 1, lr = unit / a.row_blocks, lh = lr / n, r = lr - lh * n;
  const uint32_t l = lh / H, h = lh - l * H, c0 = (unit - lr * a.row_blocks) * COLS;
  bool ok;
  const ReqShape rs = read_request(a, r, ok);
  const uint32_t rows = rs.nq * a.qpk;
  if (!ok || c0 >= rows || key_chunks(a, rs).count == 0) return;
  __shared__ alignas(16) uint8_t frag[C::QB];
  for (int col = warp; col < COLS; col += kCaPrepWarps) {
    const bool live = c0 + col < rows;
    const uint32_t row = live ? c0 + col : 0, qi = row / a.qpk;
    const uint8_t *src = a.q + int64_t(l) * a.q_l + int64_t(rs.q0 + qi) * a.q_t +
                         int64_t(h * a.qpk + (row - qi * a.qpk)) * a.q_h;
    uint16_t in[C::W];
#pragma unroll
    for (int c = 0; c < C::W; ++c)
      in[c] = live ? __ldg(reinterpret_cast<const uint16_t *>(src) + lane + 32 * c) : uint16_t(0);
    uint64_t w0 = a.c.w0, w1 = a.c.w1;
    if (a.c.vec_signs) {
      uint64_t st = a.c.seed + (uint64_t(l) * 2 * H + h) * uint64_t(D / 64) * 0x9E3779B97F4A7C15ull;
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
    float *qx = reinterpret_cast<float *>(frag + C::QF);
    if (lane == 0) {
#pragma unroll
      for (int gg = 0; gg < NG; ++gg) qx[COLS + col * NG + gg] = gs[gg] * es;
      qx[col] = 8.f / es;
    }
    // channel 32 c + lane: nibble lane % 8 of word c of lane lane / 8's chunk. Per
    // lane of the product b0, b1 of the hi parts, then of the lo parts (up to 4 rows:
    // its column's part only)
    const int nib = lane & 7, reg = nib & 1, half = nib >> 2;
#pragma unroll
    for (int c = 0; c < C::W; ++c) {
      const int kb = 2 * c + ((nib >> 1) & 1);
      float vh, vl;
      split_f16(y[c] * es, vh, vl);
      uint16_t *dst = reinterpret_cast<uint16_t *>(frag) + reg * 2 + half;
      if constexpr (NB == 1) {
        dst += ((kb * 32) + 8 * col + (lane >> 3)) * 4;
        dst[0] = __half_as_ushort(__float2half_rn(vh));
        dst[16] = __half_as_ushort(__float2half_rn(vl));  // the next column
      } else {
        dst += (((col >> 3) * C::KB + kb) * 32 + 4 * (col & 7) + (lane >> 3)) * 8;
        dst[0] = __half_as_ushort(__float2half_rn(vh));
        dst[4] = __half_as_ushort(__float2half_rn(vl));
      }
    }
  }
  __syncthreads();
  uint4 *dst = reinterpret_cast<uint4 *>(a.qws + uint64_t(unit) * C::QB);
  for (int i = tid; i < int(C::QF + (COLS * (1 + NG) * 4 + 15) / 16 * 16) / 16; i += T)
    dst[i] = reinterpret_cast<const uint4 *>(frag)[i];
}

// A warp's part of a unit.
struct Segment {
  uint32_t l, h, r, c0, nc;      // layer, kv head, request; first query row, rows
  uint32_t first, chunks;        // the segment's chunks
  uint64_t unit, u0, u1;         // the unit, and its work [u0, u1)
  int32_t any_lo, any_hi, all_lo, all_hi;  // keys that some row sees, that every row sees
  ReqShape rs;
};
// The segment at f, the place of the next one (as f). chunks may be 0: the share
// ends inside a unit's fixed work.
template <int COLS>
__device__ __forceinline__ Segment segment_at(const CacheAttnArgs &a, const uint64_t *wpre,
                                              uint64_t f_end, uint64_t &f) {
  const uint32_t n = a.n_req;
  Segment s;
  const uint64_t lh = div64(f, wpre[n]), in_lh = f - lh * wpre[n];
  s.l = uint32_t(lh) / a.c.heads;
  s.h = uint32_t(lh) - s.l * a.c.heads;
  const uint32_t lo = last_with(n, [&](uint32_t r) { return wpre[r] <= in_lh; });
  s.r = lo;
  s.rs = request_shape(a, lo);
  const KeyChunks kc = key_chunks(a, s.rs);
  const uint32_t work = unit_work(kc);
  const uint64_t in_r = in_lh - wpre[lo];
  const uint32_t block = uint32_t(div64(in_r, work)), at = uint32_t(in_r - uint64_t(block) * work);
  s.c0 = block * COLS;
  s.nc = min(uint32_t(COLS), s.rs.nq * a.qpk - s.c0);
  s.unit = (lh * n + lo) * a.row_blocks + block;
  const uint32_t end = uint32_t(min(uint64_t(work), at + (f_end - f)));
  const uint32_t c_at = at > kCaLead ? at - kCaLead : 0, c_end = end > kCaLead ? end - kCaLead : 0;
  s.first = kc.first + c_at;
  s.chunks = c_end - c_at;
  s.u0 = f - at;
  s.u1 = s.u0 + work;
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
    cache_attend_kernel(const __grid_constant__ CacheAttnArgs a) {
  using C = CaCfg<D, G, NB>;
  constexpr int NG = C::NG, COLS = C::COLS, CW = C::CW, NS = C::NS;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  uint8_t *ring = smem + C::ring + size_t(warp) * NS * C::STAGE;
  uint64_t *wpre = reinterpret_cast<uint64_t *>(smem + C::wpre);
  grid_dependency_wait();  // the first kernel's shapes, prefixes and fragments
  for (uint32_t r = tid; r <= a.n_req; r += C::THREADS) wpre[r] = a.wpre[r];
  __syncthreads();
  const uint64_t total = wpre[a.n_req] * a.c.heads * a.c.layers;
  const uint64_t share = work_per_warp(total, gridDim.x * CW);
  const uint32_t g = blockIdx.x * CW + warp;
  uint64_t f = uint64_t(g) * share;
  const uint64_t f_end = min(total, f + share);
  const uint64_t cta0 = uint64_t(blockIdx.x) * CW * share, cta1 = min(total, cta0 + CW * share);
  if (cta0 >= cta1) return;

  do {
    // a warp with nothing to do still looks whether it is to take part in a merge
    const bool idle = f >= f_end;
    uint64_t next = idle ? cta1 - 1 : f;
    Segment s = segment_at<COLS>(a, wpre, idle ? cta1 : f_end, next);
    if (idle) s.chunks = 0;
    f = next;
    // The CTA's whole share in one unit: its warps are merged to one record.
    const bool one_unit = s.u0 <= cta0 && cta1 <= s.u1;
    if (s.chunks == 0 && !one_unit) continue;

    // ---- the segment's chunks, copied ahead of their use (the unit's fragments are
    // read from the workspace at each: they stay in L1, beside 12 warps' rings)
    const uint32_t mine = s.chunks;
    const uint8_t *kbase = a.c.pool + int64_t(s.l) * a.c.s_l + int64_t(s.h) * a.c.s_h;
    const int32_t *table = a.page_table + int64_t(s.r) * a.pt_stride;
    const uint32_t last = (s.rs.len - 1) / kTileTok;  // the request's last tile
    int64_t off_l = -1;      // lane j: tile j % 2 of chunk (asked / 16) * 16 + j / 2, from kbase
    uint32_t asked = 0, have = 0;  // have: bits 2 i, 2 i + 1: the tiles of the ring's chunk i are there
    auto ask = [&]() {
      if ((asked & 15u) == 0) {
        off_l = -1;
        const uint32_t i = asked + (lane >> 1), tile = 2 * (s.first + i) + (lane & 1);
        const int32_t t0 = int32_t(tile * kTileTok);  // (t0 + 16 may be 2^31)
        if (i < mine && tile <= last && t0 < s.any_hi && t0 > s.any_lo - kTileTok) {
          const uint32_t pi = fdiv(a.tpp, tile);
          const int32_t pg = __ldg(table + pi);
          if (pg >= 0 && uint32_t(pg) < a.c.num_pages)
            off_l = int64_t(pg) * a.c.s_p + int64_t(tile - pi * a.tpp.d) * C::TB;
          else if (a.status)
            set_status(a.status, KVC_ERR_CORRUPT);
        }
      }
      const uint32_t st = asked % NS;
      uint8_t *dst = ring + size_t(st) * C::STAGE;
      uint32_t got = 0;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int64_t off = __shfl_sync(0xFFFFFFFFu, off_l, 2 * (asked & 15u) + x);
        if (off >= 0) {  // codes of keys and values, then both metas (lanes of each)
          got |= 1u << x;
          const uint8_t *k = kbase + off + 16 * lane, *v = k + a.c.s_kv;
          uint8_t *d = dst + x * C::TB + 16 * lane;
#pragma unroll
          for (int i = 0; i < int(16 * C::CB) / 512; ++i) {
            cp_async16_s(smem_u32(d + 512 * i), k + 512 * i);
            cp_async16_s(smem_u32(d + 2 * C::TB + 512 * i), v + 512 * i);
          }
          constexpr int ML = 4 * NG;  // lanes of a tile's meta
          const bool of_v = lane >= ML;
          if (lane < 2 * ML)
            cp_async16_s(smem_u32(d + 16 * C::CB + (of_v ? 2 * C::TB - 16 * ML : 0)),
                         (of_v ? v - 16 * ML : k) + 16 * C::CB);
        }
      }
      cp_async_commit();
      have = (have & ~(3u << (2 * st))) | (got << (2 * st));
      ++asked;
    };
    const uint8_t *qsrc = a.qws + s.unit * C::QB;
    for (int i = 0; i < NS; ++i) {
      if (asked < mine) ask();
      else cp_async_commit();
    }

    // ---- running state of this lane's rows: LR per block, row (NB == 1 ? tq : 8 b +
    // 2 tq + i). Scores are kept raw; n (row_factor) is a row's own, as rows weigh the same
    // keys differently.
    constexpr int R = C::RB * C::LR;
    auto row_of = [&](int i) { return NB == 1 ? tq : 8 * (i / 2) + 2 * tq + i % 2; };
    float nm[R], lim[R], ls[R], z[R][NG], oacc[C::MT][C::RB][4];
    // (four groups: their sums are read at each chunk, from L1)
    const float *qx = reinterpret_cast<const float *>(qsrc + C::QF);
    float fc[R], qsum[R][NG < 4 ? NG : 1];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      nm[i] = 0.f;          // n
      lim[i] = -INFINITY;   // most log2 p may be (-inf: no keys so far, or nothing but NaN)
      ls[i] = 0.f;
      fc[i] = mine ? __ldg(qx + row_of(i)) : 1.f;
#pragma unroll
      for (int gg = 0; gg < NG; ++gg) {
        z[i][gg] = 0.f;
        if constexpr (NG < 4) qsum[i][gg] = mine ? __ldg(qx + COLS + row_of(i) * NG + gg) : 0.f;
      }
    }
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
      for (int b = 0; b < C::RB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) oacc[mt][b][i] = 0.f;
    // rows gq and gq + 8 of a tile's token operand; the tokens of the value product's
    // columns 2 tq, 2 tq + 1 (and + 8) are then ta, tb (and + 8)
    const int tA = gq ^ ((gq >> 1) & 1), tB = tA + 8;
    const int ta = 2 * tq + (tq & 1), tb = ta ^ 1;

    for (uint32_t used = 0; used < mine; ++used) {
      cp_async_wait<NS - 1>();
      __syncwarp();
      const uint32_t st = used % NS, got = (have >> (2 * st)) & 3u;
      if (got != 0) {
        const uint8_t *kt = ring + size_t(st) * C::STAGE, *vt = kt + 2 * C::TB;
        const int32_t t0 = int32_t((s.first + used) * kChunkTok);
        float sc[2][R][2];  // tile, row, token tA / tB
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < R; ++i) sc[x][i][0] = sc[x][i][1] = 0.f;
        {
          uint32_t wA[2][C::W], wB[2][C::W];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            load_words<C::W>(kt + x * C::TB + tA * C::CB + 4 * C::W * tq, wA[x]);
            load_words<C::W>(kt + x * C::TB + tB * C::CB + 4 * C::W * tq, wB[x]);
          }
#pragma unroll
          for (int gg = 0; gg < NG; ++gg) {
            float acc[2][C::RB][4];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int b = 0; b < C::RB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[x][b][i] = 0.f;
#pragma unroll
            for (int kb = gg * G / 16; kb < (gg + 1) * G / 16; ++kb) {
              uint32_t af[2][4];
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t xa = wA[x][kb / 2] >> (8 * (kb & 1)), xb = wB[x][kb / 2] >> (8 * (kb & 1));
                af[x][0] = centred<false>(xa);
                af[x][1] = centred<false>(xb);
                af[x][2] = centred<true>(xa);
                af[x][3] = centred<true>(xb);
              }
#pragma unroll
              for (int b = 0; b < C::RB; ++b) {
                if constexpr (NB == 1) {
                  const uint2 q = reinterpret_cast<const uint2 *>(qsrc)[kb * 32 + lane];
                  mma16816(acc[0][0], af[0], q.x, q.y);
                  mma16816(acc[1][0], af[1], q.x, q.y);
                } else {
                  const uint4 q = reinterpret_cast<const uint4 *>(qsrc)[(b * C::KB + kb) * 32 + lane];
                  mma16816(acc[0][b], af[0], q.x, q.y);
                  mma16816(acc[1][b], af[1], q.x, q.y);
                  mma16816(acc[0][b], af[0], q.z, q.w);
                  mma16816(acc[1][b], af[1], q.z, q.w);
                }
              }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint8_t *mk = kt + x * C::TB + 16 * C::CB + 4 * gg;
              const uint32_t mA = *reinterpret_cast<const uint32_t *>(mk + tA * 4 * NG);
              const uint32_t mB = *reinterpret_cast<const uint32_t *>(mk + tB * 4 * NG);
              const float sA = half_lo(mA), sB = half_lo(mB), zA = zero8(mA), zB = zero8(mB);
#pragma unroll
              for (int i = 0; i < R; ++i) {
                const float cA = NB == 1 ? acc[x][0][0] + acc[x][0][1] : acc[x][i / 2][i % 2];
                const float cB = NB == 1 ? acc[x][0][2] + acc[x][0][3] : acc[x][i / 2][2 + i % 2];
                const float qg = NG < 4 ? qsum[i][NG < 4 ? gg : 0] : qx[COLS + row_of(i) * NG + gg];
                sc[x][i][0] = fmaf(sA, cA, fmaf(zA, qg, sc[x][i][0]));
                sc[x][i][1] = fmaf(sB, cB, fmaf(zB, qg, sc[x][i][1]));
              }
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
        const bool all = got == 3 && t0 >= s.all_lo && t0 <= s.all_hi - kChunkTok;
        if (!all) {
          int2 lim[R];
#pragma unroll
          for (int i = 0; i < R; ++i) {
            lim[i] = make_int2(0, 0);
            if (uint32_t(row_of(i)) < s.nc) key_range(a, s.rs, (s.c0 + row_of(i)) / a.qpk, lim[i].x, lim[i].y);
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int32_t a0 = t0 + x * kTileTok + tA, b0 = t0 + x * kTileTok + tB;
            const bool there = (got >> x) & 1u;
#pragma unroll
            for (int i = 0; i < R; ++i) {
              if (!there || a0 < lim[i].x || a0 >= lim[i].y) sc[x][i][0] = -INFINITY;
              if (!there || b0 < lim[i].x || b0 >= lim[i].y) sc[x][i][1] = -INFINITY;
            }
            // A value whose scale or zero is not finite: the rows that see the key get
            // NaN through their sums of zeros (one group's are enough: the inverse transform
            // mixes all channels), the others (and slots that no row sees, which may
            // hold anything) weigh it 0. Scores and the log-sum-exp do not depend on values.
            bool odd_a = false, odd_b = false;
#pragma unroll
            for (int gg = 0; gg < NG; ++gg) {
              odd_a |= not_finite(vA[x][gg]);
              odd_b |= not_finite(vB[x][gg]);
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
              const bool sees = (odd_a && sc[x][i][0] != -INFINITY) || (odd_b && sc[x][i][1] != -INFINITY);
              if (sees) z[i][0] = __uint_as_float(0x7FFFFFFFu);
            }
            // (slots that no row sees must not widen the range of scales either)
            const bool no_a = odd_a || a0 < s.any_lo || a0 >= s.any_hi;
            const bool no_b = odd_b || b0 < s.any_lo || b0 >= s.any_hi;
#pragma unroll
            for (int gg = 0; gg < NG; ++gg) {
              vA[x][gg] = no_a ? 0u : vA[x][gg];
              vB[x][gg] = no_b ? 0u : vB[x][gg];
            }
          }
        }
        // Could a weight pass its range?
        float smax = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int gg = 0; gg < NG; ++gg)
            smax = fmaxf(smax, fmaxf(fabsf(half_lo(vA[x][gg])), fabsf(half_lo(vB[x][gg]))));
        const float room = kWeightMost - 1.f - log2_floor(__float_as_uint(smax));
        bool raise = false;
        float top[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
          top[i] = fmaxf(fmaxf(sc[0][i][0], sc[0][i][1]), fmaxf(sc[1][i][0], sc[1][i][1]));
          raise |= fmaf(top[i], fc[i], nm[i]) > fminf(lim[i], room);
        }
        if (__any_sync(0xFFFFFFFFu, raise)) {
          float fac[R];
          // The largest and the smallest scale: where they are alike, the largest score with the
          // largest scale will do for the largest weight.
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) smax = fmaxf(smax, __shfl_xor_sync(0xFFFFFFFFu, smax, o));
          uint32_t low = ~0u;
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int gg = 0; gg < NG; ++gg)
              low = min(low, min(vA[x][gg] & 0x7FFFu, vB[x][gg] & 0x7FFFu));
          low = __reduce_min_sync(0xFFFFFFFFu, low);
          const float e_top = log2_floor(__float_as_uint(fminf(smax, 65504.f)));
          const bool look = e_top - log2_floor(__float_as_uint(half_lo(low))) > 3.f;
#pragma unroll
          for (int i = 0; i < R; ++i) {
            float x = top[i];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
            x *= fc[i];
            float w = x + e_top + 1.f;
            if (look) {
              float ps = 0.f;
#pragma unroll
              for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  float big = 0.f;
#pragma unroll
                  for (int gg = 0; gg < NG; ++gg) big = fmaxf(big, fabsf(half_lo(y ? vB[t][gg] : vA[t][gg])));
                  ps = fmaxf(ps, big * ex2(fmaf(sc[t][i][y], fc[i], -x)));
                }
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) ps = fmaxf(ps, __shfl_xor_sync(0xFFFFFFFFu, ps, o));
              w = x + lg2(ps);
            }
            fac[i] = 1.f;
            if (x > -INFINITY) {
              const bool first = lim[i] == -INFINITY;
              const float n = row_factor(nm[i], x, w, first);
              if (!first) fac[i] = ex2(n - nm[i]);
              nm[i] = n;
              lim[i] = kPMost;
            }
            ls[i] *= fac[i];
#pragma unroll
            for (int gg = 0; gg < NG; ++gg) z[i][gg] *= fac[i];
          }
#pragma unroll
          for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
            for (int b = 0; b < C::RB; ++b) {
              const float fa = fac[NB == 1 ? 0 : 2 * b], fb = fac[NB == 1 ? 0 : 2 * b + 1];
              oacc[mt][b][0] *= fa, oacc[mt][b][1] *= fb;
              oacc[mt][b][2] *= fa, oacc[mt][b][3] *= fb;
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float p[R][2];
#pragma unroll
          for (int i = 0; i < R; ++i) {
            p[i][0] = ex2(fmaf(sc[x][i][0], fc[i], nm[i]));
            p[i][1] = ex2(fmaf(sc[x][i][1], fc[i], nm[i]));
            ls[i] += p[i][0] + p[i][1];
          }
          // weights of the value product per group, as its fragments
          uint32_t pf[NG][C::RB][2];
#pragma unroll
          for (int gg = 0; gg < NG; ++gg) {
            const float sA = half_lo(vA[x][gg]), sB = half_lo(vB[x][gg]);
            const float zA = zero8(vA[x][gg]), zB = zero8(vB[x][gg]);
            float w[R][2];
#pragma unroll
            for (int i = 0; i < R; ++i) {
              w[i][0] = p[i][0] * sA;
              w[i][1] = p[i][1] * sB;
              z[i][gg] = fmaf(p[i][0], zA, fmaf(p[i][1], zB, z[i][gg]));
            }
#pragma unroll
            for (int b = 0; b < C::RB; ++b)
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                if constexpr (NB == 1) {
                  float vh, vl;
                  split_f16(w[0][q], vh, vl);
                  pf[gg][0][q] = movmatrix(f16x2(vh, vl));
                } else {
                  pf[gg][b][q] = movmatrix(f16x2(w[2 * b][q], w[2 * b + 1][q]));
                }
              }
          }
          const uint8_t *src = vt + x * C::TB + gq * (D / 16);
          uint32_t v0[C::W / 2], v1[C::W / 2], v2[C::W / 2], v3[C::W / 2];
          load_words<C::W / 2>(src + ta * C::CB, v0);
          load_words<C::W / 2>(src + tb * C::CB, v1);
          load_words<C::W / 2>(src + (ta + 8) * C::CB, v2);
          load_words<C::W / 2>(src + (tb + 8) * C::CB, v3);
#pragma unroll
          for (int q = 0; q < C::W / 2; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // 32-channel block 2 q + h
              const uint32_t u = __byte_perm(v0[q], v1[q], h ? 0x7632 : 0x5410);
              const uint32_t v = __byte_perm(v2[q], v3[q], h ? 0x7632 : 0x5410);
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint32_t af[4] = {centred<false>(u >> (8 * y)), centred<true>(u >> (8 * y)),
                                        centred<false>(v >> (8 * y)), centred<true>(v >> (8 * y))};
                const int blk = 2 * q + h, mt = 2 * blk + y;
#pragma unroll
                for (int b = 0; b < C::RB; ++b)
                  mma16816(oacc[mt][b], af, pf[blk * 32 / G][b][0], pf[blk * 32 / G][b][1]);
              }
            }
        }
      }
      __syncwarp();  // every lane has read the stage before it is filled again
      if (asked < mine) ask();
      else cp_async_commit();
    }

    // ---- the segment's record
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        ls[i] += __shfl_xor_sync(0xFFFFFFFFu, ls[i], o);
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) z[i][gg] += __shfl_xor_sync(0xFFFFFFFFu, z[i][gg], o);
      }
    }
    constexpr float up = 8.f;
    // channels 32 blk + 4 gq .. + 3 of row row_of(i)
    auto out4 = [&](int blk, int i) {
      const float zz = 8.f * z[i][blk * 32 / G];
      const auto &e = oacc[2 * blk][i / C::LR], &o = oacc[2 * blk + 1][i / C::LR];
      if constexpr (NB == 1)
        return make_float4(fmaf(e[0] + e[1], up, zz), fmaf(e[2] + e[3], up, zz),
                           fmaf(o[0] + o[1], up, zz), fmaf(o[2] + o[3], up, zz));
      else
        return make_float4(fmaf(e[i % 2], up, zz), fmaf(e[2 + i % 2], up, zz),
                           fmaf(o[i % 2], up, zz), fmaf(o[2 + i % 2], up, zz));
    };
    if (!one_unit) {
      float *rec = a.rec + (s.unit + g) * uint64_t(COLS * (4 + D));
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const uint32_t row = uint32_t(row_of(i));
        if (row >= s.nc) continue;
        if (gq == 0)
          *reinterpret_cast<float2 *>(rec + row * (4 + D)) =
              make_float2(lim[i] == -INFINITY ? -INFINITY : -nm[i], ls[i]);
#pragma unroll
        for (int blk = 0; blk < C::W; ++blk)
          *reinterpret_cast<float4 *>(rec + row * (4 + D) + 4 + 32 * blk + 4 * gq) = out4(blk, i);
      }
      continue;
    }
    // the CTA's warps, in their order
    float *part = reinterpret_cast<float *>(smem);
    float2 *ml = reinterpret_cast<float2 *>(smem + C::ml);
    float *rec = a.rec + (s.unit + uint64_t(blockIdx.x) * CW) * uint64_t(COLS * (4 + D));
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (gq == 0)
        ml[warp * COLS + row_of(i)] = make_float2(lim[i] == -INFINITY ? -INFINITY : -nm[i], ls[i]);
#pragma unroll
    for (int c0 = 0; c0 < COLS; c0 += C::MC) {
      __syncthreads();  // the ring, and the rows before, are read
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int row = row_of(i) - c0;
        if (row < 0 || row >= C::MC) continue;
#pragma unroll
        for (int blk = 0; blk < C::W; ++blk)
          *reinterpret_cast<float4 *>(part + (size_t(warp) * C::MC + row) * D + 32 * blk + 4 * gq) =
              out4(blk, i);
      }
      __syncthreads();
      const uint32_t rows = s.nc > uint32_t(c0) ? min(s.nc - c0, uint32_t(C::MC)) : 0;
      for (uint32_t i = tid; i < rows * D; i += C::THREADS) {
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
    return;
  } while (f < f_end);
}

// A row's records: one per warp that has some of the unit's chunks, one only for a CTA
// whose share lies in the unit (its first warp's).
template <int C_, int CW>
struct DecodeRecords {
  static constexpr int COLS = C_;
  static constexpr bool kWide = true;
  uint64_t unit = 0;
  uint32_t row = 0, nrec = 0, n0 = 0, s0 = 0, b0 = 0, b1 = 0;
  __device__ __forceinline__ DecodeRecords(const CacheAttnArgs &a, uint32_t grid, const ReqShape &q,
                                           uint32_t l, uint32_t h, uint32_t r, uint32_t row_) {
    const KeyChunks kc = key_chunks(a, q);
    if (kc.count == 0) return;
    const uint32_t n = a.n_req, H = a.c.heads, work = unit_work(kc);
    const uint64_t lh = uint64_t(l) * H + h, per_lh = a.wpre[n], total = per_lh * H * a.c.layers;
    const uint64_t share = work_per_warp(total, grid * CW), cta = share * CW;
    // the unit's work [u0, u1), its chunks from u0 + kCaLead; the warps that have them
    const uint32_t block = row_ / COLS;
    const uint64_t u0 = lh * per_lh + a.wpre[r] + uint64_t(block) * work, u1 = u0 + work;
    const uint32_t g0 = uint32_t(div64(u0 + kCaLead, share)), g1 = uint32_t(div64(u1 - 1, share));
    unit = (lh * n + r) * a.row_blocks + block;
    row = row_ - block * COLS;
    b0 = g0 / CW;
    b1 = g1 / CW;
    const bool m0 = uint64_t(b0) * cta >= u0 && min(total, (uint64_t(b0) + 1) * cta) <= u1;
    const bool m1 = uint64_t(b1) * cta >= u0 && min(total, (uint64_t(b1) + 1) * cta) <= u1;
    n0 = m0 ? 1 : min(g1, b0 * CW + CW - 1) - g0 + 1;  // of the first CTA
    nrec = n0 + (b1 > b0 ? (b1 - b0 - 1) + (m1 ? 1 : g1 - b1 * CW + 1) : 0);
    s0 = m0 ? b0 * CW : g0;
  }
  __device__ __forceinline__ uint32_t id(uint32_t k) const {
    if (k < n0) return s0 + k;
    k -= n0;
    return k < b1 - b0 - 1 ? (b0 + 1 + k) * CW : b1 * CW + (k - (b1 - b0 - 1));
  }
};

template <int D, int G, int NB>
cudaError_t cache_attend_t(int dtype, const CacheAttnArgs &a, int sms, cudaStream_t st) {
  using C = CaCfg<D, G, NB>;
  auto k = cache_attend_kernel<D, G, NB>;
  struct Tag {};
  cudaError_t e = prepare<Tag>(k, C::bytes(KVC_MAX_REQUESTS));
  if (e != cudaSuccess) return e;
  static_assert(C::CTAS * (C::bytes(KVC_MAX_REQUESTS) + 1024) <= 227 * 1024, "CTAs per SM");
  const uint32_t most = kCacheWarpsMax / C::CW, want = uint32_t(sms) * C::CTAS;
  const uint32_t grid = want < most ? want : most;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.stream = st;
  const uint64_t units = uint64_t(a.c.layers) * a.c.heads * a.n_req * a.row_blocks;
  cache_attend_prep_kernel<D, G, NB><<<unsigned(units + 1), kCaPrepWarps * 32, 0, st>>>(a, dtype);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::bytes(a.n_req);
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k, a);
  if (e != cudaSuccess) return e;
  // one warp per row where units are as many as CTAs (a row then has one or two
  // records), eight where a unit is spread over many CTAs
  return launch_combine<D, DecodeRecords<C::COLS, C::CW>>(dtype, units * 4 < grid, a, grid, st);
}

template <int D, int G>
cudaError_t cache_attend_g(int dtype, const CacheAttnArgs &a, int sms, cudaStream_t st) {
  const uint64_t rows = uint64_t(a.max_q) * a.qpk;
  if (rows <= 4) return cache_attend_t<D, G, 1>(dtype, a, sms, st);
  if (rows <= 8) return cache_attend_t<D, G, 2>(dtype, a, sms, st);
  return cache_attend_t<D, G, 4>(dtype, a, sms, st);
}

}  // namespace kvc
