// Attention over the paged 4-bit cache for many query rows (pieces of prompts, drafted
// tokens of wide groups): the products on the 5th-generation tensor cores
// (tcgen05.mma, fp16 in, fp32 sums in tensor memory). Mathematics as in
// kvc_cache_attend.cuh; the codes stay exact in the score product.
//
// A unit is (layer, kv head, block of 128 query rows of a request: row = query *
// q_per_kv + head), its keys are tiles of NK = 128 / (groups per vector). Per tile:
//   S_g = (Q hi + Q lo)_g (n - 8)_g^T   a 128 x NK accumulator for each group g, NG of
//         them in 128 columns: scores are s_g S_g + (z + 8 s)_g sum(Q_g), which keeps
//         codes and queries (22 bits) exact where keys rounded to fp16 would not be;
//   P     = softmax weights in fp16, written to tensor memory as the next product's
//         operand;
//   O    += P V, V dequantised to fp16 (rounded once, as P is): 128 x D.
// Floor per 128 x 128 tile pair at d = 128: 3 x 512 cycles of the tensor cores (hi and
// lo parts, values).
//
// Warps 0..7: softmax. Warp w has rows 32 (w % 4) .. + 31 (a thread per row, as tensor
// memory is read) and half w / 4 of the tile's keys; the halves' maxima meet in
// shared memory. Thread 0 starts the products: tile j + 2's scores and tile j's
// values once tile j's weights are written, so that the tensor cores work on the
// next tile's scores during a softmax. Warps 8..11: unpack the tiles, two ahead.
// Work is shared out as in kvc_cache_attend.cuh, a share per CTA (one per SM).
//
// Shared memory, 128-byte swizzle (16-byte piece c of row r at c ^ (r & 7)):
//   Q: hi, lo; 64-channel slabs of 128 rows x 128 bytes (K-major)
//   K: 64-channel slabs of NK rows x 128 bytes (K-major), V: the same (N-major: a row
//   is a token, its channels are the product's columns), two buffers each.
// Eight codes of a word come apart as (0, 4), (1, 5), (2, 6), (3, 7): channels of Q
// follow that order, and output columns are put in order when they are written.
#pragma once

#include "kvc_cache_combine.cuh"

namespace kvc {

constexpr int kPfRows = 128;
constexpr int kPfSoft = 256, kPfUnpack = 128, kPfThreads = kPfSoft + kPfUnpack;
constexpr uint32_t kPfLead = 3;  // a segment's fixed work, in tiles

template <int D, int G>
struct PfCfg {
  static constexpr int NG = D / G, NK = 128 / NG, SL = D / 64, W = D / 32;
  static constexpr uint32_t TB = cache_tile_bytes(D, G), CB = cache_code_bytes(D);
  static constexpr uint32_t QPART = SL * kPfRows * 128, KBUF = SL * NK * 128;
  static constexpr int MW = 2 * NG + 2;  // words of a key's numbers: s, z + 8 s; 2^e, bias
  static constexpr size_t q = 0;
  static constexpr size_t k = q + 2 * QPART;
  static constexpr size_t v = k + 2 * KBUF;
  static constexpr size_t meta = v + 2 * KBUF;
  static constexpr size_t fc = meta + 2 * size_t(MW) * NK * 4;
  static constexpr size_t qs = fc + kPfRows * 4;
  static constexpr size_t mx = qs + size_t(NG) * kPfRows * 4;
  static constexpr size_t wmax = mx + 2 * 2 * kPfRows * 4;  // [buffer][unpacking warp]
  static constexpr size_t wodd = wmax + 2 * 4 * 4;
  static constexpr size_t bars = wodd + 2 * 4 * 4;          // full, scores, values: two each
  static constexpr size_t ctl = bars + 6 * 8;               // tensor memory, dead
  static constexpr size_t bytes = ctl + 16;
  // columns of tensor memory: scores 2 x 128, weights 2 x 64, output
  static constexpr uint32_t tS = 0, tP = 256, tO = 384;
  static_assert(bars % 8 == 0 && fc % 16 == 0 && bytes + 1024 <= 227 * 1024, "shared memory");
};

// ------------------------------------------------------------- tcgen05 --
__device__ __forceinline__ void tm_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tm_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tm_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tm_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// 16 columns of this warp's 32 lanes. The values may be used after tm_wait_ld and
// tm_loaded (which keeps the compiler from using them earlier).
__device__ __forceinline__ void tm_ld16(uint32_t addr, float *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
        "=f"(r[14]), "=f"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tm_loaded16(float *r) {
  asm volatile(""
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]),
                 "+f"(r[6]), "+f"(r[7]), "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]),
                 "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]));
}
__device__ __forceinline__ void tm_st16(uint32_t addr, const float *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]),
      "f"(r[8]), "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15])
      : "memory");
}
__device__ __forceinline__ void tm_st8(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
// Shared-memory operand, 128-byte swizzle: start, and the strides between 64-element
// blocks of the row dimension (only where that is contiguous) and between groups of 8
// rows, in bytes.
__device__ __forceinline__ uint64_t tm_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return uint64_t((addr >> 4) & 0x3FFFu) | (uint64_t(lbo >> 4) << 16) | (uint64_t(sbo >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// fp16 x fp16 -> fp32, 128 x n; B's contiguous dimension is n (b_n) or k.
__device__ constexpr uint32_t tm_idesc(int n, bool b_n) {
  return (1u << 4) | (b_n ? 1u << 16 : 0u) | (uint32_t(n / 8) << 17) | (uint32_t(kPfRows / 16) << 24);
}
__device__ __forceinline__ void tm_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void tm_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          uint32_t add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void tm_commit(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}

// Bounded wait for the phase with the given parity; a wait that runs out marks the
// CTA (*dead), whose other waits then end at once.
__device__ __forceinline__ void pf_wait(uint64_t *bar, uint32_t parity, volatile uint32_t *dead,
                                        uint32_t *status) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = globaltimer();
  for (uint32_t i = 1; i < kWaitIters; ++i) {
    if (mbar_try_wait(bar, parity)) return;
    if ((i & 15u) == 0 && (*dead || globaltimer() - t0 > kWaitNs)) break;
  }
  *dead = 1;
  if (status) set_status(status, KVC_ERR_TIMEOUT);
}

// Blocks of 128 query rows are numbered so that no request has to know the others: the
// first of request r is floor(q0 q_per_kv / 128) + r, which leaves each its own numbers
// below max_blocks.
__device__ __forceinline__ uint32_t first_block(const CacheAttnArgs &a, uint32_t q0, uint32_t r) {
  return uint32_t(uint64_t(q0) * a.qpk / kPfRows) + r;
}

// First kernel, one CTA: the requests' shapes; each block's request, first row, first
// key tile and tiles; prefixes of the blocks' work (per layer and head).
template <int NK>
__global__ void __launch_bounds__(1024) cache_prefill_prep_kernel(const __grid_constant__ CacheAttnArgs a) {
  __shared__ uint64_t red[32];
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.n_req;
  for (uint32_t r = tid; r < n; r += 1024) {
    bool ok;
    const ReqShape s = read_request(a, r, ok);
    if (!ok && a.status) set_status(a.status, KVC_ERR_CORRUPT);
    a.shapes[r] = make_uint4(s.nq, s.q0, s.len, 0);
  }
  const uint32_t nb = a.max_blocks, per = (nb + 1023) / 1024;
  const uint32_t b0 = min(nb, tid * per), b1 = min(nb, b0 + per);
  uint64_t w = 0;
  for (uint32_t b = b0; b < b1; ++b) {
    uint32_t lo = 0, hi = n - 1;  // the last request whose first block is not past b
    while (lo < hi) {
      const uint32_t mid = (lo + hi + 1) >> 1;
      const uint32_t q0 = a.q_starts ? uint32_t(max(0, __ldg(a.q_starts + mid))) : mid;
      if (first_block(a, q0, mid) <= b) lo = mid;
      else hi = mid - 1;
    }
    bool ok;
    const ReqShape s = read_request(a, lo, ok);
    const uint32_t fb = first_block(a, s.q0, lo), rows = s.nq * a.qpk;
    uint4 info = make_uint4(lo, 0, 0, 0);
    if (ok && b >= fb && uint64_t(b - fb) * kPfRows < rows) {
      info.y = (b - fb) * kPfRows;
      int32_t k0, k1, x;
      key_range(a, s, info.y / a.qpk, k0, x);
      key_range(a, s, (min(info.y + kPfRows, rows) - 1) / a.qpk, x, k1);
      info.z = uint32_t(k0) / NK;
      info.w = k1 > k0 ? (uint32_t(k1) + NK - 1) / NK - info.z : 0;
    }
    a.blk[b] = info;
    w += info.w ? info.w + kPfLead : 0;
  }
  uint64_t wi = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t x = __shfl_up_sync(0xFFFFFFFFu, wi, o);
    if (int(lane) >= o) wi += x;
  }
  if (lane == 31) red[warp] = wi;
  __syncthreads();
  uint64_t base = wi - w;
  for (uint32_t k = 0; k < warp; ++k) base += red[k];
  for (uint32_t b = b0; b < b1; ++b) {
    a.wpre[b] = base;
    const uint32_t t = a.blk[b].w;
    base += t ? t + kPfLead : 0;
  }
  if (tid == 1023) a.wpre[nb] = base;
}

// A CTA's part of a unit.
struct PfSegment {
  uint32_t l, h, r, c0, nc;      // layer, kv head, request; the block's rows
  uint32_t first, tiles;
  uint64_t unit;
  int32_t any_lo, any_hi, all_lo, all_hi;  // keys that some row sees, that every row sees
  ReqShape rs;
};
__device__ __forceinline__ PfSegment pf_segment_at(const CacheAttnArgs &a, uint64_t f_end,
                                                   uint64_t &f) {
  const uint32_t nb = a.max_blocks;
  const uint64_t per_lh = a.wpre[nb], lh = div64(f, per_lh), in_lh = f - lh * per_lh;
  PfSegment s;
  s.l = uint32_t(lh) / a.c.heads;
  s.h = uint32_t(lh) - s.l * a.c.heads;
  const uint32_t b = last_with(nb, [&](uint32_t x) { return a.wpre[x] <= in_lh; });
  const uint4 info = a.blk[b];
  s.r = info.x;
  s.c0 = info.y;
  s.rs = request_shape(a, s.r);
  s.nc = min(uint32_t(kPfRows), s.rs.nq * a.qpk - s.c0);
  s.unit = lh * nb + b;
  const uint32_t work = info.w + kPfLead, at = uint32_t(in_lh - a.wpre[b]);
  const uint32_t end = uint32_t(min(uint64_t(work), at + (f_end - f)));
  const uint32_t c_at = at > kPfLead ? at - kPfLead : 0, c_end = end > kPfLead ? end - kPfLead : 0;
  s.first = info.z + c_at;
  s.tiles = c_end - c_at;
  f += end - at;
  key_range(a, s.rs, s.c0 / a.qpk, s.any_lo, s.all_hi);
  key_range(a, s.rs, (s.c0 + s.nc - 1) / a.qpk, s.all_lo, s.any_hi);
  return s;
}

// Unpacking warps: tile after tile of every segment into the two buffers.
template <int D, int G>
__device__ __forceinline__ void pf_unpack(const CacheAttnArgs &a, uint8_t *smem, uint64_t f,
                                          uint64_t f_end) {
  using C = PfCfg<D, G>;
  constexpr int NG = C::NG, NK = C::NK, W = C::W, RX = NK / 32;
  const uint32_t t = threadIdx.x - kPfSoft, lane = t & 31, warp = t >> 5, p = t & 3, r0 = t >> 2;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::bars), *pv = full + 4;
  volatile uint32_t *dead = reinterpret_cast<uint32_t *>(smem + C::ctl) + 1;
  uint32_t j = 0;
  while (f < f_end) {
    const PfSegment s = pf_segment_at(a, f_end, f);
    const uint8_t *base = a.c.pool + int64_t(s.l) * a.c.s_l + int64_t(s.h) * a.c.s_h;
    const int32_t *table = a.page_table + int64_t(s.r) * a.pt_stride;
    uint32_t k[RX][W], v[RX][W], mk[RX][NG], mv[RX][NG];
    bool in[RX];
    auto load = [&](uint32_t tile) {
#pragma unroll
      for (int x = 0; x < RX; ++x) {
        const int32_t tok = int32_t(tile * NK + r0 + 32 * x);
        in[x] = tok >= s.any_lo && tok < s.any_hi;
        const uint8_t *src = nullptr;
        if (in[x]) {
          const uint32_t kt = uint32_t(tok) / kTileTok, pi = fdiv(a.tpp, kt);
          const int32_t pg = __ldg(table + pi);
          in[x] = pg >= 0 && uint32_t(pg) < a.c.num_pages;
          if (in[x])
            src = base + int64_t(pg) * a.c.s_p + int64_t(kt - pi * a.tpp.d) * C::TB;
          else if (a.status)
            set_status(a.status, KVC_ERR_CORRUPT);
        }
        const uint32_t ln = uint32_t(tok) % kTileTok;
#pragma unroll
        for (int i = 0; i < W; ++i) k[x][i] = v[x][i] = 0x88888888u;  // n - 8 = 0
#pragma unroll
        for (int g = 0; g < NG; ++g) mk[x][g] = mv[x][g] = 0;
        if (src) {
          const uint8_t *kr = src + ln * C::CB + 4 * W * p, *vr = kr + a.c.s_kv;
          if constexpr (W == 4) {
            const uint4 u = __ldg(reinterpret_cast<const uint4 *>(kr));
            const uint4 y = __ldg(reinterpret_cast<const uint4 *>(vr));
            k[x][0] = u.x, k[x][1] = u.y, k[x][2] = u.z, k[x][3] = u.w;
            v[x][0] = y.x, v[x][1] = y.y, v[x][2] = y.z, v[x][3] = y.w;
          } else {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(kr));
            const uint2 y = __ldg(reinterpret_cast<const uint2 *>(vr));
            k[x][0] = u.x, k[x][1] = u.y;
            v[x][0] = y.x, v[x][1] = y.y;
          }
          const uint32_t *m = reinterpret_cast<const uint32_t *>(src + kTileTok * C::CB) + ln * NG;
          const uint32_t *n = reinterpret_cast<const uint32_t *>(reinterpret_cast<const uint8_t *>(m) + a.c.s_kv);
#pragma unroll
          for (int g = 0; g < NG; ++g) mk[x][g] = __ldg(m + g), mv[x][g] = __ldg(n + g);
        }
      }
    };
    if (s.tiles) load(s.first);
    for (uint32_t i = 0; i < s.tiles; ++i, ++j) {
      const uint32_t buf = j & 1;
      if (j >= 2) pf_wait(pv + buf, ((j >> 1) - 1) & 1u, dead, a.status);
      uint8_t *kb = smem + C::k + buf * C::KBUF, *vb = smem + C::v + buf * C::KBUF;
      float *meta = reinterpret_cast<float *>(smem + C::meta) + buf * C::MW * NK;
      uint32_t most = 0;
      bool odd = false;
#pragma unroll
      for (int x = 0; x < RX; ++x) {
        const uint32_t row = r0 + 32 * x, sw = row & 7;
        uint8_t *kr = kb + row * 128, *vr = vb + row * 128;
#pragma unroll
        for (int b = 0; b < W; ++b) {
          const uint32_t w = k[x][b];
          *reinterpret_cast<uint4 *>(kr + (b >> 1) * NK * 128 + (((4 * (b & 1) + p) ^ sw) << 4)) =
              make_uint4(centred<false>(w), centred<true>(w), centred<false>(w >> 8),
                         centred<true>(w >> 8));
        }
        // values x 2^-e, e from the largest |z + 8 s| + 8 |s|
        bool bad = false;
        float bound = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          bad |= not_finite(mv[x][g]);
          bound = fmaxf(bound, fabsf(zero8(mv[x][g])) + 8.f * fabsf(half_lo(mv[x][g])));
        }
        const uint32_t ex = (__float_as_uint(bound) >> 23) & 255u;
        const bool none = bad || bound == 0.f;
        const float scale = none ? 1.f : __uint_as_float(ex << 23);
        const float inv = none ? (bad ? 0.f : 1.f) : __uint_as_float((254u - ex) << 23);
#pragma unroll
        for (int q = 0; q < W; ++q) {
          constexpr int B = D / 32;
          const int wj = B * int(p) + q;               // stored word: halves of blocks a, a + 1
          const int ga = ((2 * q) % B) * 32 / G, gb = ((2 * q) % B + 1) * 32 / G;
          const uint32_t ma = bad ? 0u : mv[x][ga], mb = bad ? 0u : mv[x][gb];
          const uint32_t s2 = f16x2(half_lo(ma) * inv, half_lo(mb) * inv);
          const uint32_t z2 = f16x2(zero8(ma) * inv, zero8(mb) * inv);
          const uint32_t w = v[x][q];
          auto deq = [&](uint32_t n) {
            uint32_t d;
            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(n), "r"(s2), "r"(z2));
            return d;
          };
          *reinterpret_cast<uint4 *>(vr + (wj >> 3) * NK * 128 + (((wj & 7) ^ sw) << 4)) =
              make_uint4(deq(centred<false>(w)), deq(centred<true>(w)), deq(centred<false>(w >> 8)),
                         deq(centred<true>(w >> 8)));
        }
        if (int(p) < NG) {
          uint32_t m = mk[x][0];
#pragma unroll
          for (int g = 1; g < NG; ++g) m = int(p) == g ? mk[x][g] : m;
          meta[p * NK + row] = half_lo(m);
          meta[(NG + p) * NK + row] = zero8(m);
        }
        const float bias = !in[x] ? -INFINITY : bad ? __uint_as_float(0x7FFFFFFFu) : 0.f;
        if (p == 0) {
          meta[2 * NG * NK + row] = scale;
          meta[(2 * NG + 1) * NK + row] = bias;
        }
        odd |= !in[x] || bad;
        most = max(most, none ? 0u : __float_as_uint(scale));
      }
      most = __reduce_max_sync(0xFFFFFFFFu, most);
      odd = __any_sync(0xFFFFFFFFu, odd);
      if (lane == 0) {
        reinterpret_cast<uint32_t *>(smem + C::wmax)[buf * 4 + warp] = most;
        reinterpret_cast<uint32_t *>(smem + C::wodd)[buf * 4 + warp] = odd;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + buf);
      if (i + 1 < s.tiles) load(s.first + i + 1);
    }
  }
}

template <int D, int G>
__global__ void __launch_bounds__(kPfThreads, 1)
    cache_prefill_kernel(const __grid_constant__ CacheAttnArgs a, const int dtype) {
  using C = PfCfg<D, G>;
  constexpr int NG = C::NG, NK = C::NK, W = C::W, KH = NK / 2;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::bars), *sready = full + 2, *pv = full + 4;
  uint32_t *ctl = reinterpret_cast<uint32_t *>(smem + C::ctl);
  volatile uint32_t *dead = ctl + 1;
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(ctl)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 32) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(full + i, 4);
      mbar_init(sready + i, 1);
      mbar_init(pv + i, 1);
    }
    mbar_fence_init();
    *dead = 0;
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tm = *ctl;
  grid_dependency_wait();  // the first kernel's prefixes and shapes
  const uint64_t total = a.wpre[a.max_blocks] * a.c.heads * a.c.layers;
  const uint64_t share = div64(total + gridDim.x - 1, gridDim.x);
  uint64_t f = uint64_t(blockIdx.x) * share;
  const uint64_t f_end = min(total, f + share);

  if (warp >= kPfSoft / 32) {
    pf_unpack<D, G>(a, smem, f, f_end);
  } else {
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t tl = tm + (uint32_t((warp & 3) * 32) << 16);  // this warp's lanes
    float *fcs = reinterpret_cast<float *>(smem + C::fc), *qss = reinterpret_cast<float *>(smem + C::qs);
    float *mxs = reinterpret_cast<float *>(smem + C::mx);
    const uint32_t q_s = smem_u32(smem + C::q);
    uint32_t j = 0;  // tiles so far

    auto scores = [&](uint32_t jj) {  // thread 0: S of tile jj
      const uint32_t buf = jj & 1, k_s = smem_u32(smem + C::k) + buf * C::KBUF;
      pf_wait(full + buf, (jj >> 1) & 1u, dead, a.status);
      tm_fence_after();
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int st = g * G / 16; st < (g + 1) * G / 16; ++st) {
            const uint32_t o = (st & 3) * 32;
            tm_mma(tm + C::tS + buf * 128 + g * NK,
                   tm_desc(q_s + part * C::QPART + (st >> 2) * kPfRows * 128 + o, 16, 1024),
                   tm_desc(k_s + (st >> 2) * NK * 128 + o, 16, 1024), tm_idesc(NK, false),
                   part != 0 || st != g * G / 16);
          }
      tm_commit(sready + buf);
    };

    while (f < f_end) {
      const PfSegment s = pf_segment_at(a, f_end, f);
      if (s.tiles == 0) continue;
      // ---- the block's queries: qt as hi and lo parts, factors, group sums
#pragma unroll 2
      for (int q = 0; q < kPfRows / 8; ++q) {
        const int rr = warp * (kPfRows / 8) + q;
        const bool live = uint32_t(rr) < s.nc;
        const uint32_t gr = s.c0 + (live ? rr : 0), qi = gr / a.qpk;
        const uint8_t *src = a.q + int64_t(s.l) * a.q_l + int64_t(s.rs.q0 + qi) * a.q_t +
                             int64_t(s.h * a.qpk + (gr - qi * a.qpk)) * a.q_h;
        uint16_t in[W];
#pragma unroll
        for (int c = 0; c < W; ++c)
          in[c] = live ? __ldg(reinterpret_cast<const uint16_t *>(src) + lane + 32 * c) : uint16_t(0);
        uint64_t w0 = a.c.w0, w1 = a.c.w1;
        if (a.c.vec_signs) {
          uint64_t st = a.c.seed + (uint64_t(s.l) * 2 * a.c.heads + s.h) * uint64_t(D / 64) *
                                       0x9E3779B97F4A7C15ull;
          w0 = splitmix64(st);
          if constexpr (D == 128) w1 = splitmix64(st);
        }
        float y[W];
#pragma unroll
        for (int c = 0; c < W; ++c) {
          const float x = dtype == KVC_BF16 ? __uint_as_float(uint32_t(in[c]) << 16)
                                            : __half2float(__ushort_as_half(in[c]));
          const uint32_t sg = uint32_t((c < 2 ? w0 : w1) >> (32 * (c & 1) + lane)) & 1u;
          y[c] = __uint_as_float(__float_as_uint(x) ^ (sg << 31));
        }
#pragma unroll
        for (int st = 1; st < 32; st <<= 1)
#pragma unroll
          for (int c = 0; c < W; ++c) {
            const float o = __shfl_xor_sync(0xFFFFFFFFu, y[c], st);
            y[c] = (lane & st) ? o - y[c] : y[c] + o;
          }
#pragma unroll
        for (int st = 1; st < W; st <<= 1)
#pragma unroll
          for (int c = 0; c < W; ++c)
            if ((c & st) == 0) {
              const float u = y[c], v = y[c + st];
              y[c] = u + v;
              y[c + st] = u - v;
            }
        float mx = 0.f, gs[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) gs[g] = 0.f;
#pragma unroll
        for (int c = 0; c < W; ++c) {
          y[c] *= a.scale;
          mx = fmaxf(mx, fabsf(y[c]));
          gs[c * 32 / G] += y[c];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
#pragma unroll
          for (int g = 0; g < NG; ++g) gs[g] += __shfl_xor_sync(0xFFFFFFFFu, gs[g], o);
        }
        const int e = int((__float_as_uint(mx) >> 23) & 255u) - 126;
        const bool fine = mx > 0.f && isfinite(mx) && e > -100;
        const float es = fine ? __uint_as_float(uint32_t(127 + 14 - e) << 23) : 1.f;
        if (lane == 0) {
          fcs[rr] = 8.f / es;
#pragma unroll
          for (int g = 0; g < NG; ++g) qss[g * kPfRows + rr] = gs[g] * es;
        }
        const int i = lane & 7, pos = i < 4 ? 2 * i : 2 * (i - 4) + 1;
#pragma unroll
        for (int c = 0; c < W; ++c) {
          float vh, vl;
          split_f16(y[c] * es, vh, vl);
          uint8_t *dst = smem + C::q + (c >> 1) * kPfRows * 128 + rr * 128 +
                         (((4 * (c & 1) + (lane >> 3)) ^ (rr & 7)) << 4) + 2 * pos;
          *reinterpret_cast<uint16_t *>(dst) = __half_as_ushort(__float2half_rn(vh));
          *reinterpret_cast<uint16_t *>(dst + C::QPART) = __half_as_ushort(__float2half_rn(vl));
        }
      }
      fence_proxy_async_smem();
      tm_fence_before();  // (the output of the segment before is read)
      named_bar_sync(1, kPfSoft);
      if (tid == 0) {
        scores(j);
        if (s.tiles > 1) scores(j + 1);
      }
      const float fc = fcs[row];
      float qsum[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) qsum[g] = qss[g * kPfRows + row];
      int32_t lo = 0, hi = 0;
      if (uint32_t(row) < s.nc) key_range(a, s.rs, (s.c0 + row) / a.qpk, lo, hi);
      // Running state as in kvc_cache_attend.cuh: nm = -m (base 2, and - log2 of the
      // values' common exponent: weights times 2^(a value's e) reach up to 2^15).
      float nm = 0.f, mt = 0.f, thr = -INFINITY, l = 0.f, lw = 0.f, v_most = 0.f;

      for (uint32_t i = 0; i < s.tiles; ++i, ++j) {
        const uint32_t buf = j & 1;
        const int32_t t0 = int32_t((s.first + i) * NK);
        pf_wait(full + buf, (j >> 1) & 1u, dead, a.status);  // the keys' numbers
        pf_wait(sready + buf, (j >> 1) & 1u, dead, a.status);
        tm_fence_after();
        __syncwarp();
        const float *meta = reinterpret_cast<const float *>(smem + C::meta) + buf * C::MW * NK + half * KH;
        float sc[KH];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float acc[KH];
#pragma unroll
          for (int x = 0; x < KH; x += 16)
            tm_ld16(tl + C::tS + buf * 128 + g * NK + half * KH + x, acc + x);
          tm_wait_ld();
#pragma unroll
          for (int x = 0; x < KH; x += 16) tm_loaded16(acc + x);
          const float2 q2 = make_float2(qsum[g], qsum[g]);
#pragma unroll
          for (int x = 0; x < KH; x += 4) {
            const float4 ks = *reinterpret_cast<const float4 *>(meta + g * NK + x);
            const float4 kz = *reinterpret_cast<const float4 *>(meta + (NG + g) * NK + x);
            float2 u = g == 0 ? mul2(make_float2(kz.x, kz.y), q2)
                              : fma2(make_float2(kz.x, kz.y), q2, make_float2(sc[x], sc[x + 1]));
            float2 v = g == 0 ? mul2(make_float2(kz.z, kz.w), q2)
                              : fma2(make_float2(kz.z, kz.w), q2, make_float2(sc[x + 2], sc[x + 3]));
            u = fma2(make_float2(ks.x, ks.y), make_float2(acc[x], acc[x + 1]), u);
            v = fma2(make_float2(ks.z, ks.w), make_float2(acc[x + 2], acc[x + 3]), v);
            sc[x] = u.x, sc[x + 1] = u.y, sc[x + 2] = v.x, sc[x + 3] = v.y;
          }
        }
        const uint4 odd = *reinterpret_cast<const uint4 *>(smem + C::wodd + buf * 16);
        if ((odd.x | odd.y | odd.z | odd.w) || t0 < s.all_lo || t0 + NK > s.all_hi) {
#pragma unroll
          for (int x = 0; x < KH; ++x) {
            const int32_t t = t0 + half * KH + x;
            sc[x] = t >= lo && t < hi ? sc[x] + meta[(2 * NG + 1) * NK + x] : -INFINITY;
          }
        }
        float top = sc[0];
#pragma unroll
        for (int x = 1; x < KH; ++x) top = fmaxf(top, sc[x]);
        float *mx = mxs + buf * 2 * kPfRows;
        mx[half * kPfRows + row] = top;
        named_bar_sync(1, kPfSoft);
        top = fmaxf(top, mx[(1 - half) * kPfRows + row]);
        const float4 wm = *reinterpret_cast<const float4 *>(smem + C::wmax + buf * 16);
        const float vm = fmaxf(fmaxf(wm.x, wm.y), fmaxf(wm.z, wm.w));
        if (__any_sync(0xFFFFFFFFu, top > thr) || vm > v_most) {
          float fac = 1.f;
          if (thr == -INFINITY) {  // nothing but NaN so far, if anything
            if (top > -INFINITY) mt = top * fc, thr = (mt + 8.f) / fc;
          } else if (top > thr) {
            const float x = top * fc;
            fac = ex2(mt - x);
            mt = x;
            thr = (x + 8.f) / fc;
          }
          if (vm > v_most) {  // bring vm * 2^lw to 2^5; up to 2^7 is let pass
            const int ex = int(__float_as_uint(vm) >> 23) - 127;
            const float nl = float(5 - ex);
            fac *= ex2(nl - lw);
            lw = nl;
            v_most = ex2(float(ex + 2));
          }
          nm = lw - mt;
          l *= fac;
          if (i > 0) {
            const uint32_t jp = j - 1;
            pf_wait(pv + (jp & 1), (jp >> 1) & 1u, dead, a.status);
            tm_fence_after();
            __syncwarp();
#pragma unroll
            for (int x = 0; x < D / 2; x += 16) {
              float o[16];
              tm_ld16(tl + C::tO + half * (D / 2) + x, o);
              tm_wait_ld();
              tm_loaded16(o);
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] *= fac;
              tm_st16(tl + C::tO + half * (D / 2) + x, o);
            }
            tm_wait_st();
          }
        }
        const float *vs = meta + 2 * NG * NK;
        const float2 f2 = make_float2(fc, fc), n2 = make_float2(nm, nm);
        float2 l2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int x = 0; x < KH; x += 16) {
          uint32_t pk[8];
#pragma unroll
          for (int y = 0; y < 16; y += 4) {
            const float4 sv = *reinterpret_cast<const float4 *>(vs + x + y);
            const float2 u = fma2(make_float2(sc[x + y], sc[x + y + 1]), f2, n2);
            const float2 v = fma2(make_float2(sc[x + y + 2], sc[x + y + 3]), f2, n2);
            const float2 pu = make_float2(ex2(u.x), ex2(u.y)), pw = make_float2(ex2(v.x), ex2(v.y));
            l2 = add2(l2, add2(pu, pw));
            const float2 wu = mul2(pu, make_float2(sv.x, sv.y)), ww = mul2(pw, make_float2(sv.z, sv.w));
            pk[y / 2] = f16x2(wu.x, wu.y);
            pk[y / 2 + 1] = f16x2(ww.x, ww.y);
          }
          tm_st8(tl + C::tP + buf * 64 + half * (KH / 2) + x / 2, pk);
        }
        l += l2.x + l2.y;
        tm_wait_st();
        tm_fence_before();
        named_bar_sync(2, kPfSoft);
        if (tid == 0) {
          tm_fence_after();
          const uint32_t v_s = smem_u32(smem + C::v) + buf * C::KBUF;
#pragma unroll
          for (int st = 0; st < NK / 16; ++st)
            tm_mma_ts(tm + C::tO, tm + C::tP + buf * 64 + st * 8,
                      tm_desc(v_s + st * 2048, NK * 128, 1024), tm_idesc(D, true), i != 0 || st != 0);
          tm_commit(pv + buf);
          if (i + 2 < s.tiles) scores(j + 2);
        }
        __syncwarp();
      }

      // ---- the segment's record
      pf_wait(pv + ((j - 1) & 1), ((j - 1) >> 1) & 1u, dead, a.status);
      tm_fence_after();
      __syncwarp();
      float *lx = mxs + half * kPfRows;  // (the last tile's maxima are read: barrier 2)
      lx[row] = l;
      named_bar_sync(1, kPfSoft);
      float *rec = a.rec + (s.unit + blockIdx.x) * uint64_t(kPfRows * (4 + D)) + row * (4 + D);
      const bool live = uint32_t(row) < s.nc;
      if (live && half == 0)
        *reinterpret_cast<float2 *>(rec) =
            make_float2(thr == -INFINITY ? -INFINITY : mt - lw, mxs[row] + mxs[kPfRows + row]);
#pragma unroll
      for (int x = 0; x < D / 2; x += 16) {
        float o[16];
        tm_ld16(tl + C::tO + half * (D / 2) + x, o);
        tm_wait_ld();
        tm_loaded16(o);
#pragma unroll
        for (int y = 0; y < 16; y += 8) {
          // columns of stored word wj: halves of its two 32-channel blocks
          const int wj = (half * (D / 2) + x + y) / 8, hs = 2 * wj;
          const int ch = 32 * (hs % W) + 4 * (hs / W);
          if (live) {
            *reinterpret_cast<float4 *>(rec + 4 + ch) =
                make_float4(8.f * o[y], 8.f * o[y + 2], 8.f * o[y + 4], 8.f * o[y + 6]);
            *reinterpret_cast<float4 *>(rec + 4 + ch + 32) =
                make_float4(8.f * o[y + 1], 8.f * o[y + 3], 8.f * o[y + 5], 8.f * o[y + 7]);
          }
        }
      }
      tm_fence_before();
      named_bar_sync(2, kPfSoft);  // the shared arrays are free for the next segment
    }
  }
  tm_fence_before();
  __syncthreads();
  if (warp == 0) {
    tm_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512u));
  }
}

// A row's records: one per CTA that has some of the block's tiles.
struct PrefillRecords {
  static constexpr int COLS = kPfRows;
  uint64_t unit = 0;
  uint32_t row = 0, nrec = 0, g0 = 0;
  __device__ __forceinline__ PrefillRecords(const CacheAttnArgs &a, uint32_t grid, const ReqShape &q,
                                            uint32_t l, uint32_t h, uint32_t r, uint32_t row_) {
    const uint32_t nb = a.max_blocks, b = first_block(a, q.q0, r) + row_ / kPfRows;
    const uint64_t per_lh = a.wpre[nb], total = per_lh * a.c.heads * a.c.layers;
    if (total == 0 || a.wpre[b + 1] == a.wpre[b]) return;
    const uint64_t share = div64(total + grid - 1, grid), lh = uint64_t(l) * a.c.heads + h;
    unit = lh * nb + b;
    row = row_ % kPfRows;
    g0 = uint32_t(div64(lh * per_lh + a.wpre[b] + kPfLead, share));
    nrec = uint32_t(div64(lh * per_lh + a.wpre[b + 1] - 1, share)) - g0 + 1;
  }
  __device__ __forceinline__ uint32_t id(uint32_t k) const { return g0 + k; }
};

template <int D, int G>
cudaError_t cache_prefill_t(int dtype, const CacheAttnArgs &a, int sms, cudaStream_t st) {
  using C = PfCfg<D, G>;
  auto k = cache_prefill_kernel<D, G>;
  struct Tag {};
  cudaError_t e = prepare<Tag>(k, C::bytes);
  if (e != cudaSuccess) return e;
  cache_prefill_prep_kernel<C::NK><<<1, 1024, 0, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const uint32_t grid = uint32_t(sms) < kCachePrefillCtas ? uint32_t(sms) : kCachePrefillCtas;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kPfThreads);
  cfg.dynamicSmemBytes = C::bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k, a, dtype);
  if (e != cudaSuccess) return e;
  return launch_combine<D, PrefillRecords>(dtype, false, a, grid, st);
}

}  // namespace kvc
