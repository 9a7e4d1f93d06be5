// Attention over the paged 4-bit cache for many query rows (pieces of prompts, drafted
// tokens of wide groups): the products on the 5th-generation tensor cores
// (tcgen05.mma, fp16 in, fp32 sums in tensor memory). Mathematics as in
// kvc_cache_attend.cuh; the codes stay exact in the score product.
//
// A unit is (layer, kv head, block of 128 query rows of a request: row = query *
// q_per_kv + head), its keys are tiles of NK = 64 (32 with four groups). Per tile:
//   S_g = (Q hi + Q lo)_g (n - 8)_g^T   a 128 x NK accumulator for each group g: scores
//         are s_g S_g + (z + 8 s)_g sum(Q_g), which keeps codes and queries (22 bits)
//         exact where keys rounded to fp16 would not be;
//   P     = softmax weights in fp16, written to tensor memory (over the scores) as the
//         next product's operand;
//   O    += P V, V dequantised to fp16 (rounded once, as P is): 128 x D. V = z + n s times
//         a power of two per key: z and s stay exact there, so one fused multiply-add
//         rounds. (With z + 8 s and n - 8 the sum was rounded before it: the same for all
//         channels of a group, which the inverse transform puts into one.)
// Floor per 128 x 64 tile pair at d = 128: 3 x 256 cycles of the tensor cores (hi and
// lo parts, values). Measured: 1024 queries x 32 heads over 9216 keys in 252 us at 1965 MHz
// (580 TFLOP/s of the two products counted once) and in 277 at the 1815 MHz at which the
// power cap holds a loop of such calls; 1660 cycles a tile, of which the
// tensor cores are active for 770. A softmax works for most of its two tiles' time (two
// softmax and two unpacking warps share an SM quarter's issue, 62% of it used), and
// shared memory serves 840 wavefronts and the products' operands a tile. With two groups
// 322 us, with four 469 us (two tiles' scores fit, and more fused multiplies).
//
// Warps 0..3 do the even tiles' softmax, 4..7 the odd ones', a thread per row with a
// maximum, a sum and an output accumulator of its own: the two never wait for each other,
// and one's exponentials run beside the other's products. Their results meet at a
// segment's end. Warps 8..11 unpack the even tiles, 12..15 the odd ones, up to four
// tiles ahead. Warps 16 and 17 start the products (PfIssue): from a softmax warp, a start
// that waits for the tensor cores' queue held up the whole block.
// Work is shared out as in kvc_cache_attend.cuh, a share per CTA (one per SM).
//
// Shared memory, 128-byte swizzle (16-byte piece c of row r at c ^ (r & 7)):
//   Q: hi, lo; 64-channel slabs of 128 rows x 128 bytes (K-major)
//   K: 64-channel slabs of NK rows x 128 bytes (K-major), V: the same (N-major: a row
//   is a token, its channels are the product's columns), four stages each.
// Eight codes of a word come apart as (0, 4), (1, 5), (2, 6), (3, 7): channels of Q
// follow that order, and output columns are put in order when they are written.
#pragma once

#include "kvc_cache_combine.cuh"

namespace kvc {

constexpr int kPfRows = 128;
constexpr int kPfSoft = 256, kPfUnpack = 256, kPfThreads = kPfSoft + kPfUnpack + 128;
// Registers: 640 threads start with 96 each; the softmax warps take 136, the unpacking
// ones keep 72 and the last four 64 (2 x 128 x (136 + 72) + 128 x 64 = 640 x 96).
constexpr int kPfSoftRegs = 136, kPfUnpackRegs = 72, kPfIssueRegs = 64;
constexpr uint32_t kPfStages = 4;
// A segment's fixed work (queries, first tiles, record) in tiles. 2048 queries over their
// own keys with 3, 8, 10, 16: 213, 176, 169, 169 us; 1024 over 9216: 257, 255, 255, 260.
constexpr uint32_t kPfLead = 10;

template <int D, int G>
struct PfCfg {
  static constexpr int NG = D / G, NK = NG == 4 ? 32 : 64, SL = D / 64, W = D / 32;
  static constexpr uint32_t TB = cache_tile_bytes(D, G), CB = cache_code_bytes(D);
  // queries of a block, in the workspace too: parts (then each row's factor, its sums)
  static constexpr uint32_t QPART = SL * kPfRows * 128, QB = 2 * QPART + kPfRows * 4 * (1 + NG), KBUF = SL * NK * 128;
  static constexpr int MW = 2 * NG + 2;  // words of a key's numbers: s, z + 8 s; 2^e, bias
  static constexpr size_t q = 0;
  static constexpr size_t k = q + 2 * QPART;
  static constexpr size_t v = k + kPfStages * KBUF;
  static constexpr size_t meta = v + kPfStages * KBUF;
  static constexpr size_t fin = meta + kPfStages * size_t(MW) * NK * 4;  // [softmax][row] maximum, sum
  static constexpr size_t taint = fin + 2 * kPfRows * 8;        // [softmax][row]
  static constexpr size_t wmax = taint + 2 * kPfRows * 4;       // [stage][unpacking warp]
  static constexpr size_t wodd = wmax + kPfStages * 4 * 4;
  // full and values (a stage), scores and weights (a tile's scores), queries copied, ready
  static constexpr size_t bars = wodd + kPfStages * 4 * 4;
  static constexpr size_t ctl = bars + (2 * kPfStages + 8) * 8;  // tensor memory, dead
  static constexpr size_t bytes = ctl + 16;
  // Columns of tensor memory: scores (and weights) of NS tiles, two outputs, and in what is
  // left the queries' hi parts, then the lo parts. With three tiles' scores a tile's are
  // computed during the softmax before it; queries there leave shared memory's bandwidth
  // to the keys (128 x 16 of them a product, twice the bytes of its keys).
  static constexpr uint32_t SW = NG * NK, NS = 3 * SW + 2 * D <= 512 ? 3 : 2;
  static constexpr uint32_t tS = 0, tO = NS * SW, tQ = tO + 2 * D;
  static constexpr bool QH = tQ + D / 2 <= 512, QL = tQ + D <= 512;
  static_assert(tQ <= 512, "tensor memory");
  static_assert(bars % 8 == 0 && fin % 16 == 0 && ctl % 8 == 0 && bytes + 1024 <= 227 * 1024, "shared memory");
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
// One lane of a converged warp: the compiler then knows that one thread issues, and takes
// the operands from uniform registers at once.
__device__ __forceinline__ bool tm_elect() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.b32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint32_t tm_uniform(uint32_t x) {  // x is the same in all lanes
  return __reduce_max_sync(0xFFFFFFFFu, x);
}
__device__ __forceinline__ void tm_commit(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}

// The largest of three, as fmaxf: a NaN only if all are.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Bounded wait for the phase with the given parity; a wait that runs out marks the
// CTA (*dead), whose other waits then end at once (but not kOwn ones, for a copy in flight).
template <bool kOwn = false>
__device__ __forceinline__ void pf_wait(uint64_t *bar, uint32_t parity, volatile uint32_t *dead,
                                        uint32_t *status) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = globaltimer();
  for (uint32_t i = 1; i < kWaitIters; ++i) {
    if (mbar_try_wait(bar, parity)) return;
    if ((i & 15u) == 0 && ((!kOwn && *dead) || globaltimer() - t0 > kWaitNs)) break;
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

// A block's request, first row, first key tile and tiles (0: none of its rows sees a key).
template <int NK>
__device__ __forceinline__ uint4 block_info(const CacheAttnArgs &a, uint32_t b, ReqShape &s) {
  uint32_t lo = 0, hi = a.n_req - 1;  // the last request whose first block is not past b
  while (lo < hi) {
    const uint32_t mid = (lo + hi + 1) >> 1;
    const uint32_t q0 = a.q_starts ? uint32_t(max(0, __ldg(a.q_starts + mid))) : mid;
    if (first_block(a, q0, mid) <= b) lo = mid;
    else hi = mid - 1;
  }
  bool ok;
  s = read_request(a, lo, ok);
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
  return info;
}

// First kernel. CTA 0: the requests' shapes, the blocks' numbers and the prefixes of their
// work (per layer and head). The others take 32 rows of a unit's queries each: transformed,
// in fp16 hi and lo parts as the second kernel's shared memory holds them (done there, they
// took 17000 cycles a segment, in which the tensor cores waited).
constexpr int kPfPrep = 256, kPfPrepRows = 32;
template <int D, int G>
__global__ void __launch_bounds__(kPfPrep)
    cache_prefill_prep_kernel(const __grid_constant__ CacheAttnArgs a, const int dtype) {
  using C = PfCfg<D, G>;
  constexpr int NG = C::NG, NK = C::NK, W = C::W;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.n_req;
  const uint32_t nb = a.max_blocks;
  if (blockIdx.x == 0) {
    __shared__ uint64_t red[kPfPrep / 32];
    for (uint32_t r = tid; r < n; r += kPfPrep) {
      bool ok;
      const ReqShape s = read_request(a, r, ok);
      if (!ok && a.status) set_status(a.status, KVC_ERR_CORRUPT);
      a.shapes[r] = make_uint4(s.nq, s.q0, s.len, 0);
    }
    const uint32_t per = (nb + kPfPrep - 1) / kPfPrep;
    const uint32_t b0 = min(nb, tid * per), b1 = min(nb, b0 + per);
    uint64_t w = 0;
    for (uint32_t b = b0; b < b1; ++b) {
      ReqShape s;
      const uint4 info = block_info<NK>(a, b, s);
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
    if (tid == kPfPrep - 1) a.wpre[nb] = base;
    return;
  }
  constexpr uint32_t kParts = kPfRows / kPfPrepRows;
  const uint32_t unit = (blockIdx.x - 1) / kParts, r0 = (blockIdx.x - 1 - unit * kParts) * kPfPrepRows;
  const uint32_t lh = unit / nb, l = lh / a.c.heads, h = lh - l * a.c.heads;
  ReqShape rs;
  const uint4 info = block_info<NK>(a, unit - lh * nb, rs);
  if (info.w == 0) return;
  const uint32_t nc = min(uint32_t(kPfRows), rs.nq * a.qpk - info.y);
  uint64_t w0 = a.c.w0, w1 = a.c.w1;
  if (a.c.vec_signs) {
    uint64_t st = a.c.seed + (uint64_t(l) * 2 * a.c.heads + h) * uint64_t(D / 64) * 0x9E3779B97F4A7C15ull;
    w0 = splitmix64(st);
    if constexpr (D == 128) w1 = splitmix64(st);
  }
  uint8_t *image = a.qws + uint64_t(unit) * C::QB;
  float *qx = reinterpret_cast<float *>(image + 2 * C::QPART);
#pragma unroll
  for (uint32_t x = 0; x < kPfPrepRows; x += kPfPrep / 32) {
    const uint32_t rr = r0 + x + warp;
    const int i = lane & 7, pos = i < 4 ? 2 * i : 2 * (i - 4) + 1;
    uint8_t *dst = image + rr * 128 + 2 * pos;
    if (rr >= nc) {  // rows that are not there: zeros
      if (lane <= NG) qx[lane * kPfRows + rr] = lane ? 0.f : 8.f;
#pragma unroll
      for (int y = 0; y < 2 * C::SL; ++y)
        *reinterpret_cast<uint32_t *>(image + y * kPfRows * 128 + rr * 128 + 4 * lane) = 0;
      continue;
    }
    const uint32_t gr = info.y + rr, qi = gr / a.qpk;
    const uint8_t *src = a.q + int64_t(l) * a.q_l + int64_t(rs.q0 + qi) * a.q_t +
                         int64_t(h * a.qpk + (gr - qi * a.qpk)) * a.q_h;
    float y[W];
#pragma unroll
    for (int c = 0; c < W; ++c) {
      const uint16_t in = __ldg(reinterpret_cast<const uint16_t *>(src) + lane + 32 * c);
      const float x = dtype == KVC_BF16 ? __uint_as_float(uint32_t(in) << 16)
                                        : __half2float(__ushort_as_half(in));
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
      qx[rr] = 8.f / es;
#pragma unroll
      for (int g = 0; g < NG; ++g) qx[(1 + g) * kPfRows + rr] = gs[g] * es;
    }
#pragma unroll
    for (int c = 0; c < W; ++c) {
      float vh, vl;
      split_f16(y[c] * es, vh, vl);
      const uint32_t o = (c >> 1) * kPfRows * 128 + (((4 * (c & 1) + (lane >> 3)) ^ (rr & 7)) << 4);
      *reinterpret_cast<uint16_t *>(dst + o) = __half_as_ushort(__float2half_rn(vh));
      *reinterpret_cast<uint16_t *>(dst + o + C::QPART) = __half_as_ushort(__float2half_rn(vl));
    }
  }
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

// A thread's part of a tile as it is stored: pieces p of RX rows' keys and values.
template <int D, int G>
struct PfRaw {
  static constexpr int NG = D / G, W = D / 32, RX = PfCfg<D, G>::NK / 32;
  uint32_t k[RX][W], v[RX][W], mk[RX][NG], mv[RX][NG];
  bool in[RX];
};

// Unpacking warps: every second tile of the CTA's share (odd: which). A thread has
// piece t % 4 of rows r0 + 32 x; rows r and r + 4 share a quarter-warp, whose stores
// then meet different banks. The next tile's rows are asked for as soon as a tile is
// unpacked, with pages looked up a tile earlier.
template <int D, int G>
__device__ __forceinline__ void pf_unpack(const CacheAttnArgs &a, uint8_t *smem,
                                          uint32_t which, uint64_t f, uint64_t f_end) {
  using C = PfCfg<D, G>;
  using Raw = PfRaw<D, G>;
  constexpr int NG = C::NG, NK = C::NK, W = C::W, RX = Raw::RX;
  const uint32_t t = threadIdx.x & 127, lane = t & 31, warp = t >> 5, p = t & 3;
  const uint32_t r0 = 8 * warp + 4 * ((t >> 2) & 1) + ((t >> 3) & 3);
  const uint32_t flip = W == 4 ? 2 * (p >> 1) + ((t >> 2) & 1) : (t >> 2) & 1;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::bars), *pv = full + kPfStages;
  volatile uint32_t *dead = reinterpret_cast<uint32_t *>(smem + C::ctl) + 1;
  uint32_t j0 = 0;  // tiles before the segment
  for (uint32_t tiles = 0; f < f_end; j0 += tiles) {
    const PfSegment s = pf_segment_at(a, f_end, f);
    tiles = s.tiles;
    const uint32_t i0 = (which ^ j0) & 1u;  // the segment's first tile of these warps
    if (i0 >= tiles) continue;
    const uint8_t *base = a.c.pool + int64_t(s.l) * a.c.s_l + int64_t(s.h) * a.c.s_h;
    const int32_t *table = a.page_table + int64_t(s.r) * a.pt_stride;
    int32_t pg[RX];  // pages of the next tile's rows, -1: no row sees the key
    auto look = [&](uint32_t i) {
#pragma unroll
      for (int x = 0; x < RX; ++x) {
        const int32_t tok = int32_t((s.first + i) * NK + r0 + 32 * x);
        pg[x] = -1;
        if (i < s.tiles && tok >= s.any_lo && tok < s.any_hi) {
          pg[x] = __ldg(table + fdiv(a.tpp, uint32_t(tok) / kTileTok));
          pg[x] = pg[x] < 0 ? -2 : pg[x];
        }
      }
    };
    auto load = [&](Raw &w, uint32_t i) {
#pragma unroll
      for (int x = 0; x < RX; ++x) {
        const uint32_t tok = (s.first + i) * NK + r0 + 32 * x, kt = tok / kTileTok;
        w.in[x] = pg[x] >= 0 && uint32_t(pg[x]) < a.c.num_pages;
        if (pg[x] != -1 && !w.in[x] && a.status) set_status(a.status, KVC_ERR_CORRUPT);
#pragma unroll
        for (int q = 0; q < W; ++q) w.k[x][q] = w.v[x][q] = 0x88888888u;  // (n - 8 = 0; meta 0)
#pragma unroll
        for (int g = 0; g < NG; ++g) w.mk[x][g] = w.mv[x][g] = 0;
        if (w.in[x]) {
          const uint8_t *src = base + int64_t(pg[x]) * a.c.s_p +
                               int64_t(kt - fdiv(a.tpp, kt) * a.tpp.d) * C::TB;
          const uint32_t ln = tok % kTileTok;
          const uint8_t *kr = src + ln * C::CB + 4 * W * p, *vr = kr + a.c.s_kv;
          if constexpr (W == 4) {
            const uint4 u = __ldg(reinterpret_cast<const uint4 *>(kr));
            const uint4 y = __ldg(reinterpret_cast<const uint4 *>(vr));
            w.k[x][0] = u.x, w.k[x][1] = u.y, w.k[x][2] = u.z, w.k[x][3] = u.w;
            w.v[x][0] = y.x, w.v[x][1] = y.y, w.v[x][2] = y.z, w.v[x][3] = y.w;
          } else {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(kr));
            const uint2 y = __ldg(reinterpret_cast<const uint2 *>(vr));
            w.k[x][0] = u.x, w.k[x][1] = u.y;
            w.v[x][0] = y.x, w.v[x][1] = y.y;
          }
          const uint8_t *m = src + kTileTok * C::CB + ln * NG * 4;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            w.mk[x][g] = __ldg(reinterpret_cast<const uint32_t *>(m) + g);
            w.mv[x][g] = __ldg(reinterpret_cast<const uint32_t *>(m + a.c.s_kv) + g);
          }
        }
      }
      look(i + 2);
    };
    auto unpack = [&](const Raw &w, uint32_t j) {
      const uint32_t buf = j % kPfStages, turn = j / kPfStages;
      if (turn) pf_wait(pv + buf, (turn - 1) & 1u, dead, a.status);
      uint8_t *kb = smem + C::k + buf * C::KBUF, *vb = smem + C::v + buf * C::KBUF;
      float *meta = reinterpret_cast<float *>(smem + C::meta) + buf * C::MW * NK;
      uint32_t most = 0;
      bool gone = false, odd = false;  // a key that is not there, a value that is not finite
#pragma unroll
      for (int x = 0; x < RX; ++x) {
        const uint32_t row = r0 + 32 * x, sw = row & 7;
        uint8_t *kr = kb + row * 128, *vr = vb + row * 128;
#pragma unroll
        for (int b = 0; b < W; ++b) {
          const uint32_t u = w.k[x][b];
          *reinterpret_cast<uint4 *>(kr + (b >> 1) * NK * 128 + (((4 * (b & 1) + p) ^ sw) << 4)) =
              make_uint4(centred<false>(u), centred<true>(u), centred<false>(u >> 8),
                         centred<true>(u >> 8));
        }
        // values x 2^-e, e from the largest |z + 8 s| + 8 |s|
        bool bad = false;
        float bound = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          bad |= not_finite(w.mv[x][g]);
          bound = fmaxf(bound, fabsf(zero8(w.mv[x][g])) + 8.f * fabsf(half_lo(w.mv[x][g])));
        }
        const uint32_t ex = (__float_as_uint(bound) >> 23) & 255u;
        const bool none = bad || bound == 0.f;
        // (zeros weigh nothing: with a scale of 1 their weights, scaled up for small values
        // beside them, passed fp16's range)
        const float scale = none ? 0.f : __uint_as_float(ex << 23);  // (-0: not finite)
        const float inv = none ? 0.f : __uint_as_float((254u - ex) << 23);
        float sv[NG], zv[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const uint32_t m = bad ? 0u : w.mv[x][g];  // (|z|, 15 |s| <= 2 bound)
          sv[g] = half_lo(m) * inv;
          zv[g] = half_hi(m) * inv;
        }
        // a lane's words in an order of its own (q ^ flip): in step, eight lanes' pieces
        // would meet in two columns of the banks (17 of 43 million wavefronts)
        uint32_t vw[W];
#pragma unroll
        for (int q = 0; q < W; ++q) vw[q] = w.v[x][q];
        auto swap_if = [](bool yes, auto &a, auto &b) {
          const auto c = yes ? b : a;
          b = yes ? a : b;
          a = c;
        };
#pragma unroll
        for (int q = 0; q < W; q += 2) swap_if(flip & 1, vw[q], vw[q + 1]);
        if constexpr (W == 4) {
          swap_if(flip & 2, vw[0], vw[2]);
          swap_if(flip & 2, vw[1], vw[3]);
#pragma unroll
          for (int g = 0; g < NG / 2; ++g) {  // the groups of words q and q ^ 1
            swap_if(flip & 1, sv[g], sv[g + NG / 2]);
            swap_if(flip & 1, zv[g], zv[g + NG / 2]);
          }
        }
#pragma unroll
        for (int q = 0; q < W; ++q) {
          const uint32_t wj = W * p + (q ^ flip);  // stored word: halves of 32-channel blocks a, a + 1
          const int ga = ((2 * q) % W) * 32 / G, gb = ((2 * q) % W + 1) * 32 / G;
          const uint32_t s2 = f16x2(sv[ga], sv[gb]), z2 = f16x2(zv[ga], zv[gb]), u = vw[q];
          auto deq = [&](uint32_t n) {
            uint32_t d;
            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(n), "r"(s2), "r"(z2));
            return d;
          };
          *reinterpret_cast<uint4 *>(vr + (wj >> 3) * NK * 128 + (((wj & 7) ^ sw) << 4)) =
              make_uint4(deq(codes_less<false, 0>(u)), deq(codes_less<true, 0>(u)),
                         deq(codes_less<false, 0>(u >> 8)), deq(codes_less<true, 0>(u >> 8)));
        }
        if (int(p) < NG) {
          uint32_t m = w.mk[x][0];
#pragma unroll
          for (int g = 1; g < NG; ++g) m = int(p) == g ? w.mk[x][g] : m;
          meta[p * NK + row] = half_lo(m);
          meta[(NG + p) * NK + row] = zero8(m);
        }
        const float bias = !w.in[x] ? -INFINITY : 0.f;
        if (p == 3) {
          meta[2 * NG * NK + row] = bad ? -0.f : scale;
          meta[(2 * NG + 1) * NK + row] = bias;
        }
        gone |= !w.in[x];
        odd |= bad;
        most = max(most, __float_as_uint(scale));
      }
      most = __reduce_max_sync(0xFFFFFFFFu, most);
      uint32_t odds = 0;  // bit 0: some key is not there, bit 1: some value is not finite
      if (__any_sync(0xFFFFFFFFu, gone || odd))
        odds = (__any_sync(0xFFFFFFFFu, gone) ? 1u : 0u) | (__any_sync(0xFFFFFFFFu, odd) ? 2u : 0u);
      if (lane == 0) {
        reinterpret_cast<uint32_t *>(smem + C::wmax)[buf * 4 + warp] = most;
        reinterpret_cast<uint32_t *>(smem + C::wodd)[buf * 4 + warp] = odds;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + buf);
    };
    Raw raw;
    look(i0);
    load(raw, i0);
    for (uint32_t i = i0; i < tiles; i += 2) {
      unpack(raw, j0 + i);
      load(raw, i + 2);  // (past the segment's end: nothing is read)
    }
  }
}

// Starting products. A start takes as long as its products where the tensor cores' queue
// is full, and a wait some hundred cycles. With three tiles' scores one warp starts scores
// and one values (one for both was busy for 2000 cycles a tile, which bounded the kernel:
// 284 us against 268 for 1024 queries over 9216 keys). Products of two threads are not
// ordered: there a tile's scores wait until the values of the tile NS before, whose weights
// they replace, are done. With two tiles' scores that wait costs more than it gives (343 us
// with one warp, 356 with two, at two groups): one warp starts values i, then scores i + 2.
template <int D, int G>
struct PfIssue {
  using C = PfCfg<D, G>;
  static constexpr uint32_t NS = C::NS, ST = kPfStages;
  uint32_t tm, q_s, k_s, v_s, *status;
  uint64_t *full, *pv, *sready, *pready, *qready;
  volatile uint32_t *dead;
  __device__ __forceinline__ PfIssue(const CacheAttnArgs &a, uint8_t *smem, uint32_t tm_)
      : tm(tm_), q_s(smem_u32(smem + C::q)), k_s(smem_u32(smem + C::k)), v_s(smem_u32(smem + C::v)),
        status(a.status) {
    full = reinterpret_cast<uint64_t *>(smem + C::bars);
    pv = full + ST;
    sready = pv + ST;
    pready = sready + NS;
    qready = pready + NS;
    dead = reinterpret_cast<uint32_t *>(smem + C::ctl) + 1;
  }
  __device__ __forceinline__ void wait(uint64_t *bar, uint32_t phase) const {
    pf_wait(bar, phase, dead, status);
  }
  // Scores of the tile in stage st to place sb.
  __device__ __forceinline__ void scores(uint32_t st, uint32_t sb) const {
    constexpr int SG = G / 16;  // (16-channel steps of a group)
    tm_fence_after();
    __syncwarp();
    const uint64_t dq = tm_desc(q_s, 16, 1024), dk = tm_desc(k_s + st * C::KBUF, 16, 1024);
    const uint32_t ts = tm + C::tS + sb * C::SW;
    if (tm_elect()) {
#pragma unroll
      for (int g = 0; g < C::NG; ++g)
#pragma unroll
        for (int x = 0; x < 2 * SG; ++x) {  // hi parts, then lo
          const int c = g * SG + x % SG, o = (c & 3) * 2;
          const uint64_t k = dk + (((c >> 2) * C::NK * 128) >> 4) + o;
          if (x < SG ? C::QH : C::QL)
            tm_mma_ts(ts + g * C::NK, tm + C::tQ + (x / SG) * (D / 2) + c * 8, k, tm_idesc(C::NK, false),
                      x != 0);
          else
            tm_mma(ts + g * C::NK, dq + (((x / SG) * C::QPART + (c >> 2) * kPfRows * 128) >> 4) + o, k,
                   tm_idesc(C::NK, false), x != 0);
        }
      tm_commit(sready + sb);
    }
    __syncwarp();
  }
  // Weights at place sb times the values of stage st, for softmax `odd`.
  __device__ __forceinline__ void values(uint32_t st, uint32_t sb, uint32_t odd, bool add) const {
    tm_fence_after();
    __syncwarp();
    const uint64_t dv = tm_desc(v_s + st * C::KBUF, C::NK * 128, 1024);
    const uint32_t ts = tm + C::tS + sb * C::SW, to = tm + C::tO + odd * D;
    if (tm_elect()) {
#pragma unroll
      for (int x = 0; x < C::NK / 16; ++x)
        tm_mma_ts(to, ts + x * 8, dv + x * 128, tm_idesc(D, true), add || x != 0);
      tm_commit(pv + st);
    }
    __syncwarp();
  }
};
// A place among N and the phase it is in, counted on (a division per tile is dear here).
template <uint32_t N>
struct PfPlace {
  uint32_t at = 0, phase = 0;
  __device__ __forceinline__ void next() {
    phase ^= at == N - 1 ? 1u : 0u;
    at = at == N - 1 ? 0 : at + 1;
  }
};

// which: 0 scores (and values, with two tiles' scores), 1 values.
template <int D, int G>
__device__ __forceinline__ void pf_issue(const CacheAttnArgs &a, uint8_t *smem, uint32_t tm,
                                         uint32_t which, uint64_t f, uint64_t f_end) {
  using C = PfCfg<D, G>;
  constexpr uint32_t NS = C::NS, ST = kPfStages;
  const PfIssue<D, G> p(a, smem, tm);
  PfPlace<ST> ks, vs;  // stages of the next scores and values
  PfPlace<NS> sb, wb;  // places of the next scores and weights
  uint32_t before = 0, seg = 0, odd = 0;
  if (NS == 2 && which == 1) return;
  while (f < f_end) {
    const PfSegment s = pf_segment_at(a, f_end, f);
    if (s.tiles == 0) continue;
    const uint32_t tiles = tm_uniform(s.tiles);
    if (which == 0) {
      p.wait(p.qready, seg & 1u);
      ++seg;
    }
    auto scores = [&]() {
      p.wait(p.full + ks.at, ks.phase);
      p.scores(ks.at, sb.at);
      ks.next();
      sb.next();
    };
    auto values = [&](uint32_t i) {
      p.wait(p.pready + wb.at, wb.phase);
      p.values(vs.at, wb.at, odd, i > 1);
      vs.next();
      wb.next();
      odd ^= 1u;
    };
    if constexpr (NS == 2) {
      scores();
      if (tiles > 1) scores();
      for (uint32_t i = 0; i < tiles; ++i) {
        values(i);
        if (i + 2 < tiles) scores();
      }
    } else if (which == 0) {
      for (uint32_t i = 0; i < tiles; ++i) {
        if (before == NS) {  // (vs: the stage of the tile NS before)
          p.wait(p.pv + vs.at, vs.phase);
          vs.next();
        } else {
          ++before;
        }
        scores();
      }
    } else {
      for (uint32_t i = 0; i < tiles; ++i) values(i);
    }
  }
}

template <int D, int G>
__global__ void __launch_bounds__(kPfThreads, 1)
    cache_prefill_kernel(const __grid_constant__ CacheAttnArgs a) {
  using C = PfCfg<D, G>;
  constexpr int NG = C::NG, NK = C::NK, W = C::W;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::bars), *pv = full + kPfStages;
  uint64_t *sready = pv + kPfStages, *pready = sready + C::NS, *qready = pready + C::NS;
  uint64_t *qcopied = qready + 1;
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
    for (uint32_t i = 0; i < kPfStages; ++i) {
      mbar_init(full + i, 4);
      mbar_init(pv + i, 1);
    }
    for (uint32_t i = 0; i < C::NS; ++i) {
      mbar_init(sready + i, 1);
      mbar_init(pready + i, 4);
    }
    mbar_init(qready, kPfSoft / 32);
    mbar_init(qcopied, 1);
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

  if (warp >= (kPfSoft + kPfUnpack) / 32) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPfIssueRegs));
    const uint32_t which = uint32_t(warp) - (kPfSoft + kPfUnpack) / 32;
    if (which == 0) pf_issue<D, G>(a, smem, tm_uniform(tm), 0, f, f_end);
    if (which == 1) pf_issue<D, G>(a, smem, tm_uniform(tm), 1, f, f_end);
  } else if (warp >= kPfSoft / 32) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPfUnpackRegs));
    pf_unpack<D, G>(a, smem, uint32_t(warp >> 2) & 1u, f, f_end);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPfSoftRegs));
    const int which = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t tl = tm + (uint32_t((warp & 3) * 32) << 16);  // this warp's lanes
    const uint32_t tO = tl + C::tO + which * D;
    float2 *fin = reinterpret_cast<float2 *>(smem + C::fin);
    uint32_t j0 = 0, seg = 0;  // tiles and segments before

    while (f < f_end) {
      const PfSegment s = pf_segment_at(a, f_end, f);
      if (s.tiles == 0) continue;
      // ---- the block's queries, copied at once
      if (tid == 0) {
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(qcopied, 2 * C::QPART);
        bulk_g2s(smem + C::q, a.qws + s.unit * C::QB, 2 * C::QPART, qcopied);
      }
      __syncwarp();
      const float *qx = reinterpret_cast<const float *>(a.qws + s.unit * C::QB + 2 * C::QPART) + row;
      const float fc = __ldg(qx);
      float qsum[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) qsum[g] = __ldg(qx + (1 + g) * kPfRows);
      int32_t lo = 0, hi = 0;
      if (uint32_t(row) < s.nc) key_range(a, s.rs, (s.c0 + row) / a.qpk, lo, hi);
      pf_wait<true>(qcopied, seg & 1u, dead, a.status);
      ++seg;
      __syncwarp();
      // this row's hi (first softmax) or lo parts to tensor memory
      if (which == 0 ? C::QH : C::QL) {
        const uint8_t *src = smem + C::q + which * C::QPART + row * 128;
#pragma unroll
        for (int x = 0; x < D / 2; x += 8) {
          uint32_t u[8];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int piece = (x / 4 + e) & 7, sl = (x / 4 + e) >> 3;
            const uint4 v = *reinterpret_cast<const uint4 *>(src + sl * kPfRows * 128 + ((piece ^ (row & 7)) << 4));
            u[4 * e] = v.x, u[4 * e + 1] = v.y, u[4 * e + 2] = v.z, u[4 * e + 3] = v.w;
          }
          tm_st8(tl + C::tQ + which * (D / 2) + x, u);
        }
        tm_wait_st();
      }
      fence_proxy_async_smem();
      tm_fence_before();  // (the segment before has been read)
      __syncwarp();
      if (lane == 0) mbar_arrive(qready);
      // Running state as in kvc_cache_attend.cuh: n (row_factor), the sum of p. While raw scores
      // stay below thr (-inf: none seen so far, or nothing but NaN) and the values' 2^e below
      // v_most, no weight passes its range; both are those of the last tile that was not below.
      float nm = 0.f, thr = -INFINITY, l = 0.f, v_most = 0.f;
      float *taint = reinterpret_cast<float *>(smem + C::taint) + which * kPfRows + row;
      *taint = 0.f;  // NaN once the row has seen a value that is not finite

      for (uint32_t i = (which ^ j0) & 1u; i < s.tiles; i += 2) {
        const uint32_t j = j0 + i, buf = j % kPfStages, sb = j % C::NS, tS = tl + C::tS + sb * C::SW;
        const int32_t t0 = int32_t((s.first + i) * NK);
        pf_wait(full + buf, (j / kPfStages) & 1u, dead, a.status);  // the keys' numbers
        pf_wait(sready + sb, (j / C::NS) & 1u, dead, a.status);
        tm_fence_after();
        __syncwarp();
        const float *meta = reinterpret_cast<const float *>(smem + C::meta) + buf * C::MW * NK;
        float sc[NK];
#pragma unroll
        for (int x0 = 0; x0 < NK; x0 += 16) {
          float acc[NG][16];
#pragma unroll
          for (int g = 0; g < NG; ++g) tm_ld16(tS + g * NK + x0, acc[g]);
          tm_wait_ld();
#pragma unroll
          for (int g = 0; g < NG; ++g) tm_loaded16(acc[g]);
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const float2 q2 = make_float2(qsum[g], qsum[g]);
#pragma unroll
            for (int y = 0; y < 16; y += 4) {
              const int x = x0 + y;
              const float4 ks = *reinterpret_cast<const float4 *>(meta + g * NK + x);
              const float4 kz = *reinterpret_cast<const float4 *>(meta + (NG + g) * NK + x);
              float2 u = g == 0 ? mul2(make_float2(kz.x, kz.y), q2)
                                : fma2(make_float2(kz.x, kz.y), q2, make_float2(sc[x], sc[x + 1]));
              float2 v = g == 0 ? mul2(make_float2(kz.z, kz.w), q2)
                                : fma2(make_float2(kz.z, kz.w), q2, make_float2(sc[x + 2], sc[x + 3]));
              u = fma2(make_float2(ks.x, ks.y), make_float2(acc[g][y], acc[g][y + 1]), u);
              v = fma2(make_float2(ks.z, ks.w), make_float2(acc[g][y + 2], acc[g][y + 3]), v);
              sc[x] = u.x, sc[x + 1] = u.y, sc[x + 2] = v.x, sc[x + 3] = v.y;
            }
          }
        }
        const uint4 odd = *reinterpret_cast<const uint4 *>(smem + C::wodd + buf * 16);
        const uint32_t odds = odd.x | odd.y | odd.z | odd.w;
        if (odds || t0 < s.all_lo || uint32_t(t0) + NK > uint32_t(s.all_hi)) {
          if (odds & 2u) {  // values that are not finite: out is NaN for the rows that see them
#pragma unroll 1
            for (int x = max(lo - t0, 0); x < min(hi - t0, NK); ++x)
              if (__float_as_uint(meta[2 * NG * NK + x]) == 0x80000000u) *taint = __uint_as_float(0x7FFFFFFFu);
          }
#pragma unroll
          for (int x = 0; x < NK; ++x) {
            const int32_t t = t0 + x;
            sc[x] = t >= lo && t < hi ? sc[x] + meta[(2 * NG + 1) * NK + x] : -INFINITY;
          }
        }
        float tops[4] = {sc[0], sc[1], sc[2], sc[3]};
#pragma unroll
        for (int x = 4; x + 4 < NK; x += 8)
#pragma unroll
          for (int y = 0; y < 4; ++y) tops[y] = max3(tops[y], sc[x + y], sc[x + y + 4]);
#pragma unroll
        for (int y = 0; y < 4; ++y) tops[y] = fmaxf(tops[y], sc[NK - 4 + y]);
        const float top = max3(fmaxf(tops[0], tops[1]), tops[2], tops[3]);
        const float4 wm = *reinterpret_cast<const float4 *>(smem + C::wmax + buf * 16);
        const float vm = fmaxf(fmaxf(wm.x, wm.y), fmaxf(wm.z, wm.w));
        if (__any_sync(0xFFFFFFFFu, top > thr) || vm > v_most) {
          const float e_top = log2_floor(__float_as_uint(vm)), x = top * fc;
          v_most = 4.f * vm;
          const bool first = thr == -INFINITY;
          float fac = 1.f;
          const float most = fminf(kPMost, kWeightMost - 1.f - e_top);
          const bool need = x > -INFINITY && (first || x + nm > most);
          if (__any_sync(0xFFFFFFFFu, need)) {
            // the smallest e (of zeros and keys that are not there: -127)
            const uint32_t *vb = reinterpret_cast<const uint32_t *>(meta) + 2 * NG * NK;
            uint32_t low = vb[lane] & 0x7FFFFFFFu;
            if constexpr (NK == 64) low = min(low, vb[lane + 32] & 0x7FFFFFFFu);
            low = __reduce_min_sync(0xFFFFFFFFu, low);
            float w = x + e_top + 1.f;  // (where the e are alike, it will do)
            if (e_top - log2_floor(low) > 3.f) {
              w = -INFINITY;
#pragma unroll
              for (int y = 0; y < NK; y += 4) {
                const uint4 ev = *reinterpret_cast<const uint4 *>(meta + 2 * NG * NK + y);
                auto at = [&](float x, uint32_t u) {  // x fc + e (zeros: -127)
                  return fmaf(x, fc, __uint_as_float(((u >> 23) & 255u) | 0x4B000000u) - 8388735.f);
                };
                w = max3(max3(w, at(sc[y], ev.x), at(sc[y + 1], ev.y)), at(sc[y + 2], ev.z), at(sc[y + 3], ev.w));
              }
            }
            if (need) {
              const float n = row_factor(nm, x, w, first);
              if (!first) fac = ex2(n - nm);
              nm = n;
            }
          }
          if (!first || x > -INFINITY) thr = (most - nm) / fc;
          l *= fac;
          if (i > 1 && __any_sync(0xFFFFFFFFu, fac != 1.f)) {  // this softmax's last values are in
            pf_wait(pv + (j - 2) % kPfStages, ((j - 2) / kPfStages) & 1u, dead, a.status);
            tm_fence_after();
            __syncwarp();
#pragma unroll
            for (int x = 0; x < D; x += 16) {
              float o[16];
              tm_ld16(tO + x, o);
              tm_wait_ld();
              tm_loaded16(o);
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] *= fac;
              tm_st16(tO + x, o);
            }
          }
        }
        const float *vs = meta + 2 * NG * NK;
        const float2 f2 = make_float2(fc, fc), n2 = make_float2(nm, nm);
        float2 l2 = make_float2(0.f, 0.f), l3 = l2;
#pragma unroll
        for (int x = 0; x < NK; x += 16) {
          uint32_t pk[8];
#pragma unroll
          for (int y = 0; y < 16; y += 4) {
            const float4 sv = *reinterpret_cast<const float4 *>(vs + x + y);
            const float2 u = fma2(make_float2(sc[x + y], sc[x + y + 1]), f2, n2);
            const float2 v = fma2(make_float2(sc[x + y + 2], sc[x + y + 3]), f2, n2);
            const float2 pu = make_float2(ex2(u.x), ex2(u.y)), pw = make_float2(ex2(v.x), ex2(v.y));
            l2 = add2(l2, pu);
            l3 = add2(l3, pw);
            const float2 wu = mul2(pu, make_float2(sv.x, sv.y)), ww = mul2(pw, make_float2(sv.z, sv.w));
            pk[y / 2] = f16x2(wu.x, wu.y);
            pk[y / 2 + 1] = f16x2(ww.x, ww.y);
          }
          tm_st8(tS + x / 2, pk);
        }
        l2 = add2(l2, l3);
        l += l2.x + l2.y;
        tm_wait_st();
        tm_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pready + sb);
      }

      // ---- the segment's record, of both softmaxes' results
      j0 += s.tiles;
      pf_wait(pv + (j0 - 1) % kPfStages, ((j0 - 1) / kPfStages) & 1u, dead, a.status);
      tm_fence_after();
      fin[which * kPfRows + row] = make_float2(thr == -INFINITY ? -INFINITY : -nm, l);
      named_bar_sync(1, kPfSoft);
      const float2 mine[2] = {fin[row], fin[kPfRows + row]};
      const float m = fmaxf(mine[0].x, mine[1].x);
      float w[2];
      bool has[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {  // (a maximum of -inf: zeros, or NaN, which stay)
        has[x] = s.tiles > 1 || ((j0 - 1) & 1u) == uint32_t(x);
        w[x] = mine[x].x == -INFINITY ? 1.f : ex2(mine[x].x - m);
      }
      float *rec = a.rec + (s.unit + blockIdx.x) * uint64_t(kPfRows * (4 + D)) + row * (4 + D);
      const bool live = uint32_t(row) < s.nc;
      const float bad = *taint;  // (in some columns is enough: the inverse transform mixes all)
      if (live && which == 0)
        *reinterpret_cast<float2 *>(rec) = make_float2(m, mine[0].y * w[0] + mine[1].y * w[1]);
#pragma unroll
      for (int x = 0; x < D / 2; x += 16) {  // half of the columns each
        float o[16], o1[16];
        tm_ld16(tl + C::tO + which * (D / 2) + x, o);
        tm_ld16(tl + C::tO + D + which * (D / 2) + x, o1);
        tm_wait_ld();
        tm_loaded16(o);
        tm_loaded16(o1);
#pragma unroll
        for (int y = 0; y < 16; ++y)
          o[y] = 8.f * ((has[0] ? o[y] * w[0] : 0.f) + (has[1] ? o1[y] * w[1] : 0.f)) + bad;
#pragma unroll
        for (int y = 0; y < 16; y += 8) {
          // columns of stored word wj: halves of its two 32-channel blocks
          const int wj = (which * (D / 2) + x + y) / 8, hs = 2 * wj;
          const int ch = 32 * (hs % W) + 4 * (hs / W);
          if (live) {
            *reinterpret_cast<float4 *>(rec + 4 + ch) = make_float4(o[y], o[y + 2], o[y + 4], o[y + 6]);
            *reinterpret_cast<float4 *>(rec + 4 + ch + 32) =
                make_float4(o[y + 1], o[y + 3], o[y + 5], o[y + 7]);
          }
        }
      }
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
  static constexpr bool kWide = false;  // (a block has a record per CTA that it was cut for: few)
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
  static_assert(C::QB == kPfRows * (4 * D + 4 * (1 + C::NG)), "workspace");
  const uint64_t units = uint64_t(a.c.layers) * a.c.heads * a.max_blocks;
  cache_prefill_prep_kernel<D, G>
      <<<unsigned(units * (kPfRows / kPfPrepRows) + 1), kPfPrep, 0, st>>>(a, dtype);
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
  e = cudaLaunchKernelEx(&cfg, k, a);
  if (e != cudaSuccess) return e;
  return launch_combine<D, PrefillRecords>(dtype, false, a, grid, st);
}

}  // namespace kvc
