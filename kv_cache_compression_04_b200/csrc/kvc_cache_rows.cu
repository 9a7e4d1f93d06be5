// Writing, reading and loading rows of the paged 4-bit cache.
//
// A vector is held by four lanes: lane p of the four has channels 32*b + 8*p
// .. + 7 of every 32-channel block b, i.e. one 4-byte code word per block. So
// a 32-lane load takes 64 contiguous bytes of each of eight rows, the
// butterfly's strides 1, 2, 4 and 32, 64 stay in registers and only 8 and 16
// cross lanes (two shuffles per channel), and the stored orders (a key's words
// and a value's halfwords transposed, include/kvc.h) are what a lane holds:
// its words are 4 * (head_dim / 32) consecutive bytes of a key row, their
// halves two consecutive runs of a value row.
//
// 64 tokens x 8 heads are one wave of latency: written and read back in 5.2 us. Loading 4096
// tokens x 32 layers takes 75 us (0.58 of the copy rate): its warps wait for the look-ups in
// the stream's tables (12.6 of 22 stalled warps per issue; issue slots 59% used, DRAM 39%).
#include "kvc_cache_rows.cuh"

namespace kvc {

namespace {

constexpr int kRowWarps = 4;
constexpr int kRowThreads = kRowWarps * 32;
constexpr int kRowTok = kRowWarps * 8;  // tokens per CTA

// The diagonal of (layer, kv, head) lkh as masks of channel pairs in shared
// memory: word k flips the 16-bit signs of channels 2 k (bit 15) and 2 k + 1 (bit
// 31); words D / 2 + k the former at bit 31. (From the sign bits in registers, the
// masks took 96 instructions of the 666 that eight vectors took; read back, 8.)
template <int D>
__device__ __forceinline__ void sign_table(const CachePool &c, uint32_t lkh, uint32_t *mask) {
  const uint32_t k = threadIdx.x;
  if (k < D / 2) {
    uint64_t w = k < 32 ? c.w0 : c.w1;
    if (c.vec_signs) {
      uint64_t st = c.seed + uint64_t(lkh) * uint64_t(D / 64) * 0x9E3779B97F4A7C15ull;
      w = splitmix64(st);
      if (k >= 32) w = splitmix64(st);
    }
    const uint32_t b = uint32_t(w >> (2 * (k & 31)));
    mask[k] = ((b & 1u) << 15) | ((b & 2u) << 30);
    mask[D / 2 + k] = b << 31;
  }
}

// y[j][i]: channel i of blocks j and j + D / 64 (x, y). The butterfly of
// reading R2 (strides ascending, one rounding each): 1, 2, 4 between i; 8 and
// 16 between lanes (b - a as a fused a * -1 + b, the same rounding); 32 between
// j (d = 128), d / 2 inside each pair.
template <int D>
__device__ __forceinline__ void fwht_lanes(float2 (&y)[D / 64][8], uint32_t p) {
  constexpr int N = D / 64;
#pragma unroll
  for (int h = 1; h < 8; h <<= 1)
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((i & h) == 0) {
          const float2 a = y[j][i], b = y[j][i + h];
          y[j][i] = add2(a, b);
          y[j][i + h] = sub2(a, b);
        }
#pragma unroll
  for (uint32_t s = 1; s < 4; s <<= 1) {
    const float sg = (p & s) ? -1.0f : 1.0f;
    const float2 sg2 = make_float2(sg, sg);
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 o = make_float2(__shfl_xor_sync(0xFFFFFFFFu, y[j][i].x, s),
                                     __shfl_xor_sync(0xFFFFFFFFu, y[j][i].y, s));
        y[j][i] = fma2(y[j][i], sg2, o);
      }
  }
  if constexpr (N == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 a = y[0][i], b = y[1][i];
      y[0][i] = add2(a, b);
      y[1][i] = sub2(a, b);
    }
  }
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = y[j][i].x, b = y[j][i].y;
      y[j][i] = make_float2(__fadd_rn(a, b), __fsub_rn(a, b));
    }
}

// Eight 16-bit values -> fp32, signs flipped by their masks (m; lo: the even
// channels' at bit 31).
template <int DT>
__device__ __forceinline__ void widen8(const uint4 &v, const uint4 &m, const uint4 &lo,
                                       float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w}, ms[4] = {m.x, m.y, m.z, m.w};
  const uint32_t ls[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (DT == KVC_BF16) {
      f[2 * k] = __uint_as_float((w[k] << 16) + ls[k]);
      f[2 * k + 1] = __uint_as_float((w[k] ^ ms[k]) & 0xFFFF0000u);
    } else {
      const uint32_t x = w[k] ^ ms[k];
      f[2 * k] = __half2float(__ushort_as_half(uint16_t(x)));
      f[2 * k + 1] = __half2float(__ushort_as_half(uint16_t(x >> 16)));
    }
  }
}

// Minimum and maximum over the four lanes of a vector.
__device__ __forceinline__ void lanes_minmax(float &mn, float &mx) {
#pragma unroll
  for (uint32_t s = 1; s < 4; s <<= 1) {
    mn = min2n(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, s));
    mx = max2n(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, s));
  }
}

// Scale, zero and code rules of readings R5 and R19 (Enc::quantize), for one
// group's minimum and maximum.
struct Group {
  float zf, r;    // subtracted before the product, reciprocal of the scale
  uint32_t meta;  // fp16 scale, fp16 zero
  uint32_t err;   // 1: not finite, 2: fp16 overflow
};
__device__ __forceinline__ Group group_of(float mn, float mx, uint32_t sym) {
  constexpr float down = 0.125f, up = 8.0f;
  Group g{};
  mn = __fadd_rn(mn, 0.0f);
  mx = __fadd_rn(mx, 0.0f);
  __half zh, sh;
  if (sym) {
    const float am = max2n(fabsf(mn), fabsf(mx));
    sh = __float2half_ru(__fmul_rn(div_const<7>(am), down));
    zh = (__half_as_ushort(sh) & 0x7FFFu) == 0
             ? __ushort_as_half(0)
             : __float2half_rd(__fmul_rn(__half2float(sh), -8.0f));
    g.zf = 0.0f;
  } else {
    zh = __float2half_rd(__fmul_rn(mn, down));
    g.zf = __fmul_rn(__half2float(zh), up);
    sh = __float2half_ru(__fmul_rn(div_const<15>(__fsub_rn(mx, g.zf)), down));
  }
  const float sf = __fmul_rn(__half2float(sh), up);
  g.r = sf == 0.0f ? 0.0f : rcp_scale(sf);
  g.meta = uint32_t(__half_as_ushort(sh)) | (uint32_t(__half_as_ushort(zh)) << 16);
  if (!(isfinite(mn) && isfinite(mx)))
    g.err = 1u;
  else if (!(isfinite(__half2float(zh)) && isfinite(sf)))
    g.err = 2u;
  return g;
}

template <int D, int G, int DT>
__global__ void __launch_bounds__(kRowThreads)
    cache_write_kernel(const __grid_constant__ CachePool c, const __grid_constant__ RowArgs r) {
  constexpr int NB = D / 32, N = D / 64, NG = D / G;
  __shared__ alignas(16) uint32_t mask[D];
  const uint32_t lane = threadIdx.x & 31, p = lane & 3;
  const uint32_t t = blockIdx.x * kRowTok + (threadIdx.x >> 5) * 8 + (lane >> 2);
  const uint32_t slot = slot_of(r, c, t);
  for (uint32_t lkh = blockIdx.y; lkh < c.layers * 2 * c.heads; lkh += gridDim.y) {
    const uint32_t lk = lkh / c.heads, h = lkh - lk * c.heads, l = lk >> 1, kv = lk & 1;
    const uint8_t *row = kv ? r.v + int64_t(l) * r.v_l + int64_t(t) * r.v_t + int64_t(h) * r.v_h
                            : r.k + int64_t(l) * r.k_l + int64_t(t) * r.k_t + int64_t(h) * r.k_h;
    uint4 in[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
      in[b] = slot != ~0u ? __ldg(reinterpret_cast<const uint4 *>(row + 64 * b + 16 * p))
                          : make_uint4(0, 0, 0, 0);
    if (lkh != blockIdx.y) __syncthreads();  // the masks before are read
    sign_table<D>(c, lkh, mask);
    __syncthreads();
    const uint4 *mk = reinterpret_cast<const uint4 *>(mask);
    float2 y[N][8];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float a[8], b[8];
      widen8<DT>(in[j], mk[4 * j + p], mk[D / 8 + 4 * j + p], a);
      widen8<DT>(in[j + N], mk[4 * (j + N) + p], mk[D / 8 + 4 * (j + N) + p], b);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[j][i] = make_float2(a[i], b[i]);
    }
    fwht_lanes<D>(y, p);
    // minimum and maximum of every block (three at a time), of every group, over the lanes
    float mn[NB], mx[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      auto at = [&](int i) { return j < N ? y[j % N][i].x : y[j % N][i].y; };
      mn[j] = min2n(min3n(min3n(at(0), at(1), at(2)), at(3), at(4)), min3n(at(5), at(6), at(7)));
      mx[j] = max2n(max3n(max3n(at(0), at(1), at(2)), at(3), at(4)), max3n(at(5), at(6), at(7)));
    }
    Group g[NG];
    uint32_t err = 0;
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      float lo = mn[q * (G / 32)], hi = mx[q * (G / 32)];
#pragma unroll
      for (int b = 1; b < G / 32; ++b) {
        lo = min2n(lo, mn[q * (G / 32) + b]);
        hi = max2n(hi, mx[q * (G / 32) + b]);
      }
      lanes_minmax(lo, hi);
      g[q] = group_of(lo, hi, c.sym);
      err |= g[q].err;
    }
    // Codes: nearest integer (ties to even) of the fp32 product, see Enc::quantize. A
    // code is in the low bits of its float, above 0x4B400000: shifted to its place and
    // added, and the eight constants' sum taken off.
    constexpr uint32_t kBase = 0x4B400000u * 0x11111111u;
    const float magic = c.sym ? 12582920.0f : 12582912.0f;
    const float2 mag = make_float2(magic, magic), one2 = make_float2(r.one, r.one);
    uint32_t w[NB];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int ga = j * 32 / G, gb = (j + N) * 32 / G;
      uint32_t a = 0u - kBase, b = 0u - kBase;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 d = sub2(y[j][i], make_float2(g[ga].zf, g[gb].zf));
        const float2 q = fma2(mul2(d, make_float2(g[ga].r, g[gb].r)), one2, mag);
        a += __float_as_uint(q.x) << (4 * i);
        b += __float_as_uint(q.y) << (4 * i);
      }
      w[j] = a;
      w[j + N] = b;
    }
    if (slot == ~0u) continue;
    if (err) {
      note(r.status, (err & 1u) ? KVC_ERR_NONFINITE : KVC_ERR_RANGE);
#pragma unroll
      for (int j = 0; j < NB; ++j) w[j] = 0;  // (both forms store the same)
    }
    const Place<D, G> at(c, slot, l, kv, h);
    put_words<D>(at.codes, p, kv, w);
    // a vector with an error reads as NaN
    if constexpr (NG == 1) {
      if (p == 0) *reinterpret_cast<uint32_t *>(at.meta) = err ? 0x7FFF7FFFu : g[0].meta;
    } else if constexpr (NG == 2) {
      if (p < 2)
        reinterpret_cast<uint32_t *>(at.meta)[p] = err ? 0x7FFF7FFFu : p ? g[1].meta : g[0].meta;
    } else {
      const uint32_t m = p & 2 ? (p & 1 ? g[3].meta : g[2].meta) : (p & 1 ? g[1].meta : g[0].meta);
      reinterpret_cast<uint32_t *>(at.meta)[p] = err ? 0x7FFF7FFFu : m;
    }
  }
}

// y^ = zf + q * sf, the butterfly, x 2^-log2 d, signs, one rounding (reading R9;
// zf and sf pre-scaled as in Dec::vector, which shows that this is exact).
template <int D, int G, int DT>
__global__ void __launch_bounds__(kRowThreads)
    cache_read_kernel(const __grid_constant__ CachePool c, const __grid_constant__ RowArgs r) {
  constexpr int NB = D / 32, N = D / 64;
  __shared__ alignas(16) uint32_t mask[D];
  const uint32_t lane = threadIdx.x & 31, p = lane & 3;
  const uint32_t t = blockIdx.x * kRowTok + (threadIdx.x >> 5) * 8 + (lane >> 2);
  const uint32_t slot = slot_of(r, c, t);
  for (uint32_t lkh = blockIdx.y; lkh < c.layers * 2 * c.heads; lkh += gridDim.y) {
    const uint32_t lk = lkh / c.heads, h = lkh - lk * c.heads, l = lk >> 1, kv = lk & 1;
    const Place<D, G> at(c, slot != ~0u ? slot : 0, l, kv, h);
    uint32_t w[NB], m[D / G];
#pragma unroll
    for (int b = 0; b < NB; ++b) w[b] = 0;
#pragma unroll
    for (int q = 0; q < D / G; ++q) m[q] = 0;
    if (slot != ~0u) {
      get_words<D>(at.codes, p, kv, w);
#pragma unroll
      for (int q = 0; q < D / G; ++q) m[q] = reinterpret_cast<const uint32_t *>(at.meta)[q];
    }
    if (lkh != blockIdx.y) __syncthreads();  // the masks before are read
    sign_table<D>(c, lkh, mask);
    __syncthreads();
    constexpr float up = 8.0f / float(D);
    float2 y[N][8];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const uint32_t ma = m[j * 32 / G], mb = m[(j + N) * 32 / G];
      const float2 sf = make_float2(__fmul_rn(__half2float(__ushort_as_half(uint16_t(ma))), up),
                                    __fmul_rn(__half2float(__ushort_as_half(uint16_t(mb))), up));
      const float2 zf =
          make_float2(__fmul_rn(__half2float(__ushort_as_half(uint16_t(ma >> 16))), up),
                      __fmul_rn(__half2float(__ushort_as_half(uint16_t(mb >> 16))), up));
      // a byte permute puts a code into the low byte of 1.5 * 2^23
      const float2 mag = make_float2(12582912.0f, 12582912.0f);
      const uint32_t ae = w[j] & 0x0F0F0F0Fu, ao = (w[j] >> 4) & 0x0F0F0F0Fu;
      const uint32_t be = w[j + N] & 0x0F0F0F0Fu, bo = (w[j + N] >> 4) & 0x0F0F0F0Fu;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t a = __byte_perm(i & 1 ? ao : ae, 0x4B400000u, 0x7640 | (i / 2));
        const uint32_t b = __byte_perm(i & 1 ? bo : be, 0x4B400000u, 0x7640 | (i / 2));
        const float2 q = sub2(make_float2(__uint_as_float(a), __uint_as_float(b)), mag);
        y[j][i] = fma2(q, sf, zf);
      }
    }
    fwht_lanes<D>(y, p);
    if (slot == ~0u) continue;
    uint8_t *row = kv ? r.v + int64_t(l) * r.v_l + int64_t(t) * r.v_t + int64_t(h) * r.v_h
                      : r.k + int64_t(l) * r.k_l + int64_t(t) * r.k_t + int64_t(h) * r.k_h;
    const uint4 *mk = reinterpret_cast<const uint4 *>(mask);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 e = y[b % N][2 * k], f = y[b % N][2 * k + 1];
        const float lo = b < N ? e.x : e.y, hi = b < N ? f.x : f.y;
        if constexpr (DT == KVC_BF16) {
          const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
          o[k] = *reinterpret_cast<const uint32_t *>(&x);
        } else {
          const __half2 x = __floats2half2_rn(lo, hi);
          o[k] = *reinterpret_cast<const uint32_t *>(&x);
        }
      }
      const uint4 f = mk[4 * b + p];
      *reinterpret_cast<uint4 *>(row + 64 * b + 16 * p) =
          make_uint4(o[0] ^ f.x, o[1] ^ f.y, o[2] ^ f.z, o[3] ^ f.w);
    }
  }
}

// Codes and meta of the stream's vectors to their tokens' slots. Every table
// entry that a vector relies on is checked by the lanes that use it: its code
// chunk raw and in place, its meta chunk raw inside the stream or eliminated
// (then expanded, and checked, by meta_expand_kernel).
__device__ __forceinline__ void load_error(const LoadArgs &a, uint32_t code) {
  set_status(a.d.status, code);
  note(a.note, code);
}
template <int D, int G>
__global__ void __launch_bounds__(kRowThreads)
    cache_load_kernel(const __grid_constant__ CachePool c, const __grid_constant__ LoadArgs a) {
  using C = Cfg<D, 4, G>;
  __shared__ uint64_t base_s;
  grid_dependency_wait();  // the meta expansion
  const uint8_t *in = a.d.in, *table = in + kHeader;
  // A thread checks the header; all warps but its own compare the requests' lengths at the
  // same time, where the table is if the header is right.
  bool bad = false;
  if (threadIdx.x == 0) {
    if (blockIdx.x == 0)
      if (const uint32_t e = *a.d.status) note(a.note, e);  // of the meta expansion
    const StreamHdr h = parse_header<D>(a.d);
    bool ok = h.ok && h.bits == 4 && h.group == a.group && h.quant <= 1 && !h.code_elim &&
              h.vec_signs == c.vec_signs && h.seed == c.seed &&
              h.data_base + uint64_t(a.d.V) * C::CB <= h.stream_bytes;
    bad = !ok;
    base_s = h.data_base;
  } else if (threadIdx.x >= 32 && a.table_fits) {
    for (uint32_t r = threadIdx.x - 32; r < a.d.n_req; r += kRowThreads - 32)
      bad |= ld_u32(in + a.tokens_at + 4 * r) != a.lens[r];
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) load_error(a, KVC_ERR_CORRUPT);
    return;
  }
  const uint64_t base = base_s, code_bytes = uint64_t(a.d.V) * C::CB;
  const uint64_t n_code = (code_bytes + kChunk - 1) / kChunk;
  const uint32_t lane = threadIdx.x & 31, p = lane & 3;
  const uint32_t T = uint32_t(a.d.tokens), lkhs = c.layers * 2 * c.heads;
  const uint64_t stream_bytes = ld_u64(in + 56);
  // 32 tokens of one (layer, kv, head) at a time (two such blocks in step: 5 us slower
  // in 73)
  const uint32_t tbs = (T + kRowTok - 1) / kRowTok, n = tbs * lkhs;
  for (uint32_t b = blockIdx.x; b < n; b += gridDim.x) {
    const uint32_t lkh = b / tbs, t = (b - lkh * tbs) * kRowTok + (threadIdx.x >> 5) * 8 + (lane >> 2);
    if (t >= T) continue;
    const int64_t s64 = __ldg(reinterpret_cast<const long long *>(a.slots) + t);
    if (s64 < 0) continue;
    if (s64 >= int64_t(c.slots)) {
      load_error(a, KVC_ERR_CORRUPT);
      continue;
    }
    const uint32_t lk = lkh / c.heads, h = lkh - lk * c.heads, l = lk >> 1, kv = lk & 1;
    const uint32_t v = lkh * T + t;
    const uint64_t ck = uint64_t(v) * C::CB / kChunk;
    const uint64_t e = ld_u64(table + 8 * ck), rest = code_bytes - ck * kChunk;
    const uint32_t ms = v / C::VM, mlen = min(uint32_t(C::VM), a.d.V - ms * C::VM) * C::MB;
    const uint64_t em = ld_u64(table + 8 * (n_code + ms));
    const bool raw = entry_size(em) == mlen;
    if (entry_size(e) != (rest < kChunk ? rest : uint64_t(kChunk)) || entry_pipe(e) != 0 ||
        entry_offset(e) != ck * kChunk ||
        (raw && (entry_pipe(em) != 0 || base + entry_offset(em) + mlen > stream_bytes))) {
      load_error(a, KVC_ERR_CORRUPT);
      continue;
    }
    const uint32_t *src = reinterpret_cast<const uint32_t *>(in + base + uint64_t(v) * C::CB);
    uint32_t w[D / 32];
#pragma unroll
    for (int b = 0; b < D / 32; ++b) w[b] = __ldg(src + 4 * b + p);
    const uint8_t *mp = (raw ? in + base + entry_offset(em) : a.d.ws_meta + uint64_t(ms) * kChunk) +
                        uint64_t(v - ms * C::VM) * C::MB;
    const Place<D, G> at(c, uint32_t(s64), l, kv, h);
    put_words<D>(at.codes, p, kv, w);
    if (p < uint32_t(C::NG))
      reinterpret_cast<uint32_t *>(at.meta)[p] = reinterpret_cast<const uint32_t *>(mp)[p];
  }
}

dim3 row_grid(const CachePool &c, uint32_t tokens) {
  const uint32_t lkh = c.layers * 2 * c.heads;
  return dim3((tokens + kRowTok - 1) / kRowTok, lkh < 65535u ? lkh : 65535u);
}

template <int D, int G>
cudaError_t write_t(int dtype, const CachePool &c, const RowArgs &r, cudaStream_t st) {
  if (dtype == KVC_BF16)
    cache_write_kernel<D, G, KVC_BF16><<<row_grid(c, r.tokens), kRowThreads, 0, st>>>(c, r);
  else
    cache_write_kernel<D, G, KVC_FP16><<<row_grid(c, r.tokens), kRowThreads, 0, st>>>(c, r);
  return cudaGetLastError();
}
template <int D, int G>
cudaError_t read_t(int dtype, const CachePool &c, const RowArgs &r, cudaStream_t st) {
  if (dtype == KVC_BF16)
    cache_read_kernel<D, G, KVC_BF16><<<row_grid(c, r.tokens), kRowThreads, 0, st>>>(c, r);
  else
    cache_read_kernel<D, G, KVC_FP16><<<row_grid(c, r.tokens), kRowThreads, 0, st>>>(c, r);
  return cudaGetLastError();
}
template <int D, int G>
cudaError_t load_t(const CachePool &c, const LoadArgs &a, int sms, cudaStream_t st) {
  // eliminated meta chunks into the workspace; after a memset, so in plain stream order
  auto mk = meta_expand_kernel<D>;
  struct MetaTag {};
  cudaError_t e = prepare<MetaTag>(mk, meta_smem_bytes());
  if (e != cudaSuccess) return e;
  const uint32_t mcap = uint32_t(kMetaCtas) * uint32_t(sms);
  const uint32_t n = a.d.ws_meta_chunks;
  mk<<<n == 0 ? 1u : (n < mcap ? n : mcap), kMetaThreads, meta_smem_bytes(), st>>>(a.d);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  // CTAs that go on to the next block: the header is checked once for each (with a CTA
  // per block, that took half the time of a large call)
  const uint64_t blocks = uint64_t((a.d.tokens + kRowTok - 1) / kRowTok) * (c.layers * 2 * c.heads);
  const uint64_t cap = uint64_t(sms) * 16;
  cfg.gridDim = dim3(unsigned(blocks == 0 ? 1 : blocks < cap ? blocks : cap));
  cfg.blockDim = dim3(kRowThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_load_kernel<D, G>, c, a);
}

}  // namespace

#define KVC_CACHE_DISPATCH(F, ...)                    \
  (d == 128 ? (g == 128  ? F<128, 128>(__VA_ARGS__)   \
               : g == 64 ? F<128, 64>(__VA_ARGS__)    \
                         : F<128, 32>(__VA_ARGS__))   \
            : (g == 64 ? F<64, 64>(__VA_ARGS__) : F<64, 32>(__VA_ARGS__)))

// Blocks of 32 tokens (kvc_cache_blocks.cuh) in a call, 0 where it has fewer than
// `least` per SM and the four-lane form is to run. Both forms, us, 8 heads: write d = 128,
// 28 blocks per SM 15.7 (lane per vector) against 14.6, 55: 24.4 / 27.3, 443: 143 /
// 195; write d = 64, 28: 9.9 / 11.0, 443: 87 / 135. Read d = 128, 55: 24.8 / 23.8, 111:
// 48.5 / 47.7, 443: 152 / 180; read d = 64, 28: 9.3 / 9.4, 443: 87 / 115.
static uint32_t row_blocks(const CachePool &c, const RowArgs &r, int sms, uint32_t least) {
  const uint64_t n = uint64_t((r.tokens + 31) / 32) * (c.layers * 2 * c.heads);
  return n >= uint64_t(least) * uint64_t(sms) && n < (uint64_t(1) << 31) ? uint32_t(n) : 0;
}

cudaError_t launch_cache_write(int d, int g, int dtype, const CachePool &c, const RowArgs &r,
                               int sms, cudaStream_t st) {
  if (const uint32_t n = row_blocks(c, r, sms, d == 128 ? 40 : 24))
    return d == 128 ? launch_cache_write_blocks_d128(g, dtype, c, r, n, sms, st)
                    : launch_cache_write_blocks_d64(g, dtype, c, r, n, sms, st);
  return KVC_CACHE_DISPATCH(write_t, dtype, c, r, st);
}
cudaError_t launch_cache_read(int d, int g, int dtype, const CachePool &c, const RowArgs &r,
                              int sms, cudaStream_t st) {
  if (const uint32_t n = row_blocks(c, r, sms, d == 128 ? 120 : 28))
    return d == 128 ? launch_cache_read_blocks_d128(g, dtype, c, r, n, sms, st)
                    : launch_cache_read_blocks_d64(g, dtype, c, r, n, sms, st);
  return KVC_CACHE_DISPATCH(read_t, dtype, c, r, st);
}
cudaError_t launch_cache_load(int d, int g, const CachePool &c, const LoadArgs &a, int sms,
                              cudaStream_t st) {
  return KVC_CACHE_DISPATCH(load_t, c, a, sms, st);
}

}  // namespace kvc
