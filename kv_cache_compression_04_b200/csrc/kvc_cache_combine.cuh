// What the two forms of the cache's attention share (kvc_cache_attend.cuh, few query
// rows per request; kvc_cache_prefill.cuh, more): the requests' numbers, searches in
// prefixes, and the kernel that merges a row's records.
#pragma once

#include "kvc_attend_mma.cuh"
#include "kvc_cache.h"
#include "kvc_launch.cuh"

namespace kvc {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// How both forms keep a row's weights in fp16's range. All sums of a row hold p = 2^(score + n)
// (scores in base 2); the value product's weights are p s, s the values' scales (or 2^e). n
// follows the weights, not the scores: the first keys bring the largest p s to
// 2^kWeightTop, n stands while p s <= 2^kWeightMost (a bound from the largest score and the
// largest scale, both at hand, shows that), and then comes down to 2^kWeightTop again. Where a
// tile's scales lie within 2^3, the largest score and scale stand for the largest p s. So
// the largest weight so far is 2 at least, and rounding small ones (to 2^-25) costs
// 2^-26 of it: values of any sizes keep their precision beside one another. (With a factor
// from the largest scale alone, one visible value of 2^20 times the others' and no
// weight pushed their weights into the subnormals: errors of 1.6e-3, at 2^24 of 0.11.) p itself
// is kept below 2^kPMost: sums of 2^31 of them, times zeros, stay in fp32's range.
constexpr float kWeightTop = 5.f, kWeightMost = 14.f, kPTop = 60.f, kPMost = 64.f;
// The new n of a row that sees keys: x its largest score, w log2 of its largest p s but for
// n (-inf: none), first: no keys before.
__device__ __forceinline__ float row_factor(float n, float x, float w, bool first) {
  if (first || w + n > kWeightMost) n = kWeightTop - w;
  return fminf(n, kPTop - x);
}
// floor(log2 x) of a float's bits (0: -127)
__device__ __forceinline__ float log2_floor(uint32_t bits) { return float(int(bits >> 23) - 127); }
__device__ __forceinline__ float half_lo(uint32_t m) {
  return __half2float(__ushort_as_half(uint16_t(m)));
}
__device__ __forceinline__ float half_hi(uint32_t m) {
  return __half2float(__ushort_as_half(uint16_t(m >> 16)));
}

// n - kFrom of the codes n in bits 0..3 (kHigh: 4..7) of both halves, as fp16 pairs.
template <bool kHigh, int kFrom>
__device__ __forceinline__ uint32_t codes_less(uint32_t x) {
  constexpr uint32_t one = kHigh ? 0x5400u + 16 * kFrom : 0x6400u + kFrom;  // 64 (1024) + kFrom
  uint32_t t, d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;"
      : "=r"(t)
      : "r"(x), "n"(kHigh ? 0x00F000F0 : 0x000F000F), "n"(kHigh ? 0x54005400 : 0x64006400));
  asm("sub.f16x2 %0, %1, %2;" : "=r"(d) : "r"(t), "r"(one << 16 | one));
  return d;
}
template <bool kHigh>
__device__ __forceinline__ uint32_t centred(uint32_t x) {
  return codes_less<kHigh, 8>(x);
}
// Whether a meta word's scale or zero is infinite or NaN.
__device__ __forceinline__ bool not_finite(uint32_t m) {
  return (m & 0x7C00u) == 0x7C00u || (m & 0x7C000000u) == 0x7C000000u;
}
// A meta word's z + 8 s.
__device__ __forceinline__ float zero8(uint32_t m) { return fmaf(8.f, half_lo(m), half_hi(m)); }

// A request from the host's limits and its device numbers: queries, their first
// row, keys. One out of range has no queries.
struct ReqShape {
  uint32_t nq, q0, len;
};
// From the caller's arrays; ok: in range.
__device__ __forceinline__ ReqShape read_request(const CacheAttnArgs &a, uint32_t r, bool &ok) {
  const int64_t q0 = a.q_starts ? int64_t(__ldg(a.q_starts + r)) : int64_t(r);
  const int64_t q1 = a.q_starts ? int64_t(__ldg(a.q_starts + r + 1)) : int64_t(r) + 1;
  const int64_t len = __ldg(a.seq_lens + r);
  ok = q0 >= 0 && q1 >= q0 && q1 <= int64_t(a.q_tokens) && q1 - q0 <= int64_t(a.max_q) &&
       len >= 0 && len <= int64_t(a.max_len);
  return ok ? ReqShape{uint32_t(q1 - q0), uint32_t(q0), uint32_t(len)} : ReqShape{};
}
// From the first kernel's copy in the workspace.
__device__ __forceinline__ ReqShape request_shape(const CacheAttnArgs &a, uint32_t r) {
  const uint4 v = a.shapes[r];
  return ReqShape{v.x, v.y, v.z};
}
// Keys [lo, hi) that query i of a request sees.
__device__ __forceinline__ void key_range(const CacheAttnArgs &a, const ReqShape &s, uint32_t i,
                                          int32_t &lo, int32_t &hi) {
  const int64_t end = a.causal ? int64_t(s.len) - int64_t(s.nq) + int64_t(i) + 1 : int64_t(s.len);
  const int64_t beg = a.window ? end - int64_t(a.window) : 0;
  hi = int32_t(end > 0 ? end : 0);
  lo = int32_t(beg > 0 ? beg : 0);
}

// a / b, in 32 bits where they suffice (most calls).
__device__ __forceinline__ uint64_t div64(uint64_t a, uint64_t b) {
  return ((a | b) >> 32) == 0 ? uint64_t(uint32_t(a) / uint32_t(b)) : a / b;
}
// The largest r < n with in(r), for an in() that is true up to some r and false
// after it (0 if it is false at once). The warp looks at 32 places at a time.
template <class In>
__device__ __forceinline__ uint32_t last_with(uint32_t n, In in) {
  const uint32_t lane = threadIdx.x & 31;
  uint32_t lo = 0, len = n;
  while (len > 1) {
    const uint32_t step = (len + 31) / 32, p = lane * step;
    const uint32_t yes = __ballot_sync(0xFFFFFFFFu, p < len && in(lo + p));
    const uint32_t k = yes ? 31 - __clz(yes) : 0;
    lo += k * step;
    len = min(step, len - k * step);
  }
  return lo;
}

// Brings sums (L, y) under maximum M to maximum top >= M.
__device__ __forceinline__ void merge_scale(float &M, float &L, float top, float (&y)[4]) {
  if (M != -INFINITY && M != top) {
    const float k = ex2(M - top);
    L *= k;
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] *= k;
  }
  M = top;
}

// A row's records in turn, or split between WPR warps (few units, many records
// each): their merge, then S H / d.
// At: where a row's records are (a decode unit, or a block of a prompt's rows).
template <int D, class At, int DT, int WPR>
__global__ void __launch_bounds__(WPR == 1 ? 128 : WPR * 32)
    cache_combine_kernel(const __grid_constant__ CacheAttnArgs a, const uint32_t grid) {
  constexpr int W = D / 32;
  __shared__ float part[WPR == 1 ? 1 : WPR][WPR == 1 ? 1 : D];
  __shared__ float2 ml[WPR];
  grid_dependency_wait();  // the records and the prefixes
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, H = a.c.heads, Hq = H * a.qpk;
  const uint64_t i = WPR == 1 ? uint64_t(blockIdx.x) * 4 + warp : uint64_t(blockIdx.x);
  if (i >= uint64_t(a.c.layers) * a.q_tokens * Hq) return;
  const uint32_t n = a.n_req;
  const uint64_t lt = div64(i, Hq);
  const uint32_t j = uint32_t(i - lt * Hq), l = uint32_t(div64(lt, a.q_tokens));
  const uint32_t tok = uint32_t(lt - uint64_t(l) * a.q_tokens);
  uint32_t r = tok;
  if (a.q_starts) r = last_with(n + 1, [&](uint32_t x) { return __ldg(a.q_starts + x) <= int32_t(tok); });
  if (r >= n) return;
  const ReqShape rs = request_shape(a, r);
  if (tok < rs.q0 || tok - rs.q0 >= rs.nq) return;  // a row that no request names
  const uint32_t h = j / a.qpk, row = (tok - rs.q0) * a.qpk + (j - h * a.qpk);
  float y[4] = {0.f, 0.f, 0.f, 0.f}, M = -INFINITY, L = 0.f;
  const At at(a, grid, rs, l, h, r, row);
  constexpr uint32_t kStep = At::COLS * (4 + D);
  {
    const float *p0 = a.rec + at.unit * uint64_t(kStep) + at.row * (4 + D);
    // four records at a time: their loads first, then the running maximum and sums
    for (uint32_t k0 = WPR == 1 ? 0 : 4 * warp; k0 < at.nrec; k0 += 4 * WPR) {
      float2 v[4];
      float o[4][W];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool in = k0 + e < at.nrec;
        const float *p = p0 + uint64_t(at.id(in ? k0 + e : k0)) * kStep;
        v[e] = in ? *reinterpret_cast<const float2 *>(p) : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int c = 0; c < W; ++c) o[e][c] = p[4 + lane + 32 * c];
      }
      const float top = fmaxf(M, fmaxf(fmaxf(v[0].x, v[1].x), fmaxf(v[2].x, v[3].x)));
      merge_scale(M, L, top, y);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (v[e].x == -INFINITY && v[e].y == 0.f) continue;  // no key of this row in the segment
        const float w = v[e].x == -INFINITY ? 1.f : ex2(v[e].x - top);
        L = fmaf(w, v[e].y, L);
#pragma unroll
        for (int c = 0; c < W; ++c) y[c] = fmaf(w, o[e][c], y[c]);
      }
    }
  }
  if constexpr (WPR > 1) {  // in the warps' order
#pragma unroll
    for (int c = 0; c < W; ++c) part[warp][lane + 32 * c] = y[c];
    if (lane == 0) ml[warp] = make_float2(M, L);
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int w = 1; w < WPR; ++w) M = fmaxf(M, ml[w].x);
    L = 0.f;
#pragma unroll
    for (int c = 0; c < W; ++c) y[c] = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      const float2 v = ml[w];
      if (v.x == -INFINITY && v.y == 0.f) continue;
      const float k = v.x == -INFINITY ? 1.f : ex2(v.x - M);
      L = fmaf(k, v.y, L);
#pragma unroll
      for (int c = 0; c < W; ++c) y[c] = fmaf(k, part[w][lane + 32 * c], y[c]);
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


// dtype, and whether records are spread wide (eight warps a row; where At asks for it).
template <int D, class At>
cudaError_t launch_combine(int dtype, bool wide, const CacheAttnArgs &a, uint32_t grid,
                           cudaStream_t st) {
  const uint64_t rows = uint64_t(a.c.layers) * a.q_tokens * a.c.heads * a.qpk;
  const uint64_t cg = wide ? rows : (rows + 3) / 4;  // (below 2^31: checked before the first kernel)
  auto ck = dtype == KVC_BF16 ? cache_combine_kernel<D, At, KVC_BF16, 1>
                              : cache_combine_kernel<D, At, KVC_FP16, 1>;
  if constexpr (At::kWide)
    if (wide)
      ck = dtype == KVC_BF16 ? cache_combine_kernel<D, At, KVC_BF16, 8>
                             : cache_combine_kernel<D, At, KVC_FP16, 8>;
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

}  // namespace kvc
