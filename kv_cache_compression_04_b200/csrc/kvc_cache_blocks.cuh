// Writing and reading many rows of the paged 4-bit cache: a lane per vector, as the
// codec's encoder and decoder hold them (Pairs), a warp per block of 32 tokens of one
// (layer, kv, head). No shuffles, and each group's scale computed once, where the form
// with four lanes per vector (kvc_cache_rows.cu) shuffles half a vector twice and
// computes scales four times over; but a lane's chain is four times as long, so few
// rows are left to that form.
//
// A block's rows are 32 tokens apart by the token stride: 16-byte pieces go through
// the warp's swizzled buffer, half a warp per row, the next block's while this one
// is computed.
//
// Measured: 4096 tokens x 32 layers written in 145 us (0.72 of the copy rate), read in 153
// (0.69). Neither unit is full: issue slots 63% used (written) and 66% (read), the integer
// pipe 47% and 57%, DRAM 54% and 48%; the three warps of an SM quarter, all that 168 registers
// a lane leave, spend their time on one another's instructions and on results of their own.
#pragma once

#include "kvc_cache_rows.cuh"

namespace kvc {

constexpr int kBlkWarps = 12;  // per CTA, one CTA per SM: a lane's vector takes up to 168 registers
constexpr int kBlkThreads = kBlkWarps * 32;
template <int D>
constexpr size_t blk_smem() {
  return size_t(kBlkWarps) * D / 64 * 4096;
}

struct SignMasks {
  uint32_t mask[64], lo[64];  // of channel pairs, and << 16 (GlobalSigns)
};

// Block b of the call: tokens 32 tb .. + 31 of (layer, kv, head) lkh; heads first, so
// that warps at work together read rows next to one another.
struct BlockAt {
  uint32_t tb, lkh, l, kv, h;
  __device__ __forceinline__ BlockAt(const CachePool &c, uint32_t b) {
    const uint32_t n = c.layers * 2 * c.heads;
    tb = b / n;
    lkh = b - tb * n;
    const uint32_t lk = lkh / c.heads;
    h = lkh - lk * c.heads;
    l = lk >> 1;
    kv = lk & 1;
  }
  __device__ __forceinline__ uint8_t *row(const RowArgs &r, uint32_t t) const {
    return kv ? r.v + int64_t(l) * r.v_l + int64_t(t) * r.v_t + int64_t(h) * r.v_h
              : r.k + int64_t(l) * r.k_l + int64_t(t) * r.k_t + int64_t(h) * r.k_h;
  }
};

// The block's rows to the warp's buffer (tokens past the end: the last one again).
template <int D>
__device__ __forceinline__ void load_block(const RowArgs &r, const BlockAt &at, uint8_t *buf) {
  constexpr int P = D / 8, RPI = 32 / P;
  const int lane = threadIdx.x & 31, c = lane % P, rs = lane / P;
  const uint8_t *base = at.row(r, 0) + 16 * c;
  const int64_t s = at.kv ? r.v_t : r.k_t;
#pragma unroll
  for (int i = 0; i < 32 / RPI; ++i) {
    const uint32_t t = min(at.tb * 32 + i * RPI + rs, r.tokens - 1);
    cp_async16_s(smem_u32(buf + swz_offset(i * RPI + rs, c)), base + int64_t(t) * s);
  }
  cp_async_commit();
}

// This lane's row from the buffer: fp32, signs flipped, pairs (c, c + D / 2).
template <int D, int DT, class SG>
__device__ __forceinline__ void widen_row(const uint8_t *buf, const SG &sg, Pairs<D> &y) {
  const int row = threadIdx.x & 31;
#pragma unroll
  for (int q = 0; q < D / 16; ++q) {
    const uint4 va = *reinterpret_cast<const uint4 *>(buf + swz_offset(row, q));
    const uint4 vb = *reinterpret_cast<const uint4 *>(buf + swz_offset(row, q + D / 16));
    const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int k = 4 * q + e;
      if constexpr (DT == KVC_BF16) {
        y.p[2 * k] = make_float2(__uint_as_float((wa[e] << 16) + sg.lo(k)),
                                 __uint_as_float((wb[e] << 16) + sg.lo(k + D / 4)));
        y.p[2 * k + 1] = make_float2(__uint_as_float((wa[e] ^ sg.word(k)) & 0xFFFF0000u),
                                     __uint_as_float((wb[e] ^ sg.word(k + D / 4)) & 0xFFFF0000u));
      } else {
        const uint32_t a = wa[e] ^ sg.word(k), b = wb[e] ^ sg.word(k + D / 4);
        y.p[2 * k] = make_float2(__half2float(__ushort_as_half(uint16_t(a))),
                                 __half2float(__ushort_as_half(uint16_t(b))));
        y.p[2 * k + 1] = make_float2(__half2float(__ushort_as_half(uint16_t(a >> 16))),
                                     __half2float(__ushort_as_half(uint16_t(b >> 16))));
      }
    }
  }
}

template <int D, int G, int DT, bool kVec>
__global__ void __launch_bounds__(kBlkThreads, 1)
    cache_write_blocks_kernel(const __grid_constant__ CachePool c, const __grid_constant__ RowArgs r,
                              const __grid_constant__ SignMasks sm, const uint32_t blocks) {
  using E = Enc<D, 4, G>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint8_t *buf = smem + warp * (D / 64 * 4096);
  const uint32_t step = gridDim.x * kBlkWarps;
  uint32_t b = blockIdx.x * kBlkWarps + warp;
  if (b < blocks) load_block<D>(r, BlockAt(c, b), buf);
  for (; b < blocks; b += step) {
    const BlockAt at(c, b);
    const uint32_t slot = slot_of(r, c, at.tb * 32 + lane);
    cp_async_wait_all();
    __syncwarp();
    Pairs<D> y;
    if constexpr (kVec) {
      VectorSigns<D> sg;
      vec_sign_words<D>(c.seed, at.lkh, sg.S);
      widen_row<D, DT>(buf, sg, y);
    } else {
      widen_row<D, DT>(buf, GlobalSigns{sm.mask, sm.lo}, y);
    }
    __syncwarp();  // every lane has its row
    if (b + step < blocks) load_block<D>(r, BlockAt(c, b + step), buf);
    uint32_t code[D / 8], meta[D / G];
    const uint32_t err = E::vector(y, code, meta, r.one, c.sym);
    if (slot == ~0u) continue;
    if (err) {
      note(r.status, (err & 1u) ? KVC_ERR_NONFINITE : KVC_ERR_RANGE);
#pragma unroll
      for (int k = 0; k < D / 8; ++k) code[k] = 0;  // (both forms store the same)
    }
    const Place<D, G> pl(c, slot, at.l, at.kv, at.h);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      uint32_t w[D / 32];
#pragma unroll
      for (int k = 0; k < D / 32; ++k) w[k] = code[4 * k + p];
      put_words<D>(pl.codes, p, at.kv, w);
    }
    put_meta<D / G>(pl.meta, meta, err != 0);
  }
}

// Codes and meta of this lane's slot (none: zeros).
template <int D, int G>
struct StoredRow {
  uint32_t w[4][D / 32], m[D / G];
  __device__ __forceinline__ void get(const CachePool &c, const BlockAt &at, uint32_t slot) {
#pragma unroll
    for (int q = 0; q < D / G; ++q) m[q] = 0;
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int k = 0; k < D / 32; ++k) w[p][k] = 0;
    if (slot == ~0u) return;
    const Place<D, G> pl(c, slot, at.l, at.kv, at.h);
#pragma unroll
    for (int p = 0; p < 4; ++p) {  // as stored
      if constexpr (D == 128) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(pl.codes) + p);
        w[p][0] = v.x, w[p][1] = v.y, w[p][2] = v.z, w[p][3] = v.w;
      } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(pl.codes) + p);
        w[p][0] = v.x, w[p][1] = v.y;
      }
    }
#pragma unroll
    for (int q = 0; q < D / G; ++q) m[q] = __ldg(reinterpret_cast<const uint32_t *>(pl.meta) + q);
  }
  // word 4 k + p of the row in channel order
  __device__ __forceinline__ uint32_t word(int k, int p, uint32_t kv) const {
    if constexpr (D == 128) {
      const uint32_t a = w[p][k / 2], b = w[p][2 + k / 2];
      return kv ? __byte_perm(a, b, k & 1 ? 0x7632 : 0x5410) : w[p][k];
    } else {
      return kv ? __byte_perm(w[p][0], w[p][1], k & 1 ? 0x7632 : 0x5410) : w[p][k];
    }
  }
};

// y^ = zf + q * sf, the butterfly, x 2^-log2 d, signs, one rounding: reading R9 with zf
// and sf pre-scaled, as in Dec::vector, which shows that this is exact.
template <int D, int G, int DT, bool kVec>
__global__ void __launch_bounds__(kBlkThreads, 1)
    cache_read_blocks_kernel(const __grid_constant__ CachePool c, const __grid_constant__ RowArgs r,
                             const __grid_constant__ SignMasks sm, const uint32_t blocks) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint8_t *buf = smem + warp * (D / 64 * 4096);
  const uint32_t step = gridDim.x * kBlkWarps;
  constexpr float up = 8.0f / float(D);
  constexpr int P = D / 8, RPI = 32 / P;
  uint32_t b = blockIdx.x * kBlkWarps + warp;
  if (b >= blocks) return;
  StoredRow<D, G> row;
  uint32_t slot;
  {
    const BlockAt at(c, b);
    slot = slot_of(r, c, at.tb * 32 + lane);
    row.get(c, at, slot);
  }
  for (; b < blocks; b += step) {
    const BlockAt at(c, b);
    Pairs<D> y;
    const float2 mag = make_float2(12582912.0f, 12582912.0f);
#pragma unroll
    for (int k = 0; k < D / 64; ++k)
#pragma unroll
      for (int p = 0; p < 4; ++p) {  // channels 32 k + 8 p .., and D / 2 on
        const uint32_t wa = row.word(k, p, at.kv), wb = row.word(k + D / 64, p, at.kv);
        const uint32_t ae = wa & 0x0F0F0F0Fu, ao = (wa >> 4) & 0x0F0F0F0Fu;
        const uint32_t be = wb & 0x0F0F0F0Fu, bo = (wb >> 4) & 0x0F0F0F0Fu;
        const uint32_t ma = row.m[(32 * k) / G], mb = row.m[(32 * k + D / 2) / G];
        const float2 sf = make_float2(__fmul_rn(__half2float(__ushort_as_half(uint16_t(ma))), up),
                                      __fmul_rn(__half2float(__ushort_as_half(uint16_t(mb))), up));
        const float2 zf =
            make_float2(__fmul_rn(__half2float(__ushort_as_half(uint16_t(ma >> 16))), up),
                        __fmul_rn(__half2float(__ushort_as_half(uint16_t(mb >> 16))), up));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t a = __byte_perm(i & 1 ? ao : ae, 0x4B400000u, 0x7640 | (i / 2));
          const uint32_t bb = __byte_perm(i & 1 ? bo : be, 0x4B400000u, 0x7640 | (i / 2));
          const float2 q = sub2(make_float2(__uint_as_float(a), __uint_as_float(bb)), mag);
          y.p[32 * k + 8 * p + i] = fma2(q, sf, zf);
        }
      }
    // the next block's rows, while this one is computed
    const uint32_t keep = __ballot_sync(0xFFFFFFFFu, slot != ~0u);
    if (b + step < blocks) {
      const BlockAt nx(c, b + step);
      slot = slot_of(r, c, nx.tb * 32 + lane);
      row.get(c, nx, slot);
    }
    fwht_pairs<D>(y);
    auto emit = [&](const auto &sg) {
#pragma unroll
      for (int q = 0; q < D / 8; ++q) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = 4 * q + e;
          if constexpr (DT == KVC_BF16) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(y.at(2 * k), y.at(2 * k + 1));
            o[e] = *reinterpret_cast<const uint32_t *>(&x) ^ sg.word(k);
          } else {
            const __half2 x = __floats2half2_rn(y.at(2 * k), y.at(2 * k + 1));
            o[e] = *reinterpret_cast<const uint32_t *>(&x) ^ sg.word(k);
          }
        }
        *reinterpret_cast<uint4 *>(buf + swz_offset(lane, q)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    };
    if constexpr (kVec) {
      VectorSigns<D> sg;
      vec_sign_words<D>(c.seed, at.lkh, sg.S);
      emit(sg);
    } else {
      emit(GlobalSigns{sm.mask, sm.lo});
    }
    __syncwarp();
    const int pc = lane % P, rs = lane / P;
    uint8_t *base = at.row(r, 0) + 16 * pc;
    const int64_t s = at.kv ? r.v_t : r.k_t;
#pragma unroll
    for (int i = 0; i < 32 / RPI; ++i) {
      const int x = i * RPI + rs;
      const uint4 v = *reinterpret_cast<const uint4 *>(buf + swz_offset(x, pc));
      if ((keep >> x) & 1u)
        *reinterpret_cast<uint4 *>(base + int64_t(at.tb * 32 + x) * s) = v;
    }
    __syncwarp();  // the buffer is read
  }
}

inline SignMasks cache_sign_masks(const CachePool &c, int d) {
  SignMasks m{};
  if (!c.vec_signs) sign_masks(c.seed, d, m.mask);
  for (int k = 0; k < 64; ++k) m.lo[k] = m.mask[k] << 16;
  return m;
}

template <int D, int G, int DT, bool kVec, bool kWrite>
cudaError_t launch_blocks_v(const CachePool &c, const RowArgs &r, uint32_t blocks, int sms,
                            cudaStream_t st) {
  auto pick = [] {
    if constexpr (kWrite) return &cache_write_blocks_kernel<D, G, DT, kVec>;
    else return &cache_read_blocks_kernel<D, G, DT, kVec>;
  };
  auto k = pick();
  struct Tag {};
  cudaError_t e = prepare<Tag>(k, blk_smem<D>());
  if (e != cudaSuccess) return e;
  const uint32_t want = (blocks + kBlkWarps - 1) / kBlkWarps;
  k<<<want < uint32_t(sms) ? want : uint32_t(sms), kBlkThreads, blk_smem<D>(), st>>>(
      c, r, cache_sign_masks(c, D), blocks);
  return cudaGetLastError();
}
template <int D, int G, bool kWrite>
cudaError_t launch_blocks(int dtype, const CachePool &c, const RowArgs &r, uint32_t blocks, int sms,
                          cudaStream_t st) {
  if (dtype == KVC_BF16)
    return c.vec_signs ? launch_blocks_v<D, G, KVC_BF16, true, kWrite>(c, r, blocks, sms, st)
                       : launch_blocks_v<D, G, KVC_BF16, false, kWrite>(c, r, blocks, sms, st);
  return c.vec_signs ? launch_blocks_v<D, G, KVC_FP16, true, kWrite>(c, r, blocks, sms, st)
                     : launch_blocks_v<D, G, KVC_FP16, false, kWrite>(c, r, blocks, sms, st);
}

}  // namespace kvc
