// Codes of the 8-bit per-head cache, and which request a block of new tokens belongs to: what the kernels
// that write the cache share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv8.h"
#include "ptx.cuh"

namespace nvfp4mla {
namespace {

using namespace ptx;

// Two 16-bit elements (low half first) -> fp32.
template <bool kHalf>
__device__ __forceinline__ float2 widen(uint32_t w) {
  if constexpr (kHalf) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Two elements as E4M3 of x * mul: nearest even, saturating; kNan: a NaN as 0x7F with its own sign.
template <bool kHalf, bool kNan>
__device__ __forceinline__ uint32_t encode2(uint32_t w, float mul) {
  const float2 x = widen<kHalf>(w);
  uint32_t r = f32x2_to_e4m3x2(x.x * mul, x.y * mul);
  if constexpr (kNan) {
    constexpr uint32_t kInf = kHalf ? 0x7C00u : 0x7F80u;
    const uint32_t lo = w & 0xFFFFu, hi = w >> 16;
    if ((lo & 0x7FFFu) > kInf) r = (r & 0xFF00u) | 0x7Fu | ((lo >> 8) & 0x80u);
    if ((hi & 0x7FFFu) > kInf) r = (r & 0x00FFu) | ((0x7Fu | ((hi >> 8) & 0x80u)) << 8);
  }
  return r;
}
template <bool kHalf, bool kNan>
__device__ __forceinline__ uint2 encode8(const uint4& x, float mul) {
  return make_uint2(__byte_perm(encode2<kHalf, kNan>(x.x, mul), encode2<kHalf, kNan>(x.y, mul), 0x5410),
                    __byte_perm(encode2<kHalf, kNan>(x.z, mul), encode2<kHalf, kNan>(x.w, mul), 0x5410));
}

// Largest magnitude (its 16 bits) of four pairs; kFinite: of the finite ones. Magnitudes order as their
// bits do, infinities and NaN above all.
template <bool kHalf, bool kFinite>
__device__ __forceinline__ uint32_t top8(const uint4& x, uint32_t top) {
  constexpr uint32_t kInf2 = kHalf ? 0x7C007C00u : 0x7F807F80u;
  const uint32_t ws[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t a = ws[k] & 0x7FFF7FFFu;
    if constexpr (kFinite) a &= __vcmpltu2(a, kInf2);
    top = __vmaxu2(top, a);
  }
  return top;
}

// Two codes times mul (a power of two of at most 1), as codes; NaN codes stay.
__device__ __forceinline__ uint32_t shrink2(uint32_t two, float mul) {
  const uint32_t h = e4m3x2_to_f16x2(two);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
  uint32_t r = f32x2_to_e4m3x2(x.x * mul, x.y * mul);
  if ((two & 0x7Fu) == 0x7Fu) r = (r & 0xFF00u) | (two & 0xFFu);
  if ((two & 0x7F00u) == 0x7F00u) r = (r & 0x00FFu) | (two & 0xFF00u);
  return r;
}

// First block slot of request b: the slots of requests do not overlap, as a request of n tokens
// touches at most floor((n + 30) / 16) blocks and gets at least floor(n / 16) + 2 slots.
__device__ __forceinline__ int first_slot(const AppendParams& p, int b) {
  const int c = __ldg(p.cu + b);
  return (c < 0 ? 0 : (c > (int)p.num_tokens ? (int)p.num_tokens : c)) / kBlockTokens + 2 * b;
}

// The last request whose first slot is not behind `slot`: a warp, 32 probes a round.
__device__ __forceinline__ int request_of(const AppendParams& p, int slot) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5;
    const int at = lo + lane * step;
    const unsigned yes = __ballot_sync(0xFFFFFFFFu, at < hi && first_slot(p, at) <= slot) | 1u;
    const int k = 31 - __clz(yes);
    lo += k * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// The byte of the smallest scale 2^(e - 127) that takes amax (finite, not negative) to at most 448.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  // amax = m 2^t, 1 <= m < 2, and 448 = 1.75 x 2^8
  const uint32_t bits = __float_as_uint(amax);
  return (uint32_t)max((int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0), 1);
}

// How a warp holds rows of D 16-bit values: 16 bytes a lane.
template <int D>
struct Rows {
  static constexpr int kLanes = D / 8;              // lanes per row, 8 values each
  static constexpr int kAtOnce = 32 / kLanes;       // rows per load
  static constexpr int kLoads = kBlockTokens / kAtOnce;   // of a block
};

// The block's scale grew from `before` to e: the codes of its tokens from before, rows 0 .. first - 1, are
// rounded again. (codes: this lane's eight columns of the block.)
template <int D>
__device__ __forceinline__ void shrink_rows(uint8_t* codes, int row0, int first, uint32_t before, uint32_t e) {
  const float less = __uint_as_float((127u - min(e - before, 126u)) << 23);
#pragma unroll 1
  for (int row = row0; row < first; row += Rows<D>::kAtOnce) {
    uint2* at = reinterpret_cast<uint2*>(codes + row * D);
    const uint2 c = *at;
    *at = make_uint2(shrink2(c.x & 0xFFFFu, less) | (shrink2(c.x >> 16, less) << 16),
                     shrink2(c.y & 0xFFFFu, less) | (shrink2(c.y >> 16, less) << 16));
  }
}

// Rows first .. behind - 1 of a block of one head into its codes and scale byte; w: the rows, zeros elsewhere.
template <int D, bool kHalf>
__device__ __forceinline__ void put_block(const uint4 (&w)[Rows<D>::kLoads], int row0, int first, int behind, uint32_t before,
                                          uint8_t* codes, uint8_t* scale) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < Rows<D>::kLoads; ++i) top = top8<kHalf, false>(w[i], top);
  top = __reduce_max_sync(0xFFFFFFFFu, max(top & 0xFFFFu, top >> 16));
  // blocks with an infinity or a NaN are rare, and cost three times the instructions
  const bool finite = top < (kHalf ? 0x7C00u : 0x7F80u);
  if (!finite) {
    top = 0;
#pragma unroll
    for (int i = 0; i < Rows<D>::kLoads; ++i) top = top8<kHalf, true>(w[i], top);
    top = __reduce_max_sync(0xFFFFFFFFu, max(top & 0xFFFFu, top >> 16));
  }
  const uint32_t e = max(scale_byte(widen<kHalf>(top).x), before);
  const float mul = __uint_as_float((254u - e) << 23);
#pragma unroll
  for (int i = 0; i < Rows<D>::kLoads; ++i) {
    const int row = i * Rows<D>::kAtOnce + row0;
    if (row >= first && row < behind)
      *reinterpret_cast<uint2*>(codes + row * D) = finite ? encode8<kHalf, false>(w[i], mul) : encode8<kHalf, true>(w[i], mul);
  }
  if (first > 0 && e > before) shrink_rows<D>(codes, row0, first, before, e);
  if ((threadIdx.x & 31) == 0) *scale = (uint8_t)e;
}

}  // namespace
}  // namespace nvfp4mla
