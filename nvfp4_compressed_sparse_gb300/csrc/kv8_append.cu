// kv8_append: new keys and values into the 8-bit per-head cache.
//
// A warp takes one block of 16 tokens of one head's keys or values. It finds its request and block
// from its number, reads the block's new rows (all loads issued before any is used), takes the
// largest finite magnitude, and from it the block's exponent; the codes are x 2^(127 - e) rounded
// to E4M3, exact but for that one rounding, since a power of two moves no mantissa bit.
//
// The floor is the traffic, three bytes per value (two in, one out). Consecutive warps take
// consecutive heads of the same tokens, so that a token's row of all heads is read in one piece.
#include <cuda_fp16.h>

#include "../../include/nvfp4mla.h"
#include "kv8.h"
#include "ptx.cuh"

namespace nvfp4mla {
namespace {

using namespace ptx;

constexpr int kAppendThreads = 256;

// Two 16-bit elements (low half first) -> fp32.
template <bool kHalf>
__device__ __forceinline__ float2 widen(uint32_t w) {
  if constexpr (kHalf) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Two elements as E4M3 of x * mul: nearest even, saturating, NaN as 0x7F with its own sign.
template <bool kHalf>
__device__ __forceinline__ uint32_t encode2(uint32_t w, float mul) {
  const float2 x = widen<kHalf>(w);
  uint32_t r = f32x2_to_e4m3x2(x.x * mul, x.y * mul);
  constexpr uint32_t kInf = kHalf ? 0x7C00u : 0x7F80u;
  const uint32_t lo = w & 0xFFFFu, hi = w >> 16;
  if ((lo & 0x7FFFu) > kInf) r = (r & 0xFF00u) | 0x7Fu | ((lo >> 8) & 0x80u);
  if ((hi & 0x7FFFu) > kInf) r = (r & 0x00FFu) | ((0x7Fu | ((hi >> 8) & 0x80u)) << 8);
  return r;
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
__device__ __forceinline__ int64_t first_slot(const AppendParams& p, int b) {
  const int64_t c = p.cu[b];
  return (c < 0 ? 0 : (c > p.num_tokens ? p.num_tokens : c)) / kBlockTokens + 2 * (int64_t)b;
}

template <int D, bool kHalf>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
  constexpr int kLanes = D / 8;              // lanes per row, 8 values (16 bytes) each
  constexpr int kRows = 32 / kLanes;         // rows per load
  constexpr int kLoads = kBlockTokens / kRows;
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int64_t slot = item / (2 * p.kv_heads);
  if (slot >= p.slots) return;
  const int part = (int)(item - slot * (2 * p.kv_heads));
  const int which = part >= p.kv_heads ? 1 : 0, head = part - which * p.kv_heads;

  // the last request whose first slot is not behind this one: 32 probes a round
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5;
    const int at = lo + lane * step;
    const unsigned yes = __ballot_sync(0xFFFFFFFFu, at < hi && first_slot(p, at) <= slot) | 1u;
    const int k = 31 - __clz(yes);
    lo += k * step;
    hi = min(hi, lo + step);
  }
  const int b = lo;
  const int64_t c0 = p.cu[b], c1 = p.cu[b + 1];
  const int64_t nth = slot - first_slot(p, b);
  const int64_t len = p.seq_lens[b], n = c1 - c0, p0 = len - n;
  if (c0 < 0 || n < 0 || c1 > p.num_tokens || (p0 < 0 && n > 0)) {
    if (nth == 0 && part == 0 && lane == 0 && p.status != nullptr) atomicAdd(p.status + NVFP4MLA_STAT_BAD_SLOT, 1);
    return;
  }
  const int64_t t0 = (p0 / kBlockTokens + nth) * kBlockTokens;   // the block's first position
  if (nth < 0 || n == 0 || t0 >= len) return;
  const int64_t col = t0 / kPageTokens;
  const int64_t page = col < p.max_pages ? p.page_table[(int64_t)b * p.max_pages + col] : -1;
  if (page < 0 || page >= p.num_pages) {
    if (part == 0 && lane == 0 && p.status != nullptr) atomicAdd(p.status + NVFP4MLA_STAT_BAD_PAGE, 1);
    return;
  }
  const int quarter = (int)(t0 % kPageTokens) / kBlockTokens;
  uint8_t* base = p.cache + page * p.page_bytes;
  uint8_t* scale = base + kv8_scales_off(p.kv_heads, D, head) + which * kPageBlocks + quarter;
  uint8_t* codes = base + kv8_codes_off(p.kv_heads, D, which, head) + quarter * kBlockTokens * D;

  const bool has_old = p0 > t0;
  const uint32_t before = has_old ? min((uint32_t)*scale, 253u) : 0u;
  const int row0 = lane / kLanes, col8 = (lane % kLanes) * 8;
  const uint16_t* x = p.x[which] + head * p.head_stride[which] + col8;
  uint4 w[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int64_t pos = t0 + i * kRows + row0;
    w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (pos >= p0 && pos < len) w[i] = __ldg(reinterpret_cast<const uint4*>(x + (c0 + pos - p0) * p.token_stride[which]));
  }
  // magnitudes of finite elements order as their bits do
  constexpr uint32_t kInf2 = kHalf ? 0x7C007C00u : 0x7F807F80u;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const uint32_t ws[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t a = ws[k] & 0x7FFF7FFFu;
      top = __vmaxu2(top, a & __vcmpltu2(a, kInf2));
    }
  }
  top = __reduce_max_sync(0xFFFFFFFFu, max(top & 0xFFFFu, top >> 16));
  // amax = m 2^t, 1 <= m < 2, and 448 = 1.75 x 2^8
  const uint32_t bits = __float_as_uint(widen<kHalf>(top).x);
  const int t = (int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  const uint32_t e = max((uint32_t)max(t, 1), before);
  const float mul = __uint_as_float((254u - e) << 23);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int64_t pos = t0 + i * kRows + row0;
    if (pos >= p0 && pos < len) {
      const uint32_t lo2 = encode2<kHalf>(w[i].x, mul) | (encode2<kHalf>(w[i].y, mul) << 16);
      const uint32_t hi2 = encode2<kHalf>(w[i].z, mul) | (encode2<kHalf>(w[i].w, mul) << 16);
      *reinterpret_cast<uint2*>(codes + (i * kRows + row0) * D + col8) = make_uint2(lo2, hi2);
    }
  }
  if (has_old && e > before) {
    const float less = __uint_as_float((127u - min(e - before, 126u)) << 23);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (t0 + i * kRows + row0 < p0) {
        uint2* at = reinterpret_cast<uint2*>(codes + (i * kRows + row0) * D + col8);
        const uint2 c = *at;
        *at = make_uint2(shrink2(c.x & 0xFFFFu, less) | (shrink2(c.x >> 16, less) << 16),
                         shrink2(c.y & 0xFFFFu, less) | (shrink2(c.y >> 16, less) << 16));
      }
    }
  }
  if (lane == 0) *scale = (uint8_t)e;
}

}  // namespace

cudaError_t launch_kv8_append(const AppendParams& p, int head_dim, bool fp16, cudaStream_t stream) {
  const int64_t warps = p.slots * 2 * p.kv_heads;
  const unsigned blocks = (unsigned)((warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32));
  if (head_dim == 128) {
    if (fp16) append_kernel<128, true><<<blocks, kAppendThreads, 0, stream>>>(p);
    else append_kernel<128, false><<<blocks, kAppendThreads, 0, stream>>>(p);
  } else {
    if (fp16) append_kernel<64, true><<<blocks, kAppendThreads, 0, stream>>>(p);
    else append_kernel<64, false><<<blocks, kAppendThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace nvfp4mla
