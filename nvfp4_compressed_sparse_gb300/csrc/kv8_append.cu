// kv8_append: new keys and values into the 8-bit per-head cache.
//
// A warp takes one block of 16 tokens of one head, keys and values. It finds its request and block
// from its number, reads the block's new rows (all loads issued before any is used), takes the
// largest finite magnitude, and from it the block's exponent; the codes are x 2^(127 - e) rounded
// to E4M3, exact but for that one rounding, since a power of two moves no mantissa bit.
//
// The floor is the traffic, three bytes per value (two in, one out). Consecutive warps take
// consecutive heads of the same tokens, so that a token's row of all heads is read in one piece.
//
// Measured (device time): 12 prompts of 300-9,000 tokens, 8 heads of 128: 213 MB in 36.9 us, 5.8 TB/s,
// 85 % of the measured copy bandwidth, ALU pipe 55 % busy (it makes the codes); 64 requests of one token:
// 4.2 us, a launch and one chain of loads. Keys and values by one warp instead of two took 64 to 62 us,
// the path for finite blocks 62 to 40.
#include <cuda_fp16.h>

#include "../../include/nvfp4mla.h"
#include "kv8.h"
#include "ptx.cuh"

namespace nvfp4mla {
namespace {

using namespace ptx;

constexpr int kAppendThreads = 128;    // five such blocks an SM: 37 us (a row above), three of 256 threads 40

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

template <int D, bool kHalf>
__global__ void __launch_bounds__(kAppendThreads, 5) append_kernel(const AppendParams p) {
  constexpr int kLanes = D / 8;              // lanes per row, 8 values (16 bytes) each
  constexpr int kRows = 32 / kLanes;         // rows per load
  constexpr int kLoads = kBlockTokens / kRows;
  const int lane = threadIdx.x & 31;
  const unsigned item = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int slot = (int)(item / (unsigned)p.kv_heads), head = (int)(item - (unsigned)slot * (unsigned)p.kv_heads);
  if (slot >= p.slots) return;

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
  const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1), len = __ldg(p.seq_lens + b);
  const int nth = slot - first_slot(p, b);
  const int64_t n = (int64_t)c1 - c0, p0 = len - n;
  if (c0 < 0 || n < 0 || c1 > p.num_tokens || (p0 < 0 && n > 0)) {
    if (nth == 0 && head == 0 && lane == 0 && p.status != nullptr) atomicAdd(p.status + NVFP4MLA_STAT_BAD_SLOT, 1);
    return;
  }
  if (nth < 0 || n == 0) return;
  // the block's first position, its first new row, and the rows that are new: first .. behind - 1
  const int64_t t0 = (p0 / kBlockTokens + nth) * kBlockTokens;
  if (t0 >= len) return;
  const int first = p0 > t0 ? (int)(p0 - t0) : 0, behind = (int)min((int64_t)kBlockTokens, len - t0);
  const int64_t col = t0 / kPageTokens;
  const int64_t page = col < p.max_pages ? __ldg(p.page_table + (int64_t)b * p.max_pages + col) : -1;
  if (page < 0 || page >= p.num_pages) {
    if (head == 0 && lane == 0 && p.status != nullptr) atomicAdd(p.status + NVFP4MLA_STAT_BAD_PAGE, 1);
    return;
  }
  const int quarter = (int)(t0 % kPageTokens) / kBlockTokens;
  const int row0 = lane / kLanes, col8 = (lane % kLanes) * 8;
  const int64_t token = c0 + (t0 - p0);      // of the block's row 0 (behind the block's old rows: not read)
  uint8_t* base = p.cache + page * p.page_bytes;
  uint8_t* scales = base + kv8_scales_off(p.kv_heads, D, head) + quarter;

  uint4 w[2][kLoads];
  uint32_t before[2];
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const uint16_t* x = p.x[which] + head * p.head_stride[which] + col8;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = i * kRows + row0;
      w[which][i] = make_uint4(0u, 0u, 0u, 0u);
      if (row >= first && row < behind) w[which][i] = __ldcs(reinterpret_cast<const uint4*>(x + (token + row) * p.token_stride[which]));
    }
    before[which] = first > 0 ? min((uint32_t)scales[which * kPageBlocks], 253u) : 0u;
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    uint8_t* codes = base + kv8_codes_off(p.kv_heads, D, which, head) + quarter * kBlockTokens * D + col8;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) top = top8<kHalf, false>(w[which][i], top);
    top = __reduce_max_sync(0xFFFFFFFFu, max(top & 0xFFFFu, top >> 16));
    // blocks with an infinity or a NaN are rare, and cost three times the instructions
    const bool finite = top < (kHalf ? 0x7C00u : 0x7F80u);
    if (!finite) {
      top = 0;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) top = top8<kHalf, true>(w[which][i], top);
      top = __reduce_max_sync(0xFFFFFFFFu, max(top & 0xFFFFu, top >> 16));
    }
    // amax = m 2^t, 1 <= m < 2, and 448 = 1.75 x 2^8
    const uint32_t bits = __float_as_uint(widen<kHalf>(top).x);
    const int t = (int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    const uint32_t e = max((uint32_t)max(t, 1), before[which]);
    const float mul = __uint_as_float((254u - e) << 23);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = i * kRows + row0;
      if (row >= first && row < behind)
        *reinterpret_cast<uint2*>(codes + row * D) = finite ? encode8<kHalf, false>(w[which][i], mul) : encode8<kHalf, true>(w[which][i], mul);
    }
    if (first > 0 && e > before[which]) {
      const float less = __uint_as_float((127u - min(e - before[which], 126u)) << 23);
#pragma unroll 1
      for (int row = row0; row < first; row += kRows) {
        uint2* at = reinterpret_cast<uint2*>(codes + row * D);
        const uint2 c = *at;
        *at = make_uint2(shrink2(c.x & 0xFFFFu, less) | (shrink2(c.x >> 16, less) << 16),
                         shrink2(c.y & 0xFFFFu, less) | (shrink2(c.y >> 16, less) << 16));
      }
    }
    if (lane == 0) scales[which * kPageBlocks] = (uint8_t)e;
  }
}

}  // namespace

cudaError_t launch_kv8_append(const AppendParams& p, int head_dim, bool fp16, cudaStream_t stream) {
  const int64_t warps = p.slots * p.kv_heads;
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
