// kv8_decode: attention of a step's queries over the 8-bit per-head cache.
//
// One block per (request, query, query head): the cached tokens in chunks of 128, thread = token
// for the scores and thread = dim for the values, with the running maximum and sum of a softmax.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/nvfp4mla.h"
#include "kv8.h"
#include "ptx.cuh"

namespace nvfp4mla {
namespace {

using namespace ptx;

__device__ __forceinline__ float code_value(uint8_t c) {
  const uint32_t h = e4m3x2_to_f16x2(c);
  return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu)));
}
template <bool kHalf>
__device__ __forceinline__ float widen1(uint16_t x) {
  if constexpr (kHalf) return __half2float(__ushort_as_half(x));
  return __uint_as_float((uint32_t)x << 16);
}

template <int D, bool kHalf>
__global__ void __launch_bounds__(128) decode_simple(const Kv8DecodeParams p) {
  __shared__ float qs[D], ps[128], red[4];
  __shared__ int64_t pages[2];
  const int tid = threadIdx.x;
  int64_t row = blockIdx.x;                       // (b, j, h)
  const int h = (int)(row % p.H);
  const int j = (int)(row / p.H % p.Q);
  const int b = (int)(row / p.H / p.Q);
  const int kvh = h / p.group;
  const float kNegInf = __int_as_float(0xff800000);
  if (tid < D) qs[tid] = widen1<kHalf>(p.q[((int64_t)b * p.Q + j) * p.q_token_stride + h * p.q_head_stride + tid]);
  const int64_t len = p.seq_lens[b], at = len - p.Q + j;
  const int64_t from = p.window > 0 && at - p.window + 1 > 0 ? at - p.window + 1 : 0;
  const int64_t all_from = p.window > 0 && len - p.Q - p.window + 1 > 0 ? len - p.Q - p.window + 1 : 0;
  float m = kNegInf, l = 0.f, o = 0.f;
  for (int64_t t0 = all_from / 128 * 128; t0 < len; t0 += 128) {
    __syncthreads();
    if (tid < 2) {
      const int64_t col = t0 / kPageTokens + tid;
      int64_t page = col < p.max_pages ? p.page_table[(int64_t)b * p.max_pages + col] : -1;
      if (page < 0 || page >= p.num_pages) {
        page = -1;
        if (h == 0 && j == 0 && col * kPageTokens < len && (col + 1) * kPageTokens > all_from && p.status != nullptr)
          atomicAdd(p.status + NVFP4MLA_STAT_BAD_PAGE, 1);
      }
      pages[tid] = page;
    }
    __syncthreads();
    const int64_t t = t0 + tid, page = pages[tid / kPageTokens];
    const int r = tid % kPageTokens;
    float z = kNegInf;
    const bool ok = t >= from && t <= at && t < len && page >= 0;
    if (ok) {
      const uint8_t* base = p.cache + page * p.page_bytes;
      const uint8_t* k = base + kv8_codes_off(p.kv_heads, D, 0, kvh) + r * D;
      float s = 0.f;
      for (int d = 0; d < D; ++d) s += qs[d] * code_value(k[d]);
      z = s * __uint_as_float((uint32_t)base[kv8_scales_off(p.kv_heads, D, kvh) + r / kBlockTokens] << 23) * p.scale_log2;
    }
    float top = z;
    for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));
    if ((tid & 31) == 0) red[tid >> 5] = top;
    __syncthreads();
    const float m_new = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float base_m = m_new == kNegInf ? 0.f : m_new;
    const float e = ok ? exp2f(z - base_m) : 0.f;
    ps[tid] = e;
    const float keep = exp2f((m == kNegInf ? base_m : m) - base_m);
    __syncthreads();
    float lc = 0.f, oc = 0.f;   // the chunk's own sums: a long run of small terms is not added one by one to a large one
    for (int i = 0; i < 128; ++i) {
      const int64_t pg = pages[i / kPageTokens];
      if (pg < 0 || t0 + i < from || t0 + i > at || t0 + i >= len) continue;
      lc += ps[i];
      if (tid < D) {
        const uint8_t* base = p.cache + pg * p.page_bytes;
        const int ri = i % kPageTokens;
        oc += ps[i] * (code_value(base[kv8_codes_off(p.kv_heads, D, 1, kvh) + ri * D + tid]) *
                      __uint_as_float((uint32_t)base[kv8_scales_off(p.kv_heads, D, kvh) + kPageBlocks + ri / kBlockTokens] << 23));
      }
    }
    l = l * keep + lc;
    o = o * keep + oc;
    m = m_new;
  }
  const bool empty = l == 0.f;
  const float v = empty ? 0.f : o / l;
  if (tid < D) {
    if constexpr (kHalf) p.out[row * D + tid] = __half_as_ushort(__float2half_rn(v));
    else p.out[row * D + tid] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
  if (tid == 0) p.lse[row] = empty ? kNegInf : (m + log2f(l)) * 0.69314718055994530942f;
}

}  // namespace

cudaError_t launch_kv8_decode(const Kv8DecodeParams& p, int head_dim, bool fp16, cudaStream_t stream) {
  const unsigned blocks = (unsigned)((int64_t)p.B * p.Q * p.H);
  if (head_dim == 128) {
    if (fp16) decode_simple<128, true><<<blocks, 128, 0, stream>>>(p);
    else decode_simple<128, false><<<blocks, 128, 0, stream>>>(p);
  } else {
    if (fp16) decode_simple<64, true><<<blocks, 128, 0, stream>>>(p);
    else decode_simple<64, false><<<blocks, 128, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace nvfp4mla
