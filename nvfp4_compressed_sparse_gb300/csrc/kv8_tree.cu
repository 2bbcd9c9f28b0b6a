// kv8_decode_tree: attention of a tree of drafted tokens over the 8-bit per-head cache.
//
// A CTA takes one node and query head: its warps take positions in turn, a lane holding D / 32 dims, each warp with
// a running maximum, sum and weighted values of its own, which are joined at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/nvfp4mla.h"
#include "kv8.h"
#include "kv8_codes.cuh"
#include "ptx.cuh"

namespace nvfp4mla {
namespace {

using namespace ptx;

constexpr int kTreeWarps = 4;
constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

template <int D, bool kHalf>
__global__ void __launch_bounds__(kTreeWarps * 32) tree_kernel(const __grid_constant__ Kv8TreeParams p) {
  constexpr int kN = D / 32;
  __shared__ float acc_of[kTreeWarps][D], m_of[kTreeWarps], l_of[kTreeWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;
  const int h = (int)(row % p.H), kvh = h / p.group;
  const int64_t node = row / p.H;
  const int b = (int)(node / p.Q);
  const int len = max(0, p.seq_lens[b]), base = len - p.Q;
  const uint64_t mask = p.masks[node], used = p.Q == 64 ? mask : mask & ((1ull << p.Q) - 1);
  const int place = base + __popcll(used) - 1;
  const int64_t from = p.window > 0 ? (int64_t)place - p.window + 1 : 0;
  float q[kN];
  bool finite = true;
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const uint16_t x = p.q[node * p.q_token_stride + h * p.q_head_stride + lane * kN + k];
    q[k] = widen<kHalf>(x).x;
    finite = finite && fabsf(q[k]) < __int_as_float(0x7f800000);
  }
  finite = __all_sync(kFull, finite);
  float m = neg_inf(), l = 0.f, acc[kN] = {};
  for (int t = warp; t < len; t += kTreeWarps) {
    if (mask == 0 || (t < base ? t < from : ((used >> (t - base)) & 1) == 0)) continue;
    const int col = t / kPageTokens, r = t % kPageTokens;
    const int page = col < p.max_pages ? p.page_table[(int64_t)b * p.max_pages + col] : -1;
    if (page < 0 || page >= p.num_pages) continue;
    const uint8_t* at = p.cache + page * p.page_bytes;
    const uint8_t* sc = at + kv8_scales_off(p.kv_heads, D, kvh) + r / kBlockTokens;
    const float ks = __uint_as_float((uint32_t)sc[0] << 23), vs = __uint_as_float((uint32_t)sc[4] << 23);
    const uint8_t* kc = at + kv8_codes_off(p.kv_heads, D, 0, kvh) + r * D + lane * kN;
    const uint8_t* vc = at + kv8_codes_off(p.kv_heads, D, 1, kvh) + r * D + lane * kN;
    float z = 0.f, v[kN];
#pragma unroll
    for (int k = 0; k < kN; k += 2) {
      const uint32_t kh = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(kc + k)), vh = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(vc + k));
      const float2 a = widen<true>(kh), c = widen<true>(vh);
      z = fmaf(a.x, q[k], fmaf(a.y, q[k + 1], z));
      v[k] = c.x;
      v[k + 1] = c.y;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) z += __shfl_xor_sync(kFull, z, d);
    z = finite ? z * (p.scale_log2 * ks) : __int_as_float(0x7fc00000);
    const float now = fmaxf(m, z);
    const float keep = m == now ? 1.f : ex2_approx(m - now), w = z == now ? 1.f : ex2_approx(z - now);
    l = l * keep + w;
#pragma unroll
    for (int k = 0; k < kN; ++k) acc[k] = acc[k] * keep + w * (v[k] * vs);
    m = now;
  }
#pragma unroll
  for (int k = 0; k < kN; ++k) acc_of[warp][lane * kN + k] = acc[k];
  if (lane == 0) {
    m_of[warp] = m;
    l_of[warp] = l;
  }
  __syncthreads();
  float top = neg_inf(), sum = 0.f;
  for (int w = 0; w < kTreeWarps; ++w) top = fmaxf(top, m_of[w]);
  for (int w = 0; w < kTreeWarps; ++w) sum += m_of[w] == top ? l_of[w] : l_of[w] * ex2_approx(m_of[w] - top);
  const bool none = !(sum != 0.f);
  for (int d = threadIdx.x; d < D; d += kTreeWarps * 32) {
    float o = 0.f;
    for (int w = 0; w < kTreeWarps; ++w) o += acc_of[w][d] * (m_of[w] == top ? 1.f : ex2_approx(m_of[w] - top));
    o = none ? 0.f : o / sum;
    p.out[row * D + d] = kHalf ? __half_as_ushort(__float2half_rn(o)) : __bfloat16_as_ushort(__float2bfloat16_rn(o));
  }
  if (threadIdx.x == 0) p.lse[row] = none ? neg_inf() : (top + log2f(sum)) * 0.69314718055994530942f;
  // pages that are none, once
  if (h == 0 && node % p.Q == 0 && p.status != nullptr) {
    const int64_t cols = ((int64_t)len + kPageTokens - 1) / kPageTokens;
    const int64_t first = p.window > 0 ? max((int64_t)0, (int64_t)base - p.window + 1) / kPageTokens : 0;
    for (int64_t col = first + threadIdx.x; col < cols; col += kTreeWarps * 32) {
      const int page = col < p.max_pages ? p.page_table[(int64_t)b * p.max_pages + col] : -1;
      if (page < 0 || page >= p.num_pages) atomicAdd(p.status + NVFP4MLA_STAT_BAD_PAGE, 1);
    }
  }
}

}  // namespace

int kv8_tree_columns(int Q, int group) { return 128; }

cudaError_t launch_kv8_decode_tree(const Kv8TreeParams& p, int head_dim, bool fp16, cudaStream_t stream) {
  const unsigned blocks = (unsigned)((int64_t)p.B * p.Q * p.H);
  if (head_dim == 128) {
    if (fp16) tree_kernel<128, true><<<blocks, kTreeWarps * 32, 0, stream>>>(p);
    else tree_kernel<128, false><<<blocks, kTreeWarps * 32, 0, stream>>>(p);
  } else {
    if (fp16) tree_kernel<64, true><<<blocks, kTreeWarps * 32, 0, stream>>>(p);
    else tree_kernel<64, false><<<blocks, kTreeWarps * 32, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace nvfp4mla
