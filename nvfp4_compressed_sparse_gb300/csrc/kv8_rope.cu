// kv8_append_rope: queries and keys normalised and rotated on the way, keys and values into the 8-bit
// per-head cache.
//
// What it computes. Of a row x of D values: y = x w / sqrt(mean(x^2) + eps), where a norm is given, then
// each pair (a, b) of y turned by its angle, (a c - b s, b c + a s), all in fp32. Queries are rounded once,
// to their type; keys once, to E4M3 under their block's scale, which is taken from the turned values.
//
// A CTA takes a block of 16 tokens of one request and a share of its rows' heads: it stages the cosines and
// sines of its tokens once, then each warp takes a head at a time, 16 bytes a lane.
#include <cmath>

#include "../../include/nvfp4mla.h"
#include "kv8.h"
#include "kv8_codes.cuh"
#include "ptx.cuh"

namespace nvfp4mla {
namespace {

using namespace ptx;

constexpr int kRopeWarps = 8;
constexpr unsigned kFull = 0xFFFFFFFFu;

template <bool kHalf>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
  if constexpr (kHalf) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The staged row of a token: `rot` floats, in the order in which lanes read them, 16 bytes at a time.
// Pairs of halves (a = x[i], b = x[i + rot/2]): a lane's eight dims need eight cosines and eight sines, and
// neighbouring lanes' first four lie side by side. Interleaved (a = x[2i], b = x[2i + 1]): four of each.
template <bool kInter>
__device__ __forceinline__ int staged_at(int rot, int i, int sine) {
  if constexpr (kInter) return sine * (rot / 2) + i;
  const int chunks = rot / 16;
  return ((sine * 2 + ((i >> 2) & 1)) * chunks + (i >> 3)) * 4 + (i & 3);
}

// Eight values of a row, of dims 8 chunk .. 8 chunk + 7, normalised and turned.
template <int D, bool kHalf, bool kInter>
__device__ __forceinline__ void turn(const uint4& raw, const uint4& w4, bool norm, float eps, const float* sheet, int rot, int chunk,
                                     float (&y)[8]) {
  constexpr int kLanes = Rows<D>::kLanes;
  const uint32_t ws[4] = {raw.x, raw.y, raw.z, raw.w}, gs[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = widen<kHalf>(ws[k]);
    y[2 * k] = x.x;
    y[2 * k + 1] = x.y;
  }
  if (norm) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum = fmaf(y[k], y[k], sum);
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) sum += __shfl_xor_sync(kFull, sum, d);
    const float inv = rsqrtf(sum * (1.f / D) + eps);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 g = widen<kHalf>(gs[k]);
      y[2 * k] = y[2 * k] * inv * g.x;
      y[2 * k + 1] = y[2 * k + 1] * inv * g.y;
    }
  }
  const bool turned = 8 * chunk < rot;
  if constexpr (kInter) {
    if (turned) {
      const float4 c = *reinterpret_cast<const float4*>(sheet + 4 * chunk), s = *reinterpret_cast<const float4*>(sheet + rot / 2 + 4 * chunk);
      const float cs[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = y[2 * k], b = y[2 * k + 1];
        y[2 * k] = a * cs[k] - b * ss[k];
        y[2 * k + 1] = b * cs[k] + a * ss[k];
      }
    }
  } else {
    const int chunks = rot / 16;                           // of either half
    const bool second = chunk >= chunks;
    const int lane = threadIdx.x & 31, at = second ? chunk - chunks : chunk;
    const int other = turned ? (second ? lane - chunks : lane + chunks) : lane;
    float z[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) z[k] = __shfl_sync(kFull, y[k], other);
    if (turned) {
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const float4 c = *reinterpret_cast<const float4*>(sheet + (f * chunks + at) * 4), s = *reinterpret_cast<const float4*>(sheet + ((2 + f) * chunks + at) * 4);
        const float cs[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float sine = second ? ss[k] : -ss[k];
          y[4 * f + k] = y[4 * f + k] * cs[k] + z[4 * f + k] * sine;
        }
      }
    }
  }
}

template <int D, bool kHalf, bool kInter>
__global__ void __launch_bounds__(kRopeWarps * 32, 2) rope_kernel(const __grid_constant__ RopeParams p, int per) {
  using R = Rows<D>;
  __shared__ __align__(16) float sheets[kBlockTokens][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slot = blockIdx.x;
  const int b = request_of(p, slot);
  const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1), len = __ldg(p.seq_lens + b);
  const int nth = slot - first_slot(p, b);
  const int64_t n = (int64_t)c1 - c0, p0 = len - n;
  const bool speaks = blockIdx.y == 0 && threadIdx.x == 0 && p.status != nullptr;
  if (c0 < 0 || n < 0 || c1 > p.num_tokens || (p0 < 0 && n > 0)) {
    if (nth == 0 && speaks) atomicAdd(p.status + NVFP4MLA_STAT_BAD_SLOT, 1);
    return;
  }
  if (nth < 0 || n == 0) return;
  const int64_t t0 = (p0 / kBlockTokens + nth) * kBlockTokens;
  if (t0 >= len) return;
  const int first = p0 > t0 ? (int)(p0 - t0) : 0, behind = (int)min((int64_t)kBlockTokens, len - t0);
  const int64_t token = c0 + (t0 - p0);      // of the block's row 0 (behind the block's old rows: not read)

  // cosines and sines of the new tokens
  const int half = p.rot / 2;
  for (int i = threadIdx.x; i < (behind - first) * half; i += kRopeWarps * 32) {
    const int row = first + i / half, pair = i - i / half * half;
    int axis = 0;
    if (p.positions != nullptr) {
#pragma unroll
      for (int a = 0; a < kMaxAxes - 1; ++a) axis += a + 1 < p.axes && pair >= p.ends[a] ? 1 : 0;
    }
    const int64_t at = p.positions != nullptr ? (int64_t)__ldg(p.positions + axis * p.axis_stride + token + row) : t0 + row;
    float c = __int_as_float(0x7fc00000), s = c;           // no position of the table: NaN, and counted
    if (at >= 0 && at < p.max_positions) {
      c = __ldg(p.cos_sin + at * p.rot + pair);
      s = __ldg(p.cos_sin + at * p.rot + half + pair);
    }
    sheets[row][staged_at<kInter>(p.rot, pair, 0)] = c;
    sheets[row][staged_at<kInter>(p.rot, pair, 1)] = s;
  }
  if (blockIdx.y == 0 && (int)threadIdx.x >= first && (int)threadIdx.x < behind && p.status != nullptr) {
    bool bad = false;
    for (int a = 0; a < (p.positions != nullptr ? p.axes : 1); ++a) {
      const int64_t at = p.positions != nullptr ? (int64_t)__ldg(p.positions + a * p.axis_stride + token + threadIdx.x) : t0 + threadIdx.x;
      bad = bad || at < 0 || at >= p.max_positions;
    }
    if (bad) atomicAdd(p.status + NVFP4MLA_STAT_BAD_INDEX, 1);
  }
  __syncthreads();

  const int64_t col = t0 / kPageTokens;
  const int64_t page = col < p.max_pages ? __ldg(p.page_table + (int64_t)b * p.max_pages + col) : -1;
  const bool have = page >= 0 && page < p.num_pages;
  if (!have && speaks) atomicAdd(p.status + NVFP4MLA_STAT_BAD_PAGE, 1);
  const int quarter = (int)(t0 % kPageTokens) / kBlockTokens;
  const int row0 = lane / R::kLanes, chunk = lane % R::kLanes;
  uint8_t* base = p.cache + page * p.page_bytes;

  const int items = p.heads + 2 * p.kv_heads, end = min(items, (int)(blockIdx.y + 1) * per);
  for (int item = blockIdx.y * per + warp; item < end; item += kRopeWarps) {
    const int kind = item < p.heads ? 0 : (item < p.heads + p.kv_heads ? 1 : 2);     // a query, a key, a value
    const int head = kind == 0 ? item : (kind == 1 ? item - p.heads : item - p.heads - p.kv_heads);
    if (kind != 0 && !have) continue;
    const uint16_t* x = (kind == 0 ? p.q + head * p.q_head_stride : p.x[kind - 1] + head * p.head_stride[kind - 1]) + 8 * chunk;
    const int64_t stride = kind == 0 ? p.q_token_stride : p.token_stride[kind - 1];
    uint4 w[R::kLoads];
#pragma unroll
    for (int i = 0; i < R::kLoads; ++i) {
      const int row = i * R::kAtOnce + row0;
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (row >= first && row < behind) w[i] = *reinterpret_cast<const uint4*>(x + (token + row) * stride);
    }
    const uint16_t* weight = kind == 2 ? nullptr : p.weight[kind];
    const uint4 g = weight != nullptr ? __ldg(reinterpret_cast<const uint4*>(weight + 8 * chunk)) : make_uint4(0u, 0u, 0u, 0u);
    if (kind == 0) {
#pragma unroll
      for (int i = 0; i < R::kLoads; ++i) {
        const int row = i * R::kAtOnce + row0;
        if ((i + 1) * R::kAtOnce <= first || i * R::kAtOnce >= behind) continue;
        float y[8];
        turn<D, kHalf, kInter>(w[i], g, weight != nullptr, p.eps, sheets[row], p.rot, chunk, y);
        if (row >= first && row < behind)
          *reinterpret_cast<uint4*>(p.q_out + (token + row) * p.out_token_stride + head * p.out_head_stride + 8 * chunk) =
              make_uint4(narrow2<kHalf>(y[0], y[1]), narrow2<kHalf>(y[2], y[3]), narrow2<kHalf>(y[4], y[5]), narrow2<kHalf>(y[6], y[7]));
      }
      continue;
    }
    uint8_t* codes = base + kv8_codes_off(p.kv_heads, D, kind - 1, head) + quarter * kBlockTokens * D + 8 * chunk;
    uint8_t* scale = base + kv8_scales_off(p.kv_heads, D, head) + (kind - 1) * kPageBlocks + quarter;
    const uint32_t before = first > 0 ? min((uint32_t)*scale, 253u) : 0u;
    __syncwarp();
    if (kind == 2) {
      put_block<D, kHalf>(w, row0, first, behind, before, codes, scale);
      continue;
    }
    float y[R::kLoads][8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < R::kLoads; ++i) {
      const int row = i * R::kAtOnce + row0;
      if ((i + 1) * R::kAtOnce <= first || i * R::kAtOnce >= behind) continue;
      turn<D, kHalf, kInter>(w[i], g, weight != nullptr, p.eps, sheets[row], p.rot, chunk, y[i]);
      if (row >= first && row < behind) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t a = __float_as_uint(y[i][k]) & 0x7FFFFFFFu;
          top = a < 0x7F800000u ? max(top, a) : top;
        }
      }
    }
    top = __reduce_max_sync(kFull, top);
    const uint32_t e = max(scale_byte(__uint_as_float(top)), before);
    const float mul = __uint_as_float((254u - e) << 23);
#pragma unroll
    for (int i = 0; i < R::kLoads; ++i) {
      const int row = i * R::kAtOnce + row0;
      if (row < first || row >= behind) continue;
      uint32_t two[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = y[i][2 * k] * mul, c = y[i][2 * k + 1] * mul;
        two[k] = f32x2_to_e4m3x2(a, c);
        // a NaN of this arithmetic has no sign
        if (a != a) two[k] = (two[k] & 0xFF00u) | 0x7Fu;
        if (c != c) two[k] = (two[k] & 0x00FFu) | 0x7F00u;
      }
      *reinterpret_cast<uint2*>(codes + row * D) = make_uint2(__byte_perm(two[0], two[1], 0x5410), __byte_perm(two[2], two[3], 0x5410));
    }
    if (first > 0 && e > before) shrink_rows<D>(codes, row0, first, before, e);
    if (lane == 0) *scale = (uint8_t)e;
  }
}

template <int D, bool kHalf>
void launch(const RopeParams& p, bool interleaved, cudaStream_t stream) {
  // CTAs enough for every SM to hold its two, and no more shares of a block than leave each warp a head
  const int items = p.heads + 2 * p.kv_heads;
  int shares = (items + kRopeWarps - 1) / kRopeWarps;
  const int64_t want = (int64_t)4 * device_sm_count();
  const int64_t need = (want + p.slots - 1) / p.slots;
  if (need < shares) shares = (int)need;
  int per = (items + shares - 1) / shares;
  per = (per + kRopeWarps - 1) / kRopeWarps * kRopeWarps;
  const dim3 grid((unsigned)p.slots, (unsigned)((items + per - 1) / per));
  if (interleaved) rope_kernel<D, kHalf, true><<<grid, kRopeWarps * 32, 0, stream>>>(p, per);
  else rope_kernel<D, kHalf, false><<<grid, kRopeWarps * 32, 0, stream>>>(p, per);
}

}  // namespace

cudaError_t launch_kv8_append_rope(const RopeParams& p, int head_dim, bool fp16, bool interleaved, cudaStream_t stream) {
  if (head_dim == 128) {
    if (fp16) launch<128, true>(p, interleaved, stream);
    else launch<128, false>(p, interleaved, stream);
  } else {
    if (fp16) launch<64, true>(p, interleaved, stream);
    else launch<64, false>(p, interleaved, stream);
  }
  return cudaGetLastError();
}

}  // namespace nvfp4mla
