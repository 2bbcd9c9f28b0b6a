// kv8_append_rope: queries and keys normalised and rotated on the way, keys and values into the 8-bit
// per-head cache.
//
// What it computes. Of a row x of D values: y = x w / sqrt(mean(x^2) + eps), where a norm is given, then
// each pair (a, b) of y turned by its angle, (a c - b s, b c + a s), all in fp32. Queries are rounded once,
// to their type; keys once, to E4M3 under their block's scale, which is taken from the turned values.
//
// What bounds it: memory, four bytes a query's value and three a key's or value's, once a row costs few enough
// instructions: some 60 for two rows. A lane has four pairs: two runs of four dims, half the turned dims apart, or eight
// dims side by side where pairs are neighbours, so that nothing but the sum of squares crosses lanes; behind the turned
// dims it has eight dims of its own. A key is turned twice, for its block's scale and for its code, as holding 16 turned
// rows would leave too few warps.
//
// A CTA takes a block of 16 tokens of one request and a share of its rows' heads: it stages the cosines and
// sines of its tokens once, then each warp takes a head at a time.
#include <cmath>

#include "../../include/nvfp4mla.h"
#include "kv8.h"
#include "kv8_codes.cuh"
#include "ptx.cuh"

namespace nvfp4mla {
namespace {

using namespace ptx;

constexpr int kRopeWarps = 8, kRopeBlocks = 4;   // of an SM
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

// A lane's values of a row: two runs of four.
struct Eight {
  float2 a[2], b[2];
};
template <bool kHalf>
__device__ __forceinline__ Eight widen8(const uint2& a, const uint2& b) {
  return Eight{{widen<kHalf>(a.x), widen<kHalf>(a.y)}, {widen<kHalf>(b.x), widen<kHalf>(b.y)}};
}
__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }

// The values normalised (g: the weights) and turned (c, s: of the lane's four pairs).
template <int D, bool kInter>
__device__ __forceinline__ void turn(Eight& y, bool norm, const Eight& g, float eps, bool turns, const float* sheet, int half) {
  if (norm) {
    float2 sum = __fmul2_rn(y.a[0], y.a[0]);
    sum = __ffma2_rn(y.a[1], y.a[1], sum);
    sum = __ffma2_rn(y.b[0], y.b[0], sum);
    sum = __ffma2_rn(y.b[1], y.b[1], sum);
    float all = sum.x + sum.y;
#pragma unroll
    for (int d = 1; d < Rows<D>::kLanes; d <<= 1) all += __shfl_xor_sync(kFull, all, d);
    const float2 inv = twice(rsqrtf(all * (1.f / D) + eps));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      y.a[k] = __fmul2_rn(__fmul2_rn(y.a[k], inv), g.a[k]);
      y.b[k] = __fmul2_rn(__fmul2_rn(y.b[k], inv), g.b[k]);
    }
  }
  if (!turns) return;
  const float4 c = *reinterpret_cast<const float4*>(sheet), s = *reinterpret_cast<const float4*>(sheet + half);
  if constexpr (kInter) {
    const float cs[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float2& v = k < 2 ? y.a[k] : y.b[k - 2];
      v = make_float2(fmaf(-v.y, ss[k], v.x * cs[k]), fmaf(v.x, ss[k], v.y * cs[k]));
    }
  } else {
    const float2 cs[2] = {make_float2(c.x, c.y), make_float2(c.z, c.w)}, ss[2] = {make_float2(s.x, s.y), make_float2(s.z, s.w)};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 a = y.a[k], b = y.b[k];
      y.a[k] = __ffma2_rn(b, make_float2(-ss[k].x, -ss[k].y), __fmul2_rn(a, cs[k]));
      y.b[k] = __ffma2_rn(a, ss[k], __fmul2_rn(b, cs[k]));
    }
  }
}

// Two values as E4M3 of x * mul, saturating; a NaN becomes 0x7F.
__device__ __forceinline__ uint32_t code2(float2 x, float mul) {
  x = __fmul2_rn(x, twice(mul));
  return f32x2_to_e4m3x2(x.x, x.y);
}

// A block of 16 tokens, and a warp's part in it.
struct Block {
  int64_t token;                   // of its row 0 (behind the block's old rows: not read)
  int first, behind;               // its new rows
  int quarter;                     // of its page
  uint8_t* page;
};

// Where a lane's two runs of four dims lie, and which rows of a warp's loads are new.
template <int D, bool kInter>
struct Lane {
  using R = Rows<D>;
  int row0, l, at_a, at_b;
  bool turns;
  uint32_t rows, steps;            // bit i: load i's row of this lane is new; of any lane
  __device__ __forceinline__ Lane(const Block& b, int rot) {
    const int lane = threadIdx.x & 31;
    row0 = lane / R::kLanes;
    l = lane % R::kLanes;
    turns = l < rot / 8;
    at_a = !kInter && turns ? 4 * l : 8 * l;
    at_b = !kInter && turns ? rot / 2 + 4 * l : 8 * l + 4;
    rows = steps = 0;
#pragma unroll
    for (int i = 0; i < R::kLoads; ++i) {
      const int row = i * R::kAtOnce + row0;
      rows |= (row >= b.first && row < b.behind ? 1u : 0u) << i;
      steps |= ((i + 1) * R::kAtOnce > b.first && i * R::kAtOnce < b.behind ? 1u : 0u) << i;
    }
  }
  __device__ __forceinline__ bool is_new(int i) const { return (rows >> i) & 1; }
  __device__ __forceinline__ bool is_step(int i) const { return (steps >> i) & 1; }
  // Rows of one head, x at the lane's row 0; zeros where a row is not new.
  __device__ __forceinline__ void load(const uint16_t* x, int64_t stride, uint4 (&w)[R::kLoads]) const {
#pragma unroll
    for (int i = 0; i < R::kLoads; ++i) {
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (is_new(i)) {
        if constexpr (kInter) {
          w[i] = *reinterpret_cast<const uint4*>(x + at_a);
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(x + at_a), v = *reinterpret_cast<const uint2*>(x + at_b);
          w[i] = make_uint4(u.x, u.y, v.x, v.y);
        }
      }
      x += R::kAtOnce * stride;
    }
  }
};

template <int D, bool kHalf, bool kInter>
__device__ __forceinline__ void queries(const RopeParams& p, const Block& b, const float (*sheets)[D], int head, int end) {
  using R = Rows<D>;
  const Lane<D, kInter> lane(b, p.rot);
  const bool norm = p.weight[0] != nullptr;
  Eight g = {};
  if (norm) g = widen8<kHalf>(__ldg(reinterpret_cast<const uint2*>(p.weight[0] + lane.at_a)), __ldg(reinterpret_cast<const uint2*>(p.weight[0] + lane.at_b)));
#pragma unroll 1
  for (; head < end; head += kRopeWarps) {
    uint4 w[R::kLoads];
    lane.load(p.q + (b.token + lane.row0) * p.q_token_stride + head * p.q_head_stride, p.q_token_stride, w);
    uint16_t* to = p.q_out + (b.token + lane.row0) * p.out_token_stride + head * p.out_head_stride;
#pragma unroll
    for (int i = 0; i < R::kLoads; ++i) {
      if (lane.is_step(i)) {
        Eight y = widen8<kHalf>(make_uint2(w[i].x, w[i].y), make_uint2(w[i].z, w[i].w));
        turn<D, kInter>(y, norm, g, p.eps, lane.turns, sheets[i * R::kAtOnce + lane.row0] + 4 * lane.l, p.rot / 2);
        const uint2 u = make_uint2(narrow2<kHalf>(y.a[0].x, y.a[0].y), narrow2<kHalf>(y.a[1].x, y.a[1].y));
        const uint2 v = make_uint2(narrow2<kHalf>(y.b[0].x, y.b[0].y), narrow2<kHalf>(y.b[1].x, y.b[1].y));
        if (lane.is_new(i)) {
          if constexpr (kInter) {
            *reinterpret_cast<uint4*>(to + lane.at_a) = make_uint4(u.x, u.y, v.x, v.y);
          } else {
            *reinterpret_cast<uint2*>(to + lane.at_a) = u;
            *reinterpret_cast<uint2*>(to + lane.at_b) = v;
          }
        }
      }
      to += R::kAtOnce * p.out_token_stride;
    }
  }
}

template <int D, bool kHalf, bool kInter>
__device__ __forceinline__ void keys(const RopeParams& p, const Block& b, const float (*sheets)[D], int head, int end) {
  using R = Rows<D>;
  const Lane<D, kInter> lane(b, p.rot);
  const bool norm = p.weight[1] != nullptr;
  Eight g = {};
  if (norm) g = widen8<kHalf>(__ldg(reinterpret_cast<const uint2*>(p.weight[1] + lane.at_a)), __ldg(reinterpret_cast<const uint2*>(p.weight[1] + lane.at_b)));
#pragma unroll 1
  for (; head < end; head += kRopeWarps) {
    uint4 w[R::kLoads];
    lane.load(p.x[0] + (b.token + lane.row0) * p.token_stride[0] + head * p.head_stride[0], p.token_stride[0], w);
    uint8_t* codes = b.page + kv8_codes_off(p.kv_heads, D, 0, head) + b.quarter * kBlockTokens * D;
    uint8_t* scale = b.page + kv8_scales_off(p.kv_heads, D, head) + b.quarter;
    const uint32_t before = b.first > 0 ? min((uint32_t)*scale, 253u) : 0u;
    __syncwarp();
    auto turned = [&](int i) {
      Eight y = widen8<kHalf>(make_uint2(w[i].x, w[i].y), make_uint2(w[i].z, w[i].w));
      turn<D, kInter>(y, norm, g, p.eps, lane.turns, sheets[i * R::kAtOnce + lane.row0] + 4 * lane.l, p.rot / 2);
      return y;
    };
    // the largest; of the finite ones, once there is an infinity (a NaN is never the larger)
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < R::kLoads; ++i) {
      if (!lane.is_step(i)) continue;
      const Eight y = turned(i);
      const float most = fmaxf(fmaxf(fmaxf(fabsf(y.a[0].x), fabsf(y.a[0].y)), fmaxf(fabsf(y.a[1].x), fabsf(y.a[1].y))),
                               fmaxf(fmaxf(fabsf(y.b[0].x), fabsf(y.b[0].y)), fmaxf(fabsf(y.b[1].x), fabsf(y.b[1].y))));
      if (lane.is_new(i)) top = fmaxf(top, most);
    }
    uint32_t bits = __reduce_max_sync(kFull, __float_as_uint(top));
    if (__builtin_expect(bits >= 0x7F800000u, 0)) {
      bits = 0;
#pragma unroll
      for (int i = 0; i < R::kLoads; ++i) {
        if (!lane.is_step(i)) continue;
        const Eight y = turned(i);
        const float x[8] = {y.a[0].x, y.a[0].y, y.a[1].x, y.a[1].y, y.b[0].x, y.b[0].y, y.b[1].x, y.b[1].y};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t a = __float_as_uint(x[k]) & 0x7FFFFFFFu;
          if (lane.is_new(i) && a < 0x7F800000u) bits = max(bits, a);
        }
      }
      bits = __reduce_max_sync(kFull, bits);
    }
    const uint32_t e = max(scale_byte(__uint_as_float(bits)), before);
    const float mul = __uint_as_float((254u - e) << 23);
    uint8_t* to = codes + lane.row0 * D;
#pragma unroll
    for (int i = 0; i < R::kLoads; ++i) {
      if (!lane.is_step(i)) continue;
      const Eight y = turned(i);
      if (!lane.is_new(i)) continue;
      *reinterpret_cast<uint32_t*>(to + i * R::kAtOnce * D + lane.at_a) = __byte_perm(code2(y.a[0], mul), code2(y.a[1], mul), 0x5410);
      *reinterpret_cast<uint32_t*>(to + i * R::kAtOnce * D + lane.at_b) = __byte_perm(code2(y.b[0], mul), code2(y.b[1], mul), 0x5410);
    }
    if (b.first > 0 && e > before) shrink_rows<D>(codes + 8 * lane.l, lane.row0, b.first, before, e);
    if ((threadIdx.x & 31) == 0) *scale = (uint8_t)e;
  }
}

template <int D, bool kHalf>
__device__ __forceinline__ void values(const RopeParams& p, const Block& b, int head, int end) {
  using R = Rows<D>;
  const int row0 = (threadIdx.x & 31) / R::kLanes, at = (threadIdx.x & 31) % R::kLanes * 8;
#pragma unroll 1
  for (; head < end; head += kRopeWarps) {
    const uint16_t* x = p.x[1] + (b.token + row0) * p.token_stride[1] + head * p.head_stride[1] + at;
    uint4 w[R::kLoads];
#pragma unroll
    for (int i = 0; i < R::kLoads; ++i) {
      const int row = i * R::kAtOnce + row0;
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (row >= b.first && row < b.behind) w[i] = *reinterpret_cast<const uint4*>(x);
      x += R::kAtOnce * p.token_stride[1];
    }
    uint8_t* scale = b.page + kv8_scales_off(p.kv_heads, D, head) + kPageBlocks + b.quarter;
    const uint32_t before = b.first > 0 ? min((uint32_t)*scale, 253u) : 0u;
    __syncwarp();
    put_block<D, kHalf>(w, row0, b.first, b.behind, before, b.page + kv8_codes_off(p.kv_heads, D, 1, head) + b.quarter * kBlockTokens * D + at, scale);
  }
}

// blockIdx.y: shares of the queries' heads, then of the keys', then of the values', so that a CTA has one code.
template <int D, bool kHalf, bool kInter>
__global__ void __launch_bounds__(kRopeWarps * 32, kRopeBlocks) rope_kernel(const __grid_constant__ RopeParams p, int q_shares, int kv_shares, int q_per, int kv_per) {
  __shared__ __align__(16) float sheets[kBlockTokens][D];      // of a token: cosines of its pairs, then sines
  const int warp = threadIdx.x >> 5;
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
  Block block;
  block.first = p0 > t0 ? (int)(p0 - t0) : 0;
  block.behind = (int)min((int64_t)kBlockTokens, len - t0);
  block.token = c0 + (t0 - p0);
  block.quarter = (int)(t0 % kPageTokens) / kBlockTokens;
  const int64_t col = t0 / kPageTokens;
  const int64_t page = col < p.max_pages ? __ldg(p.page_table + (int64_t)b * p.max_pages + col) : -1;
  const bool have = page >= 0 && page < p.num_pages;
  if (!have && speaks) atomicAdd(p.status + NVFP4MLA_STAT_BAD_PAGE, 1);
  block.page = p.cache + page * p.page_bytes;

  const int kind = (int)blockIdx.y < q_shares ? 0 : ((int)blockIdx.y < q_shares + kv_shares ? 1 : 2);
  const int share = blockIdx.y - (kind == 0 ? 0 : (kind == 1 ? q_shares : q_shares + kv_shares));
  const int per = kind == 0 ? q_per : kv_per, head = share * per + warp, end = min(kind == 0 ? p.heads : p.kv_heads, (share + 1) * per);
  if (kind != 0 && !have) return;
  if (kind == 2) {
    values<D, kHalf>(p, block, head, end);
    return;
  }
  const int half = p.rot / 2;
#pragma unroll 1
  for (int i = threadIdx.x; i < (block.behind - block.first) * half; i += kRopeWarps * 32) {
    const int row = block.first + i / half, pair = i - i / half * half;
    int axis = 0;
    if (p.positions != nullptr) {
#pragma unroll
      for (int a = 0; a < kMaxAxes - 1; ++a) axis += a + 1 < p.axes && pair >= p.ends[a] ? 1 : 0;
    }
    const int64_t at = p.positions != nullptr ? (int64_t)__ldg(p.positions + axis * p.axis_stride + block.token + row) : t0 + row;
    float c = __int_as_float(0x7fc00000), s = c;           // no position of the table: NaN, and counted
    if (at >= 0 && at < p.max_positions) {
      c = __ldg(p.cos_sin + at * p.rot + pair);
      s = __ldg(p.cos_sin + at * p.rot + half + pair);
    }
    sheets[row][pair] = c;
    sheets[row][half + pair] = s;
  }
  if (blockIdx.y == 0 && (int)threadIdx.x >= block.first && (int)threadIdx.x < block.behind && p.status != nullptr) {
    bool bad = false;
    for (int a = 0; a < (p.positions != nullptr ? p.axes : 1); ++a) {
      const int64_t at = p.positions != nullptr ? (int64_t)__ldg(p.positions + a * p.axis_stride + block.token + threadIdx.x) : t0 + threadIdx.x;
      bad = bad || at < 0 || at >= p.max_positions;
    }
    if (bad) atomicAdd(p.status + NVFP4MLA_STAT_BAD_INDEX, 1);
  }
  __syncthreads();
  if (kind == 0) queries<D, kHalf, kInter>(p, block, sheets, head, end);
  else keys<D, kHalf, kInter>(p, block, sheets, head, end);
}

template <int D, bool kHalf>
void launch(const RopeParams& p, bool interleaved, cudaStream_t stream) {
  // CTAs enough for every SM to hold its own, and no more shares of a block than leave each warp a head
  const int64_t want = (int64_t)2 * kRopeBlocks * device_sm_count(), blocks = p.slots < want ? (want + p.slots - 1) / p.slots : 1;
  auto shares_of = [&](int heads, int most) {
    const int each = (heads + kRopeWarps - 1) / kRopeWarps;
    return each < most ? each : most;
  };
  auto per_of = [&](int heads, int shares) { return ((heads + shares - 1) / shares + kRopeWarps - 1) / kRopeWarps * kRopeWarps; };
  const int most = (int)(blocks < 65535 / 4 ? blocks : 65535 / 4);
  const int q_per = per_of(p.heads, shares_of(p.heads, most)), kv_per = per_of(p.kv_heads, shares_of(p.kv_heads, most));
  const int q_shares = (p.heads + q_per - 1) / q_per, kv_shares = (p.kv_heads + kv_per - 1) / kv_per;
  const dim3 grid((unsigned)p.slots, (unsigned)(q_shares + 2 * kv_shares));
  if (interleaved) rope_kernel<D, kHalf, true><<<grid, kRopeWarps * 32, 0, stream>>>(p, q_shares, kv_shares, q_per, kv_per);
  else rope_kernel<D, kHalf, false><<<grid, kRopeWarps * 32, 0, stream>>>(p, q_shares, kv_shares, q_per, kv_per);
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
