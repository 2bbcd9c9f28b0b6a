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
// dims it has eight dims of its own.
//
// A CTA takes a block of 16 tokens of one request and a share of the heads of one kind (queries, keys, values: one code a
// CTA): it stages the cosines and sines of its tokens once, then a warp takes a query's or value's head at a time, two
// warps a key's, whose turned rows are held until the block's scale is known: in registers, but for 40 to 76 bytes a thread
// at 128 dims, where the 64 registers that leave room for four CTAs an SM do not hold all of a key warp's (none at 64).
// Shares are cut finer where blocks are few, down to a head a warp, so that every SM has CTAs.
//
// Measured, back to back, against 6.77 TB/s of measured copy bandwidth: 34,700 prompt tokens of 32 query heads over 8 of
// 128: 146 us (81 %); 512 tokens of 16 trees 5.1 us, one token of 64 requests 7.1 us: latency, as a block's request, lengths,
// positions and angles are read one after the other, and rows, which need none of the angles, only behind the barrier that
// those wait at. A request has two blocks' CTAs at least, so that with one token each half of them have nothing to do (476 of
// 924 here, where 608 run at a time). A warp a key head, whose rows are turned twice, took 159 us;
// kinds mixed in a CTA 235.
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
  // Rows of one head, from load i0 on, x at the lane's row of that; zeros where a row is not new.
  template <int kN>
  __device__ __forceinline__ void load(const uint16_t* x, int64_t stride, int i0, uint4 (&w)[kN]) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (is_new(i0 + i)) {
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
    lane.load(p.q + (b.token + lane.row0) * p.q_token_stride + head * p.q_head_stride, p.q_token_stride, 0, w);
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

// Two warps a head, half of the block's rows each, so that the turned rows stay in registers until the scale is known.
template <int D, bool kHalf, bool kInter>
__device__ __forceinline__ void keys(const RopeParams& p, const Block& b, const float (*sheets)[D], int first_head, int end) {
  using R = Rows<D>;
  constexpr int kN = R::kLoads / 2;
  __shared__ uint32_t tops[2][kRopeWarps];
  const Lane<D, kInter> lane(b, p.rot);
  const bool norm = p.weight[1] != nullptr;
  const int warp = threadIdx.x >> 5, i0 = (warp & 1) * kN;
  Eight g = {};
  if (norm) g = widen8<kHalf>(__ldg(reinterpret_cast<const uint2*>(p.weight[1] + lane.at_a)), __ldg(reinterpret_cast<const uint2*>(p.weight[1] + lane.at_b)));
  // the larger of this warp's and the other's
  auto exchange = [&](int round, uint32_t bits) {
    bits = __reduce_max_sync(kFull, bits);
    if ((threadIdx.x & 31) == 0) tops[round][warp] = bits;
    asm volatile("barrier.cta.sync %0, 64;" ::"r"(1 + (warp >> 1)) : "memory");
    return max(bits, tops[round][warp ^ 1]);
  };
#pragma unroll 1
  for (int head = first_head + (warp >> 1); head < end; head += kRopeWarps / 2) {
    const int64_t row = b.token + i0 * R::kAtOnce + lane.row0;
    uint4 w[kN];
    lane.load(p.x[0] + row * p.token_stride[0] + head * p.head_stride[0], p.token_stride[0], i0, w);
    uint8_t* codes = b.page + kv8_codes_off(p.kv_heads, D, 0, head) + b.quarter * kBlockTokens * D;
    uint8_t* scale = b.page + kv8_scales_off(p.kv_heads, D, head) + b.quarter;
    const uint32_t before = b.first > 0 ? min((uint32_t)*scale, 253u) : 0u;
    Eight y[kN];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      y[i] = widen8<kHalf>(make_uint2(w[i].x, w[i].y), make_uint2(w[i].z, w[i].w));
      turn<D, kInter>(y[i], norm, g, p.eps, lane.turns, sheets[(i0 + i) * R::kAtOnce + lane.row0] + 4 * lane.l, p.rot / 2);
      const float most = fmaxf(fmaxf(fmaxf(fabsf(y[i].a[0].x), fabsf(y[i].a[0].y)), fmaxf(fabsf(y[i].a[1].x), fabsf(y[i].a[1].y))),
                               fmaxf(fmaxf(fabsf(y[i].b[0].x), fabsf(y[i].b[0].y)), fmaxf(fabsf(y[i].b[1].x), fabsf(y[i].b[1].y))));
      if (lane.is_new(i0 + i)) top = fmaxf(top, most);
    }
    // the largest; of the finite ones, once there is an infinity (a NaN is never the larger)
    uint32_t bits = exchange(0, __float_as_uint(top));
    if (__builtin_expect(bits >= 0x7F800000u, 0)) {
      bits = 0;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const float x[8] = {y[i].a[0].x, y[i].a[0].y, y[i].a[1].x, y[i].a[1].y, y[i].b[0].x, y[i].b[0].y, y[i].b[1].x, y[i].b[1].y};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t a = __float_as_uint(x[k]) & 0x7FFFFFFFu;
          if (lane.is_new(i0 + i) && a < 0x7F800000u) bits = max(bits, a);
        }
      }
      bits = exchange(1, bits);
    }
    const uint32_t e = max(scale_byte(__uint_as_float(bits)), before);
    const float mul = __uint_as_float((254u - e) << 23);
    uint8_t* to = codes + (i0 * R::kAtOnce + lane.row0) * D;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      if (!lane.is_new(i0 + i)) continue;
      *reinterpret_cast<uint32_t*>(to + i * R::kAtOnce * D + lane.at_a) = __byte_perm(code2(y[i].a[0], mul), code2(y[i].a[1], mul), 0x5410);
      *reinterpret_cast<uint32_t*>(to + i * R::kAtOnce * D + lane.at_b) = __byte_perm(code2(y[i].b[0], mul), code2(y[i].b[1], mul), 0x5410);
    }
    if ((warp & 1) == 0) {
      if (b.first > 0 && e > before) shrink_rows<D>(codes + 8 * lane.l, lane.row0, b.first, before, e);
      if ((threadIdx.x & 31) == 0) *scale = (uint8_t)e;
    }
    // (what the other reads of `tops` it has read before the next head's exchange is complete)
    asm volatile("barrier.cta.sync %0, 64;" ::"r"(1 + (warp >> 1)) : "memory");
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

// How the heads of a kind are shared by CTAs: n of them, `per` heads each.
struct Shares {
  int n, per;
};

// blockIdx.y: shares of the queries' heads, then of the keys', then of the values', so that a CTA has one code.
template <int D, bool kHalf, bool kInter>
__global__ void __launch_bounds__(kRopeWarps * 32, kRopeBlocks) rope_kernel(const __grid_constant__ RopeParams p, const Shares q, const Shares k, const Shares v) {
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

  const int kind = (int)blockIdx.y < q.n ? 0 : ((int)blockIdx.y < q.n + k.n ? 1 : 2);
  const int share = blockIdx.y - (kind == 0 ? 0 : (kind == 1 ? q.n : q.n + k.n)), per = kind == 0 ? q.per : (kind == 1 ? k.per : v.per);
  const int head = share * per, end = min(kind == 0 ? p.heads : p.kv_heads, head + per);
  if (kind != 0 && !have) return;
  if (kind == 2) {
    values<D, kHalf>(p, block, head + warp, end);
    return;
  }
  // cosines and sines, four pairs at a time: a thread a row and quad
  const int half = p.rot / 2;
  {
    const int row = threadIdx.x & 15;
    const bool vec = (reinterpret_cast<uintptr_t>(p.cos_sin) & 15) == 0;
    const float nan = __int_as_float(0x7fc00000);          // no position of the table: NaN, and counted
#pragma unroll 1
    for (int pair = (threadIdx.x >> 4) * 4; pair < half && row >= block.first && row < block.behind; pair += kRopeWarps * 32 / 16 * 4) {
      auto axis_of = [&](int i) {
        int axis = 0;
#pragma unroll
        for (int a = 0; a < kMaxAxes - 1; ++a) axis += a + 1 < p.axes && i >= p.ends[a] ? 1 : 0;
        return axis;
      };
      auto position = [&](int axis) { return p.positions != nullptr ? (int64_t)__ldg(p.positions + axis * p.axis_stride + block.token + row) : t0 + row; };
      const int axis = axis_of(pair);
      float4 c = make_float4(nan, nan, nan, nan), s = c;
      if (vec && axis_of(pair + 3) == axis) {
        const int64_t at = position(axis);
        if (at >= 0 && at < p.max_positions) {
          c = __ldg(reinterpret_cast<const float4*>(p.cos_sin + at * p.rot + pair));
          s = __ldg(reinterpret_cast<const float4*>(p.cos_sin + at * p.rot + half + pair));
        }
      } else {
        float cs[4], ss[4];
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          const int64_t at = position(axis_of(pair + k));
          const bool in = at >= 0 && at < p.max_positions;
          const float x = in ? __ldg(p.cos_sin + at * p.rot + pair + k) : nan, y = in ? __ldg(p.cos_sin + at * p.rot + half + pair + k) : nan;
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            cs[n] = n == k ? x : cs[n];
            ss[n] = n == k ? y : ss[n];
          }
        }
        c = make_float4(cs[0], cs[1], cs[2], cs[3]);
        s = make_float4(ss[0], ss[1], ss[2], ss[3]);
      }
      *reinterpret_cast<float4*>(sheets[row] + pair) = c;
      *reinterpret_cast<float4*>(sheets[row] + half + pair) = s;
    }
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
  if (kind == 0) queries<D, kHalf, kInter>(p, block, sheets, head + warp, end);
  else keys<D, kHalf, kInter>(p, block, sheets, head, end);
}

template <int D, bool kHalf>
void launch(const RopeParams& p, bool interleaved, cudaStream_t stream) {
  // CTAs enough for every SM to hold its own, and no more shares of a block than leave each warp a head
  const int64_t want = (int64_t)2 * kRopeBlocks * device_sm_count(), blocks = p.slots < want ? (want + p.slots - 1) / p.slots : 1;
  const int most = (int)(blocks < 65535 / 4 ? blocks : 65535 / 4);
  auto shares = [&](int heads, int at_once) {
    const int each = (heads + at_once - 1) / at_once, n = each < most ? each : most;
    const int per = ((heads + n - 1) / n + at_once - 1) / at_once * at_once;
    return Shares{(heads + per - 1) / per, per};
  };
  const Shares q = shares(p.heads, kRopeWarps), k = shares(p.kv_heads, kRopeWarps / 2), v = shares(p.kv_heads, kRopeWarps);
  const dim3 grid((unsigned)p.slots, (unsigned)(q.n + k.n + v.n));
  if (interleaved) rope_kernel<D, kHalf, true><<<grid, kRopeWarps * 32, 0, stream>>>(p, q, k, v);
  else rope_kernel<D, kHalf, false><<<grid, kRopeWarps * 32, 0, stream>>>(p, q, k, v);
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
