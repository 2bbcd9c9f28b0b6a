// spec_verify: which drafted tokens the target's distribution accepts, and the token after them.
//
// What it computes. p_j is the softmax of node j's logits over their temperature. From node 0 on, the
// children of the current node are tried in order: with r = p and s = 1 at first, a child's token x is taken
// when u q(x) s < r(x), else r becomes max(r - s q, 0) and s the sum of r. (q: the distribution that the
// children were drawn from; a draft without one stands for itself, q(x) = 1, and its refusal takes x out of
// r.) When no child is taken, the next token is drawn from r by its running sum.
//
// What bounds it. The answer needs the rows of the nodes that the walk reaches, one more than are accepted, and a row of
// the drafts' distribution for each of those at which a child is refused; which ones these are is known on the way only. So
// stats_kernel reads every node's row once, for its largest value and its sum of exponentials, before the walk: memory,
// where there are many rows, most of which a tree's walk does not come to. It goes by chunks of 4 KB, a warp each, whose
// values stay in registers; the chunks' sums are kept, since with them a token can be drawn by reading a single chunk
// again. walk_kernel has a CTA a request (with draft distributions a cluster of eight, since what a refusal leaves is a sum
// over the vocabulary): all nodes' probabilities are found at once, so that the walk itself is a few comparisons. It is a
// chain of some eight dependent reads, and of code that runs once. Running sums over chunks are in 64 bits: what is drawn
// changes where they cross a border between tokens.
//
// Measured, back to back: 64 chains of 5 nodes over 128,000 bf16 logits with draft distributions 31 us, of which some 17
// are stats_kernel's (82 MB at 71 % of the 6.77 TB/s of measured copy bandwidth) and 14 the walk's: the rows that were
// needed, 2.7 of 5 a request, and the distributions are 61 MB, 9 us. 16 trees of 32 over 100,003 without distributions 30
// us (20 for 99 MB, and 10): of 31 rows a request 2.2 were needed, 7 MB, 1 us. One chain of 5 over 32,000 fp32 10 us (all
// latency). What was tried and not kept: chunks that come to shared memory ahead of a warp's work, by a ring of three a
// warp (37 to 40, 37 and 12 us); a walk in 64 bits, or unrolled (its code is fetched once a call, some 16 cycles an
// instruction); the next distribution brought to L2 (no difference).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>

#include "../../include/nvfp4mla.h"
#include "kv8.h"
#include "ptx.cuh"

namespace nvfp4mla {
namespace {

using namespace ptx;

constexpr int kChunkBytes = 4096;      // of a row that a warp takes: eight 16-byte loads a lane, all in flight
constexpr int kStatsThreads = 128;
constexpr int kWalkCtas = 8;           // of a request, with draft distributions
constexpr int kMaxNodes = 64;
constexpr int kFine = 8;               // warps' loads of a chunk
constexpr unsigned kFull = 0xFFFFFFFFu;

template <typename T>
struct Vec {
  static constexpr int kN = 16 / (int)sizeof(T);           // logits of a load
  static constexpr int kChunk = kChunkBytes / (int)sizeof(T);
  static constexpr int kLoads = kChunkBytes / (32 * 16);
};

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
// The logits of a load as they are.
__device__ __forceinline__ void widen(const uint4& w, float (&x)[4], const float*) {
  x[0] = __uint_as_float(w.x);
  x[1] = __uint_as_float(w.y);
  x[2] = __uint_as_float(w.z);
  x[3] = __uint_as_float(w.w);
}
template <typename T>
__device__ __forceinline__ void widen(const uint4& w, float (&x)[8], const T*) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float2 two;
    if constexpr (sizeof(T) == 2 && __is_same(T, __half)) two = __half22float2(*reinterpret_cast<const __half2*>(&ws[k]));
    else two = make_float2(__uint_as_float(ws[k] << 16), __uint_as_float(ws[k] & 0xFFFF0000u));
    x[2 * k] = two.x;
    x[2 * k + 1] = two.y;
  }
}
// A NaN is no candidate.
__device__ __forceinline__ float clean(float v) { return v != v ? neg_inf() : v; }

// log2(e) / temperature as hi + lo: rounded to one fp32, its error would grow with a logit's distance from the
// largest. Both above 0, so that an infinite distance stays one, but by no more than fp32's smallest step: at an infinite
// temperature the largest finite distance, 2^128, then costs a weight 2 x 2^-149 x 2^128 = 2^-20 of an exponent.
// hi < 0: greedy, which is asked for by 0 (and by what is no temperature).
struct Rate {
  float hi, lo;
};
__device__ __forceinline__ Rate rate_of(const VerifyParams& p, int b) {
  const float t = p.temperatures != nullptr ? p.temperatures[b] : 1.f;
  if (!(t > 0.f)) return Rate{-1.f, 0.f};
  constexpr float kHi = 1.4426950408889634f, kLo = (float)(1.4426950408889634 - (double)kHi);
  const float step = __int_as_float(1);
  float hi = fmaxf(kHi / t, step);
  if (!(hi < 3e38f)) return Rate{3e38f, step};
  if (hi > 1e-30f) hi = __uint_as_float(__float_as_uint(hi) - 1);        // at or below the quotient
  return Rate{hi, fmaxf((fmaf(-hi, t, kHi) + kLo) / t, step)};
}
// exp((x - m) / T) for x <= m; 0 for x = -inf, 1 for x = m whatever they are.
__device__ __forceinline__ float weight(float x, float m, Rate rate) {
  const float d = x - m;
  return x == neg_inf() ? 0.f : (x == m ? 1.f : ex2_approx(fmaf(d, rate.hi, d * rate.lo)));
}

// A row's chunks begin at 16-byte boundaries, so that the first may begin before the row.
template <typename T>
__device__ __forceinline__ int lead_of(const T* row) {
  return (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
}
template <typename T>
__device__ __forceinline__ int chunks_of(const T* row, int V) {
  return (int)(((int64_t)V + lead_of(row) + Vec<T>::kChunk - 1) / Vec<T>::kChunk);
}
// The load from logit `at` on, -inf outside of the row.
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T* row, int64_t at, int64_t V) {
  if (at >= 0 && at + Vec<T>::kN <= V) return __ldg(reinterpret_cast<const uint4*>(row + at));
  constexpr uint32_t kInf = sizeof(T) == 4 ? 0xff800000u : (__is_same(T, __half) ? 0xfc00fc00u : 0xff80ff80u);
  uint4 w = make_uint4(kInf, kInf, kInf, kInf);
  T* t = reinterpret_cast<T*>(&w);
  for (int k = 0; k < Vec<T>::kN; ++k)
    if (at + k >= 0 && at + k < V) t[k] = row[at + k];
  return w;
}

__device__ __forceinline__ bool is_node(const VerifyParams& p, int row) {
  const int j = row % p.Q;
  if (j == 0) return true;
  const int up = p.parents[row];
  return up >= 0 && up < j;
}

// The largest, whatever a NaN beside it.
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// The largest logit of some loads; a NaN counts as none. Pairs of 16 bits are compared as they are.
template <int kLoads>
__device__ __forceinline__ float largest_of(const uint4 (&w)[kLoads], const float*) {
  float m = neg_inf();
#pragma unroll
  for (int i = 0; i < kLoads; ++i)
    m = fmaxf(fmaxf(fmaxf(m, __uint_as_float(w[i].x)), fmaxf(__uint_as_float(w[i].y), __uint_as_float(w[i].z))), __uint_as_float(w[i].w));
  return m;
}
template <int kLoads, typename T>
__device__ __forceinline__ float largest_of(const uint4 (&w)[kLoads], const T*) {
  uint32_t m[2] = {w[0].x, w[0].y};
  auto more = [](uint32_t& m, uint32_t x) {
    if constexpr (__is_same(T, __half)) asm("max.f16x2 %0, %0, %1;" : "+r"(m) : "r"(x));
    else asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(x));
  };
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    more(m[0], w[i].x);
    more(m[1], w[i].y);
    more(m[0], w[i].z);
    more(m[1], w[i].w);
  }
  more(m[0], m[1]);
  float two[8];
  widen(make_uint4(m[0], m[0], m[0], m[0]), two, (const T*)nullptr);
  return fmaxf(fmaxf(two[0], two[1]), neg_inf());        // (-inf, should all of them be NaN)
}

// A chunk's largest logit, and the sum of its exponentials against that; greedy: where the largest is first.
template <typename T>
__global__ void __launch_bounds__(kStatsThreads) stats_kernel(const __grid_constant__ VerifyParams p) {
  using V = Vec<T>;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x, chunk = blockIdx.y * (kStatsThreads / 32) + (threadIdx.x >> 5);
  const T* row = static_cast<const T*>(p.logits) + (int64_t)r * p.row_stride;
  const int64_t at = (int64_t)chunk * V::kChunk - lead_of(row);
  if (at >= p.V || !is_node(p, r)) return;
  uint4 w[V::kLoads];
#pragma unroll
  for (int i = 0; i < V::kLoads; ++i) w[i] = load_vec(row, at + (i * 32 + lane) * V::kN, p.V);
  const Rate rate = rate_of(p, r / p.Q);
  const float m = warp_max(largest_of(w, row));
  const int64_t to = (int64_t)r * p.chunks + chunk;
  if (rate.hi < 0.f) {
    int where = INT_MAX;
#pragma unroll
    for (int i = V::kLoads - 1; i >= 0; --i) {
      float x[V::kN];
      widen(w[i], x, row);
#pragma unroll
      for (int k = V::kN - 1; k >= 0; --k) where = x[k] == m ? (int)(at + (i * 32 + lane) * V::kN + k) : where;
    }
    where = __reduce_min_sync(kFull, where);
    if (lane == 0) {
      p.chunk_ms[to] = make_float2(m, 0.f);
      p.chunk_at[to] = where;
    }
    return;
  }
  float sum = 0.f;
  if (fabsf(m) < __int_as_float(0x7f800000)) {
    const float2 less = make_float2(-m, -m), hi = make_float2(rate.hi, rate.hi), lo = make_float2(rate.lo, rate.lo);
    float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int i = 0; i < V::kLoads; ++i) {
      float x[V::kN];
      widen(w[i], x, row);
#pragma unroll
      for (int k = 0; k < V::kN; k += 2) {
        const float2 d = __fadd2_rn(make_float2(x[k], x[k + 1]), less);
        const float2 e = __ffma2_rn(d, hi, __fmul2_rn(d, lo));
        part[(k >> 1) & 1] = __fadd2_rn(part[(k >> 1) & 1], make_float2(ex2_approx(e.x), ex2_approx(e.y)));
      }
    }
    sum = (part[0].x + part[0].y) + (part[1].x + part[1].y);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
  }
  if (!(sum > 0.f) || !(fabsf(m) < __int_as_float(0x7f800000))) {
    // a NaN, or infinities
    sum = 0.f;
#pragma unroll 1
    for (int i = 0; i < V::kLoads; ++i) {
      float x[V::kN];
      widen(load_vec(row, at + (i * 32 + lane) * V::kN, p.V), x, row);
      for (int k = 0; k < V::kN; ++k) sum += weight(clean(x[k]), m, rate);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
  }
  if (lane == 0) p.chunk_ms[to] = make_float2(m, sum);
}

struct WalkShared {
  float top[kMaxNodes];                // a node's largest logit
  float inverse[kMaxNodes];            // 1 / its sum of exponentials against that
  int best[kMaxNodes];
  float have[kMaxNodes];               // probability of a draft's token under its parent
  float drawn[kMaxNodes];              // and under what it was drawn from
  int parent[kMaxNodes], token[kMaxNodes];
  float u[kMaxNodes];
  float left[kMaxNodes];               // s before each refusal at the current node
  int out[kMaxNodes];                  // tokens that were refused there
  double sum;                          // of what is left
  float part[2][kFine], need;
  int entry, pick, last;
  // the walk
  int at, count, refused, next_node, ends;
};

template <typename T, bool kProbs, int kThreads>
struct Walker {
  using V = Vec<T>;
  static constexpr int kWarps = kThreads / 32;
  const VerifyParams& p;
  WalkShared& sh;
  int b, rank, ctas;
  Rate rate;

  __device__ const T* row_of(int j) const { return static_cast<const T*>(p.logits) + ((int64_t)b * p.Q + j) * p.row_stride; }
  __device__ const float* probs_of(int j) const { return p.probs + ((int64_t)b * p.Q + j) * p.probs_stride; }

  // Code that a CTA runs once costs what its fetching costs, some 16 cycles an instruction: so every thread has one load
  // of a chunk, and the loops are loops.
  struct Load {
    float x[V::kN];
  };
  // What is left, after `refused` refusals at node j, of the tokens of the load from `at` on: of their probabilities (with
  // draft distributions), or of their exponentials.
  struct Raw {
    uint4 w;
    Load q;                              // of the distribution that refusals take off
  };
  __device__ __forceinline__ Raw ask(int j, int64_t at, int refused) const {
    Raw r;
    r.w = load_vec(row_of(j), at, p.V);
    Load& q = r.q;
    if (kProbs && refused > 0) {
      const float* from = probs_of(j) + at;
      if (at >= 0 && at + V::kN <= p.V && (reinterpret_cast<uintptr_t>(from) & 15) == 0) {
#pragma unroll
        for (int k = 0; k < V::kN; k += 4) *reinterpret_cast<float4*>(q.x + k) = __ldg(reinterpret_cast<const float4*>(from + k));
      } else {
#pragma unroll
        for (int k = 0; k < V::kN; ++k) q.x[k] = at + k >= 0 && at + k < p.V ? __ldg(from + k) : 0.f;
      }
    }
    return r;
  }
  __device__ __forceinline__ Load rest(const Raw& raw, int j, int64_t at, int refused) const {
    const float m = sh.top[j], inv = kProbs ? sh.inverse[j] : 1.f;
    const Load& q = raw.q;
    Load r;
    widen(raw.w, r.x, (const T*)nullptr);
    if (fabsf(m) < __int_as_float(0x7f800000)) {
#pragma unroll
      for (int k = 0; k < V::kN; ++k) {
        const float d = fmaxf(r.x[k], neg_inf()) - m;      // (a NaN is no candidate)
        r.x[k] = ex2_approx(fmaf(d, rate.hi, d * rate.lo)) * inv;
      }
    } else {
#pragma unroll
      for (int k = 0; k < V::kN; ++k) r.x[k] = r.x[k] == m && m != neg_inf() ? inv : 0.f;
    }
#pragma unroll 1
    for (int i = 0; i < refused; ++i) {
      const float s = sh.left[i];
      const int64_t out = sh.out[i] - at;
#pragma unroll
      for (int k = 0; k < V::kN; ++k) r.x[k] = kProbs ? fmaxf(fmaf(-s, q.x[k], r.x[k]), 0.f) : (out == k ? 0.f : r.x[k]);
    }
    return r;
  }
  __device__ __forceinline__ Load rest(int j, int64_t at, int refused) const { return rest(ask(j, at, refused), j, at, refused); }
  static __device__ __forceinline__ float add_up(const Load& r) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < V::kN; ++k) s += r.x[k];
    return s;
  }
  static __device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(kFull, x, d);
    return x;
  }

  __device__ __forceinline__ float rest_of_warp(int j, int64_t at, int refused) const { return warp_sum(add_up(rest(j, at, refused))); }

  // What is left at node j is summed by entries: a warp's loads, where a distribution has been taken off, else chunks.
  __device__ __forceinline__ bool fine(int refused) const { return kProbs && refused > 0; }
  __device__ __forceinline__ int entry_tokens(int refused) const { return fine(refused) ? 32 * V::kN : V::kChunk; }
  __device__ int entries(int j, int refused) const {
    return (p.V + lead_of(row_of(j)) + entry_tokens(refused) - 1) / entry_tokens(refused);
  }
  __device__ __forceinline__ double* entry_sums() const { return p.entry_sum + (int64_t)b * p.chunks * kFine; }

  // The entries' sums, and from there of all: sh.sum, the same in every CTA. A lane of warp 0 has a run of them; returns
  // what lies before it, and what it has. again: not the first time.
  __device__ double2 sums(int j, int refused, bool again) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = entries(j, refused);
    double* to = entry_sums();
    if (again) {                         // (all have read the sums before these)
      if (ctas > 1) cluster_sync_all();
      else __syncthreads();
    }
    const int64_t start = -(int64_t)lead_of(row_of(j));
    if (fine(refused)) {
      // (the next entry's loads are on their way while this one's are added up)
      auto at_of = [&](int c) { return start + ((int64_t)c * 32 + lane) * V::kN; };
      int c = rank * kWarps + warp;
      Raw next{};
      if (c < n) next = ask(j, at_of(c), refused);
#pragma unroll 1
      for (; c < n; c += ctas * kWarps) {
        const Raw now = next;
        if (c + ctas * kWarps < n) next = ask(j, at_of(c + ctas * kWarps), refused);
        const float s = warp_sum(add_up(rest(now, j, at_of(c), refused)));
        if (lane == 0) to[c] = (double)s;
      }
    } else if (rank == 0) {
      const int64_t first = ((int64_t)b * p.Q + j) * p.chunks;
      const float m = sh.top[j], scale = kProbs ? sh.inverse[j] : 1.f;
#pragma unroll 1
      for (int c = threadIdx.x; c < n; c += kThreads) {
        const float2 ms = __ldcg(p.chunk_ms + first + c);
        to[c] = (double)(ms.y * weight(ms.x, m, rate) * scale);
      }
      if (!kProbs && refused > 0) {
        // again, where a refused token lies: eight warps a chunk
        __syncthreads();
        constexpr int kGroups = kWarps / kFine;
#pragma unroll 1
        for (int i0 = 0; i0 < refused; i0 += kGroups) {
          const int group = warp / kFine, i = i0 + group;
          const int c = i < refused ? (int)((sh.out[i] - start) / V::kChunk) : 0;
          if (i < refused) {
            const float s = rest_of_warp(j, start + (int64_t)c * V::kChunk + (threadIdx.x & 255) * V::kN, refused);
            if (lane == 0) sh.part[group][warp % kFine] = s;
          }
          __syncthreads();
          if (i < refused && (threadIdx.x & 255) == 0) {
            float s = 0.f;
#pragma unroll 1
            for (int k = 0; k < kFine; ++k) s += sh.part[group][k];
            to[c] = (double)s;           // (two refused tokens of a chunk: the same sum twice)
          }
          __syncthreads();
        }
      }
    }
    if (ctas > 1) cluster_sync_all();
    else __syncthreads();
    double mine = 0., incl = 0.;
    if (warp == 0) {
      const int per = (n + 31) / 32;
#pragma unroll 8
      for (int i = 0; i < per; ++i) mine += lane * per + i < n ? __ldcg(to + lane * per + i) : 0.;
      incl = mine;
#pragma unroll 1
      for (int d = 1; d < 32; d <<= 1) {
        const double o = __shfl_up_sync(kFull, incl, d);
        if (lane >= d) incl += o;
      }
      if (lane == 31) sh.sum = incl;
      if (lane == 0) {
        sh.entry = sh.pick = INT_MAX;
        sh.last = -1;
      }
    }
    __syncthreads();
    return make_double2(incl - mine, mine);
  }

  // The first token whose running sum of what is left at node j exceeds `share` of it all, else the last that has
  // anything: the threads of one CTA, behind sums(), whose result is `run`.
  __device__ int draw(int j, float share, double2 run, int refused) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = entries(j, refused);
    if (warp == 0) {
      const double* of = entry_sums();
      const double want = (double)share * sh.sum;
      const int per = (n + 31) / 32;
      // the lane whose run crosses the border, else the last that has anything; and there, 32 entries at a time
      const unsigned some = __ballot_sync(kFull, run.y > 0.), past = __ballot_sync(kFull, run.y > 0. && run.x + run.y > want);
      if (some != 0) {
        const int of_lane = past != 0 ? __ffs(past) - 1 : 31 - __clz(some);
        double before = __shfl_sync(kFull, run.x, of_lane);
        int entry = -1;
        double at_entry = 0.;
#pragma unroll 1
        for (int i0 = 0; i0 < per; i0 += 32) {
          const int i = of_lane * per + i0 + lane;
          const double x = i0 + lane < per && i < n ? __ldcg(of + i) : 0.;
          double incl = x;
#pragma unroll 1
          for (int d = 1; d < 32; d <<= 1) {
            const double o = __shfl_up_sync(kFull, incl, d);
            if (lane >= d) incl += o;
          }
          const unsigned has = __ballot_sync(kFull, x > 0.), over = __ballot_sync(kFull, x > 0. && before + incl > want);
          const int pick = over != 0 ? __ffs(over) - 1 : 31 - __clz(has);
          if (has != 0) {
            entry = __shfl_sync(kFull, i, pick);
            at_entry = __shfl_sync(kFull, before + (incl - x), pick);
          }
          if (over != 0) break;
          before += __shfl_sync(kFull, incl, 31);
        }
        if (lane == 0 && entry >= 0) {
          sh.entry = entry;
          sh.need = (float)(want - at_entry);
        }
      }
    }
    __syncthreads();
    const int entry = sh.entry, loads = entry_tokens(refused) / V::kN;
    if (entry == INT_MAX) return -1;
    const int64_t at = (int64_t)entry * entry_tokens(refused) - lead_of(row_of(j)) + threadIdx.x * V::kN;
    Load r;
    float sum = 0.f, incl = 0.f;
    if (warp * 32 < loads) {
      r = rest(j, at, refused);
      incl = sum = add_up(r);
#pragma unroll 1
      for (int d = 1; d < 32; d <<= 1) {
        const float o = __shfl_up_sync(kFull, incl, d);
        if (lane >= d) incl += o;
      }
      if (lane == 31) sh.part[0][warp] = incl;
    }
    __syncthreads();
    if (warp * 32 < loads) {
      float run = incl - sum;
#pragma unroll 1
      for (int k = 0; k < warp; ++k) run += sh.part[0][k];
#pragma unroll
      for (int k = 0; k < V::kN; ++k) {
        run += r.x[k];
        if (r.x[k] > 0.f) {
          atomicMax(&sh.last, (int)(at + k));
          if (run > sh.need) atomicMin(&sh.pick, (int)(at + k));
        }
      }
    }
    __syncthreads();
    return sh.pick != INT_MAX ? sh.pick : sh.last;
  }

  // From where the walk stands to its end, or to a refusal behind which a sum is needed: warp 0. left: s of what is left,
  // below 0 where it is not known.
  __device__ void walk(bool greedy, float left) {
    const int lane = threadIdx.x & 31;
    const int up0 = lane < p.Q ? sh.parent[lane] : -1, up1 = 32 + lane < p.Q ? sh.parent[32 + lane] : -1;
    int at = sh.at, count = sh.count, refused = sh.refused, from = sh.next_node;
    bool ends = true;
    __syncwarp();
    for (;;) {
      // the next child of the current node
      const uint64_t children = ((uint64_t)__ballot_sync(kFull, up1 == at) << 32 | __ballot_sync(kFull, up0 == at)) & (from < 64 ? ~0ull << from : 0ull);
      if (children == 0) break;
      const int j = __ffsll((long long)children) - 1;
      from = j + 1;
      bool yes;
      if (greedy) {
        yes = sh.best[at] == sh.token[j];
      } else {
        if (kProbs && left < 0.f) {      // another child after a refusal
          from = j;
          ends = false;
          break;
        }
        float r = sh.have[j];
        const float q = sh.drawn[j];
#pragma unroll 1
        for (int i = 0; i < refused; ++i) {
          if (kProbs) r = fmaxf(fmaf(-sh.left[i], q, r), 0.f);
          else if (sh.out[i] == sh.token[j]) r = 0.f;
        }
        yes = sh.u[j] * q * left < r;
        if (!yes) {
          __syncwarp();
          if (lane == 0) {
            sh.left[refused] = left;
            sh.out[refused] = sh.token[j];
          }
          __syncwarp();
          ++refused;
          left = kProbs ? -1.f : fmaxf(left - r, 0.f);      // (below 0 after a refusal that was asked for)
        }
      }
      if (yes) {
        if (rank == 0 && lane == 0) {
          p.path[(int64_t)b * p.Q + count] = j;
          p.tokens[(int64_t)b * p.Q + count] = sh.token[j];
        }
        ++count;
        at = j;
        refused = 0;
        left = 1.f;
      }
    }
    if (lane == 0) {
      sh.at = at;
      sh.count = count;
      sh.refused = refused;
      sh.next_node = from;
      sh.ends = ends;
    }
  }
};

template <typename T, bool kProbs, int kThreads>
__global__ void __launch_bounds__(kThreads) walk_kernel(const __grid_constant__ VerifyParams p) {
  constexpr int kWarps = kThreads / 32;
  __shared__ WalkShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ctas = kProbs ? kWalkCtas : 1, b = blockIdx.x / ctas, rank = kProbs ? (int)cluster_ctarank() : 0;
  const int Q = p.Q;
  const Rate rate = rate_of(p, b);
  const bool greedy = rate.hi < 0.f;
  Walker<T, kProbs, kThreads> w{p, sh, b, rank, ctas, rate};
  bool bad = false;
  float logit = 0.f;
  if (tid < Q) {
    const int64_t r = (int64_t)b * Q + tid;
    int up = tid == 0 ? -1 : p.parents[r];
    const int x = p.drafts[r];
    if (tid > 0 && up != -1) {
      bad = up < 0 || up >= tid || x < 0 || x >= p.V;
      if (bad) up = -1;
    }
    sh.parent[tid] = up;
    sh.token[tid] = x;
    const float u = p.uniforms[r];
    sh.u[tid] = u < 1.f ? fmaxf(u, 0.f) : __int_as_float(0x7f800000);
    sh.drawn[tid] = kProbs && up >= 0 ? __ldg(w.probs_of(up) + x) : 1.f;
    if (up >= 0) logit = clean(as_float(w.row_of(up)[x]));
  }
  if (tid == 0) {
    sh.at = sh.count = sh.refused = 0;
    sh.next_node = 1;
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // nodes' largest logits and sums, a warp a node
#pragma unroll 1
  for (int j = warp; j < Q; j += kWarps) {
    if (j > 0 && sh.parent[j] < 0) continue;
    const int64_t first = ((int64_t)b * Q + j) * p.chunks;
    const int chunks = chunks_of(w.row_of(j), p.V);
    float m = neg_inf(), sum = 0.f;
    int where = INT_MAX;
#pragma unroll 1
    for (int c0 = 0; c0 < chunks; c0 += 128) {           // four loads in flight
      float2 ms[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) ms[i] = c0 + i * 32 + lane < chunks ? __ldcg(p.chunk_ms + first + c0 + i * 32 + lane) : make_float2(neg_inf(), 0.f);
      const float now = warp_max(fmaxf(fmaxf(m, fmaxf(ms[0].x, ms[1].x)), fmaxf(ms[2].x, ms[3].x)));
      if (greedy) {
        if (now > m) {
#pragma unroll
          for (int i = 3; i >= 0; --i) where = ms[i].x == now ? c0 + i * 32 + lane : where;
          where = __reduce_min_sync(kFull, ms[0].x == now || ms[1].x == now || ms[2].x == now || ms[3].x == now ? where : INT_MAX);
        }
      } else {
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) part += ms[i].y * weight(ms[i].x, now, rate);
        sum = fmaf(sum, weight(m, now, rate), part);
      }
      m = now;
    }
    sum = w.warp_sum(sum);
    if (lane == 0) {
      sh.top[j] = m;
      sh.inverse[j] = sum > 0.f ? 1.f / sum : 0.f;
      sh.best[j] = greedy && m != neg_inf() ? __ldcg(p.chunk_at + first + where) : -1;
    }
  }
  __syncthreads();
  if (tid < Q && sh.parent[tid] >= 0 && !greedy) {
    const int up = sh.parent[tid];
    const float m = sh.top[up], d = logit - m, a = d * rate.hi;
    // exp2 of a, and of what rounding took from it; 0 where that is 0, as of a distance so wide (from +inf, of the type's lowest
    // number) that d or a is infinite, when the rest is none
    const float e = exp2f(a), have = logit == m ? (m == neg_inf() ? 0.f : 1.f) : (e > 0.f ? fmaf(e, 0.69314718f * (fmaf(d, rate.hi, -a) + d * rate.lo), e) : 0.f);
    sh.have[tid] = have * sh.inverse[up];
  }
  __syncthreads();
  if (warp == 0) w.walk(greedy, 1.f);
  __syncthreads();
  bool again = false;
  if constexpr (kProbs) {
    while (!sh.ends) {
      const int at = sh.at, refused = sh.refused;
      w.sums(at, refused, again);
      again = true;
      if (warp == 0) w.walk(greedy, (float)sh.sum);
      __syncthreads();
    }
  }
  const int at = sh.at, count = sh.count;
  int refused = sh.refused, next = greedy ? sh.best[at] : -1;
  if (!greedy && sh.top[at] != neg_inf()) {
    double2 run = w.sums(at, refused, again);
    if (!(sh.sum > 0.) && refused > 0) {   // nothing is left: from the target's own
      refused = 0;
      run = w.sums(at, 0, true);
    }
    if (rank == 0) next = w.draw(at, sh.u[0], run, refused);
  }
  if (rank == 0) {
    if (tid == 0) {
      p.tokens[(int64_t)b * Q + count] = next;
      p.path[(int64_t)b * Q + count] = -1;
      p.accepted[b] = count;
    }
    if (tid > count && tid < Q) {
      p.tokens[(int64_t)b * Q + tid] = -1;
      p.path[(int64_t)b * Q + tid] = -1;
    }
    if (p.status != nullptr && (bad || (tid == 0 && next < 0))) atomicAdd(p.status + NVFP4MLA_STAT_BAD_INDEX, 1);
  }
}

template <typename T, bool kProbs, int kThreads>
cudaError_t launch_walk(const VerifyParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * (kProbs ? kWalkCtas : 1)), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kWalkCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kProbs ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, walk_kernel<T, kProbs, kThreads>, p);
}

template <typename T>
cudaError_t launch(VerifyParams p, cudaStream_t stream) {
  p.chunks = (p.V + Vec<T>::kN - 1) / Vec<T>::kChunk + 1;
  const dim3 grid((unsigned)(p.B * p.Q), (unsigned)((p.chunks + kStatsThreads / 32 - 1) / (kStatsThreads / 32)));
  stats_kernel<T><<<grid, kStatsThreads, 0, stream>>>(p);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  return p.probs != nullptr ? launch_walk<T, true, 256>(p, stream) : launch_walk<T, false, 512>(p, stream);
}

}  // namespace

int verify_chunks(int64_t V) { return (int)((V + 7) / (kChunkBytes / 4) + 1); }
int verify_entries(int64_t V) { return verify_chunks(V) * kFine; }
int verify_requests() { return INT_MAX / kWalkCtas; }

cudaError_t launch_spec_verify(const VerifyParams& p, int type, cudaStream_t stream) {
  if (type == NVFP4MLA_FP32) return launch<float>(p, stream);
  return type == NVFP4MLA_FP16 ? launch<__half>(p, stream) : launch<__nv_bfloat16>(p, stream);
}

}  // namespace nvfp4mla
