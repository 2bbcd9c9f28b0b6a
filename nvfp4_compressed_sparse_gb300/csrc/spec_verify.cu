// spec_verify: which drafted tokens the target's distribution accepts, and the token after them.
//
// What it computes. p_j is the softmax of node j's logits over their temperature. From node 0 on, the
// children of the current node are tried in order: with r = p and s = 1 at first, a child's token x is taken
// when u q(x) s < r(x), else r becomes max(r - s q, 0) and s the sum of r. (q: the distribution that the
// children were drawn from; a draft without one stands for itself, q(x) = 1, and its refusal takes x out of
// r.) When no child is taken, the next token is drawn from r by its running sum.
//
// What bounds it. Every row of logits is read once, for its largest value and its sum of exponentials.
// stats_kernel does that by chunks of 1,024 logits, a warp each, whose values stay in registers; the chunks'
// sums are kept, since with them a token can be drawn by reading a single chunk again. walk_kernel has a CTA
// a request (with draft distributions a cluster of eight, since what a refusal leaves is a sum over the
// vocabulary): all nodes' probabilities are found at once, so that the walk itself is a few comparisons.
// Sums over chunks, and what is compared, are in 64 bits: the results are whole numbers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>

#include "../../include/nvfp4mla.h"
#include "kv8.h"
#include "ptx.cuh"

namespace nvfp4mla {
namespace {

using namespace ptx;

constexpr int kChunk = 1024;           // logits
constexpr int kStatsThreads = 256;
constexpr int kWalkThreads = 256, kWalkWarps = kWalkThreads / 32;
constexpr int kWalkCtas = 8;           // of a request, with draft distributions
constexpr int kMaxNodes = 64;
constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
// A NaN is no candidate.
template <typename T>
__device__ __forceinline__ float logit(T x) {
  const float v = as_float(x);
  return v != v ? neg_inf() : v;
}

// log2(e) / temperature as hi + lo: rounded to one fp32, its error would grow with a logit's distance from the
// largest. hi < 0: greedy, which is asked for by 0 (and by what is no temperature).
struct Rate {
  float hi, lo;
};
__device__ __forceinline__ Rate rate_of(const VerifyParams& p, int b) {
  const float t = p.temperatures != nullptr ? p.temperatures[b] : 1.f;
  if (!(t > 0.f)) return Rate{-1.f, 0.f};
  constexpr float kHi = 1.4426950408889634f, kLo = (float)(1.4426950408889634 - (double)kHi);
  const float hi = kHi / t;
  if (!(hi < 3e38f)) return Rate{3e38f, 0.f};
  return Rate{hi, (fmaf(-hi, t, kHi) + kLo) / t};
}
// exp((x - m) / T) for x <= m; 0 for x = -inf, 1 for x = m whatever they are.
__device__ __forceinline__ float weight(float x, float m, Rate rate) {
  const float d = x - m;
  return x == neg_inf() ? 0.f : (x == m ? 1.f : ex2_approx(fmaf(d, rate.hi, d * rate.lo)));
}

template <typename T>
struct Vec {
  static constexpr int kN = 16 / (int)sizeof(T);
};

// A row's chunks begin at 16-byte boundaries, so that the first may begin before the row.
template <typename T>
__device__ __forceinline__ int lead_of(const T* row) {
  return (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
}
// The kN logits from `at` on, -inf outside of the row.
template <typename T>
__device__ __forceinline__ void load_vec(const T* row, int64_t at, int64_t V, float (&x)[Vec<T>::kN]) {
  constexpr int kN = Vec<T>::kN;
  if (at >= 0 && at + kN <= V) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(row + at));
    const T* t = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int k = 0; k < kN; ++k) x[k] = logit(t[k]);
  } else {
#pragma unroll
    for (int k = 0; k < kN; ++k) x[k] = at + k >= 0 && at + k < V ? logit(row[at + k]) : neg_inf();
  }
}

__device__ __forceinline__ bool is_node(const VerifyParams& p, int64_t row) {
  const int j = (int)(row % p.Q);
  if (j == 0) return true;
  const int up = p.parents[row];
  return up >= 0 && up < j;
}

template <typename T>
__global__ void __launch_bounds__(kStatsThreads) stats_kernel(const VerifyParams p) {
  constexpr int kN = Vec<T>::kN, kLoads = kChunk / (32 * kN);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * (kStatsThreads / 32) + (threadIdx.x >> 5);
  const int64_t r = item / p.chunks;
  const int chunk = (int)(item - r * p.chunks);
  if (r >= (int64_t)p.B * p.Q || !is_node(p, r)) return;
  const T* row = static_cast<const T*>(p.logits) + r * p.row_stride;
  const int64_t at = (int64_t)chunk * kChunk - lead_of(row);
  if (at >= p.V) return;
  float x[kLoads][kN];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) load_vec(row, at + (i * 32 + lane) * kN, p.V, x[i]);
  const Rate rate = rate_of(p, (int)(r / p.Q));
  float m = neg_inf();
  int where = INT_MAX;
#pragma unroll
  for (int i = 0; i < kLoads; ++i)
#pragma unroll
    for (int k = 0; k < kN; ++k)
      if (x[i][k] > m) {
        m = x[i][k];
        where = (int)(at + (i * 32 + lane) * kN + k);
      }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const float om = __shfl_xor_sync(kFull, m, d);
    const int ow = __shfl_xor_sync(kFull, where, d);
    if (om > m || (om == m && ow < where)) {
      m = om;
      where = ow;
    }
  }
  float sum = 0.f;
  if (rate.hi >= 0.f) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
#pragma unroll
      for (int k = 0; k < kN; ++k) sum += weight(x[i][k], m, rate);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
  }
  if (lane == 0) {
    p.chunk_ms[r * p.chunks + chunk] = make_float2(m, sum);
    p.chunk_at[r * p.chunks + chunk] = where;
  }
}

struct WalkShared {
  float top[kMaxNodes];                // a node's largest logit
  double total[kMaxNodes];             // its sum of exponentials against that
  int best[kMaxNodes];
  double have[kMaxNodes];              // probability of a draft's token under its parent
  float drawn[kMaxNodes];              // and under what it was drawn from
  int parent[kMaxNodes], token[kMaxNodes];
  float u[kMaxNodes];
  double left[kMaxNodes];              // s before each refusal at the current node
  int out[kMaxNodes];                  // tokens that were refused there
  double sum;
  int pick;
};

template <typename T, bool kProbs>
struct Walker {
  const VerifyParams& p;
  WalkShared& sh;
  int b, rank, ctas;
  Rate rate;

  __device__ const T* row_of(int j) const { return static_cast<const T*>(p.logits) + ((int64_t)b * p.Q + j) * p.row_stride; }
  __device__ const float* probs_of(int j) const { return p.probs + ((int64_t)b * p.Q + j) * p.probs_stride; }
  __device__ int chunks_of(int j) const { return (int)((p.V + lead_of(row_of(j)) + kChunk - 1) / kChunk); }

  // What is left of node j's probability of a token after `refused` refusals, times the node's sum of exponentials
  // without draft distributions (an order of magnitude that a draw does not need).
  __device__ float rest(int j, float w, int64_t at, float inv, int refused) const {
    if constexpr (kProbs) {
      float r = w * inv;
      if (refused > 0 && at >= 0 && at < p.V) {
        const float q = __ldg(probs_of(j) + at);
        for (int i = 0; i < refused; ++i) r = fmaxf(r - (float)sh.left[i] * q, 0.f);
      }
      return r;
    } else {
      for (int i = 0; i < refused; ++i) w = sh.out[i] == at ? 0.f : w;
      return w;
    }
  }

  // A chunk's rest by one warp, lane by lane; the sum in every lane.
  __device__ double chunk_rest(int j, int chunk, float m, float inv, int refused) const {
    constexpr int kN = Vec<T>::kN, kLoads = kChunk / (32 * kN);
    const int lane = threadIdx.x & 31;
    const T* row = row_of(j);
    const int64_t at = (int64_t)chunk * kChunk - lead_of(row);
    double sum = 0.;
    for (int i = 0; i < kLoads; ++i) {
      float x[kN], part = 0.f;
      const int64_t from = at + (i * 32 + lane) * kN;
      load_vec(row, from, p.V, x);
#pragma unroll
      for (int k = 0; k < kN; ++k) part += rest(j, weight(x[k], m, rate), from + k, inv, refused);
      sum += part;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
    return sum;
  }

  __device__ void everyone() const {
    __syncthreads();
    if (ctas > 1) cluster_sync_all();
  }

  // Sums of the chunks of what is left at node j, into chunk_sum; their sum, the same in every CTA.
  __device__ double sums(int j, int refused) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, chunks = chunks_of(j);
    double* to = p.chunk_sum + (int64_t)b * p.chunks;
    const float m = sh.top[j], inv = (float)(1. / sh.total[j]);
    if (kProbs && refused > 0) {
      for (int c = rank * kWalkWarps + warp; c < chunks; c += ctas * kWalkWarps) {
        const double s = chunk_rest(j, c, m, inv, refused);
        if (lane == 0) to[c] = s;
      }
    } else {
      // the chunks' sums, and again where a refused token lies
      const int64_t first = ((int64_t)b * p.Q + j) * p.chunks;
      const float scale = kProbs ? inv : 1.f;
      if (rank == 0) {
        for (int c = threadIdx.x; c < chunks; c += kWalkThreads) {
          const float2 ms = __ldcg(p.chunk_ms + first + c);
          to[c] = (double)(ms.y * weight(ms.x, m, rate)) * scale;
        }
        if (!kProbs) {
          __syncthreads();
          const int lead = lead_of(row_of(j));
          for (int i = warp; i < refused; i += kWalkWarps) {
            const int c = (sh.out[i] + lead) / kChunk;
            const double s = chunk_rest(j, c, m, inv, refused);     // (two refused tokens of a chunk: the same sum twice)
            if (lane == 0) to[c] = s;
          }
        }
      }
    }
    everyone();
    if (warp == 0) {
      double s = 0.;
      for (int c = lane; c < chunks; c += 32) s += __ldcg(to + c);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
      if (lane == 0) sh.sum = s;
    }
    __syncthreads();
    const double s = sh.sum;
    everyone();                          // nobody writes the sums again before all have read them
    return s;
  }

  // The first token whose running sum of what is left at node j exceeds `share` of it all: warp 0 of the first CTA.
  __device__ int draw(int j, double share, double total, int refused) {
    constexpr int kN = Vec<T>::kN, kLoads = kChunk / (32 * kN);
    const int lane = threadIdx.x & 31, chunks = chunks_of(j);
    const double* of = p.chunk_sum + (int64_t)b * p.chunks;
    const double want = share * total;
    double before = 0.;
    int chunk = -1, last = -1;
    double last_before = 0.;
    for (int c0 = 0; c0 < chunks && chunk < 0; c0 += 32) {
      const double mine = c0 + lane < chunks ? __ldcg(of + c0 + lane) : 0.;
      double incl = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const double o = __shfl_up_sync(kFull, incl, d);
        if (lane >= d) incl += o;
      }
      const unsigned some = __ballot_sync(kFull, mine > 0.), past = __ballot_sync(kFull, mine > 0. && before + incl > want);
      const int at = past != 0 ? __ffs(past) - 1 : (some != 0 ? 31 - __clz(some) : -1);
      if (at >= 0) {
        const double upto = __shfl_sync(kFull, incl - mine, at);
        last = c0 + at;
        last_before = before + upto;
        if (past != 0) chunk = last;
      }
      before += __shfl_sync(kFull, incl, 31);
    }
    chunk = last;                        // (none past it: the last that has anything)
    if (chunk < 0) return -1;
    const T* row = row_of(j);
    const int64_t at = (int64_t)chunk * kChunk - lead_of(row);
    const float m = sh.top[j], inv = (float)(1. / sh.total[j]);
    before = last_before;
    int found = -1;
    for (int i = 0; i < kLoads; ++i) {
      float x[kN];
      const int64_t from = at + (i * 32 + lane) * kN;
      load_vec(row, from, p.V, x);
      double part = 0.;
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        x[k] = rest(j, weight(x[k], m, rate), from + k, inv, refused);
        part += x[k];
      }
      double incl = part;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const double o = __shfl_up_sync(kFull, incl, d);
        if (lane >= d) incl += o;
      }
      // this lane's first token past `want`, else its last that has anything
      double run = before + incl - part;
      int mine = -1;
      bool past = false;
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        run += x[k];
        if (x[k] > 0.f && !past) {
          mine = (int)(from + k);
          past = run > want;
        }
      }
      const unsigned some = __ballot_sync(kFull, mine >= 0), hit = __ballot_sync(kFull, past);
      if (some != 0) found = __shfl_sync(kFull, mine, hit != 0 ? __ffs(hit) - 1 : 31 - __clz(some));
      if (hit != 0) break;
      before += __shfl_sync(kFull, incl, 31);
    }
    return found;
  }
};

template <typename T, bool kProbs>
__global__ void __launch_bounds__(kWalkThreads) walk_kernel(const VerifyParams p) {
  __shared__ WalkShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ctas = kProbs ? kWalkCtas : 1, b = blockIdx.x / ctas, rank = kProbs ? (int)cluster_ctarank() : 0;
  const int Q = p.Q;
  const Rate rate = rate_of(p, b);
  const bool greedy = rate.hi < 0.f;
  bool bad = false;
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
    sh.u[tid] = fmaxf(p.uniforms[r], 0.f);
    if (!(p.uniforms[r] == p.uniforms[r])) sh.u[tid] = __int_as_float(0x7f800000);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // nodes' largest logits and sums, a warp a node
  for (int j = warp; j < Q; j += kWalkWarps) {
    if (!is_node(p, (int64_t)b * Q + j)) continue;
    const int64_t first = ((int64_t)b * Q + j) * p.chunks;
    const T* row = static_cast<const T*>(p.logits) + ((int64_t)b * Q + j) * p.row_stride;
    const int chunks = (int)((p.V + lead_of(row) + kChunk - 1) / kChunk);
    float m = neg_inf();
    int where = INT_MAX;
    for (int c = lane; c < chunks; c += 32) {
      const float2 ms = __ldcg(p.chunk_ms + first + c);
      if (ms.x > m) {
        m = ms.x;
        where = __ldcg(p.chunk_at + first + c);
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const float om = __shfl_xor_sync(kFull, m, d);
      const int ow = __shfl_xor_sync(kFull, where, d);
      if (om > m || (om == m && ow < where)) {
        m = om;
        where = ow;
      }
    }
    double sum = 0.;
    if (!greedy)
      for (int c = lane; c < chunks; c += 32) {
        const float2 ms = __ldcg(p.chunk_ms + first + c);
        sum += ms.y * weight(ms.x, m, rate);
      }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
    if (lane == 0) {
      sh.top[j] = m;
      sh.total[j] = sum;
      sh.best[j] = m == neg_inf() ? -1 : where;
    }
  }
  __syncthreads();
  Walker<T, kProbs> w{p, sh, b, rank, ctas, rate};
  if (tid < Q && sh.parent[tid] >= 0) {
    const int up = sh.parent[tid], x = sh.token[tid];
    const float l = logit(w.row_of(up)[x]), m = sh.top[up];
    double have = 0.;
    if (!greedy && l != neg_inf()) have = (l == m ? 1. : exp2(((double)l - (double)m) * ((double)rate.hi + (double)rate.lo))) / sh.total[up];
    sh.have[tid] = have;
    sh.drawn[tid] = kProbs ? __ldg(w.probs_of(up) + x) : 1.f;
  }
  __syncthreads();

  // the walk, the same in every thread
  int at = 0, count = 0, refused = 0;
  double left = 1.;
  bool known = true;                     // left is that of what is left now
  for (int j = 1; j < Q; ++j) {
    if (sh.parent[j] != at) continue;
    bool yes;
    if (greedy) {
      yes = sh.best[at] == sh.token[j];
    } else {
      if constexpr (kProbs) {
        if (!known) {
          left = w.sums(at, refused);
          known = true;
        }
      }
      double r = sh.have[j];
      const double q = sh.drawn[j];
      for (int i = 0; i < refused; ++i) {
        if (kProbs) r = fmax(r - sh.left[i] * q, 0.);
        else if (sh.out[i] == sh.token[j]) r = 0.;
      }
      yes = (double)sh.u[j] * q * left < r;
      if (!yes) {
        __syncthreads();                 // (the lists below have been read)
        if (tid == 0) {
          sh.left[refused] = left;
          sh.out[refused] = sh.token[j];
        }
        __syncthreads();
        ++refused;
        if (kProbs) known = false;
        else left -= r;
      }
    }
    if (yes) {
      if (rank == 0 && tid == 0) {
        p.path[(int64_t)b * Q + count] = j;
        p.tokens[(int64_t)b * Q + count] = sh.token[j];
      }
      ++count;
      at = j;
      refused = 0;
      left = 1.;
      known = true;
    }
  }
  int next = greedy ? sh.best[at] : -1;
  if (!greedy && sh.top[at] != neg_inf()) {
    double total = w.sums(at, refused);
    if (!(total > 0.) && refused > 0) {  // nothing is left: from the target's own
      refused = 0;
      total = w.sums(at, 0);
    }
    if (warp == 0 && rank == 0) next = w.draw(at, (double)sh.u[0], total, refused);
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

template <typename T>
cudaError_t launch(const VerifyParams& p, cudaStream_t stream) {
  const int64_t warps = (int64_t)p.B * p.Q * p.chunks;
  stats_kernel<T><<<(unsigned)((warps + kStatsThreads / 32 - 1) / (kStatsThreads / 32)), kStatsThreads, 0, stream>>>(p);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  const bool probs = p.probs != nullptr;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * (probs ? kWalkCtas : 1)), 1, 1);
  cfg.blockDim = dim3(kWalkThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kWalkCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = probs ? 2 : 1;
  return probs ? cudaLaunchKernelEx(&cfg, walk_kernel<T, true>, p) : cudaLaunchKernelEx(&cfg, walk_kernel<T, false>, p);
}

}  // namespace

int verify_chunks(int64_t V) { return (int)((V + 7) / kChunk + 1); }

cudaError_t launch_spec_verify(const VerifyParams& p, int type, cudaStream_t stream) {
  if (type == NVFP4MLA_FP32) return launch<float>(p, stream);
  return type == NVFP4MLA_FP16 ? launch<__half>(p, stream) : launch<__nv_bfloat16>(p, stream);
}

}  // namespace nvfp4mla
