// kv8_decode_tree: attention of a tree of drafted tokens over the 8-bit per-head cache.
//
// What it computes. For one request and key/value head the columns (node, head of the group) share every key
// and value row. 128 of them are the rows of two products over a page of 64 tokens:
//   S[c, t] = q_c . K[t, :]            z = scale 2^(ek_t - 127) S        (ek, ev: scale bytes)
//   O[c, d] += sum_t w[c, t] V[t, d]   w = 2^(z log2e - m_c + ev_t - 127 - W_c)
// with running references m_c of the scores and W_c of the weights, whole numbers, so that raising one scales what
// has been summed by a power of two, exactly. The softmax's own sum l_c = sum_t 2^(z log2e - m_c) is made of the
// same exponentials: within a block of 16 tokens they differ from w by one power of two.
//
// What bounds it. A tree has some ten times the columns of a plain step: 16 nodes of 8 heads are 128, at which a
// token costs 2 D bytes and 512 D operations, near the ratio of the tensor cores' rate to the memory's. So:
//   S  8-bit products, as in kv8_decode: keys are used as they lie in the cache, and a query is a sum of E4M3
//      numbers (two of a bf16, three of an fp16, the row's largest element at 2^7 to 2^8): what is left after them is
//      half of E4M3's smallest step, 2^-10, 2^-17 of the largest. The parts are further steps along K: one sum.
//   O  fp16 products of weights in fp16 and codes, which an fp16 holds exactly. A column's largest is held above 2^8
//      and below 2^16, so half a step is 2^-11 of a weight just above a power of two (2^-12 just below one), and at
//      the lower end 2^-25 in those units: 2^-33 of the largest. (Weights as 8-bit parts, as kv8_decode has them, need
//      four for such a range: twice the tensor time, and some thirty instructions for a pair of weights where a conversion
//      is one. There the codes need no conversion instead, which is 2 D a token and does not grow with the columns.)
//
// One CTA per SM, persistent; the tiles (two pages, 128 tokens: one product's N) of all units (request, key/value head,
// 128 columns) form one sequence, cut into one contiguous range a CTA. Its warps:
//   0        producer: page numbers, then each tile's keys (TMA, swizzled), values (as they lie) and scale bytes
//   1        issues S = q K;  3: issues O += w V (two threads, so that neither waits for the other)
//   2        what the units' columns attend to, and their queries into L2, up to two units ahead
//   4-7      feeders: the unit's queries as parts, then each page's values as fp16
//   8-15     softmax: a warpgroup a page of each tile, a thread a column, so that maxima and sums need no exchange
//            but one between a column's two threads. S has three buffers, w lies in the place of its S, O is one
// A unit that several CTAs share leaves means and sums in the workspace, which join_kernel adds up.
//
// Measured, back to back, against 6.77 TB/s of measured copy bandwidth: 16 requests of 2,000 to 16,000 tokens, 32 nodes of
// 32 heads over 8 of 128: 94 us (45 % of it); one of 131,001 tokens, 16 nodes of 64 heads: 89 us (45 %); 24 requests of
// 900 to 9,000 tokens, 64 nodes of 32 heads over 4 of 64, a window of 4,096, fp16: 89 us; one request of 1,000 tokens:
// 17 us. A tile of 128 columns takes some 2,000 cycles, in which the tensor cores work for 1,100, and the softmax's chain
// (its scores' arrival, 64 exponentials a thread, the two threads' vote, the weights' store) is as long as the tile is;
// so is the feeders'. A unit costs some 11,000 more: its queries, its first and masked tiles, its results. What was tried
// and not kept, in the order of the first three: a stream of tiles, and an O, for each warpgroup (112, 99, 100 us); keys
// and values in rings of their own (92, 86, 113); queries fetched a tile ahead (100, 93, 92); the blocks of a page unrolled
// instead of two at a time (97, 91, 95: the code of all warps together counts).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cstddef>
#include <mutex>

#include "../../include/nvfp4mla.h"
#include "kv8.h"
#include "kv8_units.cuh"
#include "ptx.cuh"

namespace nvfp4mla {
namespace {

using namespace ptx;

constexpr int kCols = 128;             // of a unit: (node, head)
constexpr int kTile = 2 * kPageTokens; // tokens of a stage: two pages, which one product with the queries takes
constexpr int kHalves = 2;
constexpr int kBufs = 3;               // tiles whose scores, or weights in their place, tensor memory holds
constexpr int kTreeThreads = 512;
constexpr int kFeeders = 128;          // threads
constexpr int kSoftmaxThreads = 256;
constexpr int kUnitCost = 4;           // of a unit, in tiles
constexpr int kMinTiles = 2;           // of a CTA, on average
constexpr float kWeightScale = 9.f;    // log2: a weight at its reference is held as 2^9
constexpr float kMostWeights = 64512.f;   // of 16 weights together, so that an fp16 holds each (65,504)
constexpr float kSumHeadroom = 60.f;   // log2: how far above its reference a score may come, for the sum's sake
constexpr unsigned kFull = 0xFFFFFFFFu;
enum { kBarFeeders = 1, kBarSoftmax = 2, kBarQuarter = 3 };   // (one for each quarter of the columns)

template <int D, int kQ>
struct Shape {
  static constexpr int kQImage = kCols * D;                     // bytes of a part
  static constexpr int kQBytes = kQ * kQImage;
  static constexpr int kCodes = kPageTokens * D;                // bytes of a page's keys, or values
  static constexpr int kStageBytes = 2 * kHalves * kCodes;      // keys of both pages, then values
  static constexpr int kVBytes = 2 * kCodes;                    // a page's values as fp16
  static constexpr int kVBufs = 2 * kHalves;                    // of two tiles
  static constexpr int kControl = 13312;
  static constexpr int kFit = (232448 - 1024 - kControl - kQBytes - kVBufs * kVBytes) / kStageBytes;
  static constexpr int kStages = kFit < 16 ? kFit : 16;
  static constexpr uint32_t kSw = D == 128 ? SW_128B : SW_64B;  // of rows of D bytes
  static constexpr int kOCol = kBufs * kTile;                   // TMEM columns: buffers of S, then O
  static constexpr uint32_t kTmem = 512;
  static_assert(kOCol + D <= 512 && kStages >= 3, "fits");
};

template <int kStages>
struct Control {
  uint64_t full[kStages], empty[kStages];
  uint64_t q_full[2], q_empty, done[2];                // done: softmax has ended a segment
  uint64_t s_full[kBufs], w_full[kBufs], v_full[2];
  uint64_t o_done[kBufs];                              // the product is complete: weights and values are used, O is at rest
  uint64_t drain[2];
  alignas(16) uint4 scales[kStages][kHalves];          // the scale bytes of two neighbouring heads
  int pages_ok[kStages];                               // bit per page: it is one
  alignas(16) float f[2][kCols];                       // per segment parity: score of a column per unit of S, log2 units
  uint64_t mask[2][kCols];
  int lo[2][kCols];                                    // first position before the tree that a column attends to
  int row[2][kCols];                                   // of out and lse, -1: no column
  uint64_t any_mask[2], all_mask[2];                   // nodes that some, and that all of the tree attend to
  int any_lo[2], all_lo[2];
  uint32_t poison[2][kCols][4];                        // dims that a NaN value reaches
  int any_poison[2];
  alignas(8) float2 most[kHalves][kCols];              // of a half: the largest score, and weight
  float l[kHalves][kCols];                             // at a segment's end: the sum of a half's weights
  int scan_sum[kTreeThreads / 32];
  int start_before, start_b;
  int abort;
  uint32_t tmem_base;
};

// What join_kernel is to add up, by the CTA that has a shared unit's first pages.
struct Shared {
  int last;                            // CTA, -1: none
  int slot;                            // of its own part: 0 or 1
  int b, kvh, ct;
};

template <bool kHalf>
__device__ __forceinline__ float2 widen2(uint32_t w) {
  if constexpr (kHalf) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <bool kHalf>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
  if constexpr (kHalf) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Four E4M3 codes -> two pairs of fp16.
__device__ __forceinline__ uint2 codes4(uint32_t w) {
  uint2 r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(w));
  return r;
}
// A pair of fp16 as kParts pairs of E4M3 numbers whose sum it is, but for the last one's rounding. Magnitudes below 256: what
// a part leaves an fp16 holds exactly.
template <int kParts>
__device__ __forceinline__ void split(uint32_t h, uint32_t (&part)[kParts]) {
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    part[i] = f16x2_to_e4m3x2(h);
    const uint32_t held = e4m3x2_to_f16x2(part[i]);
    const __half2 left = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&held));
    h = *reinterpret_cast<const uint32_t*>(&left);
  }
}
// bits lo .. hi - 1 of 64, none if there are none
__device__ __forceinline__ uint64_t bits(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 64);
  return lo >= hi ? 0ull : (hi - lo == 64 ? ~0ull : ((1ull << (hi - lo)) - 1) << lo);
}
// a tree's nodes, the first of which is position `base`, among the 64 positions from t0 on
__device__ __forceinline__ uint64_t nodes_at(uint64_t mask, int base, int t0) {
  const int d = base - t0;
  return d >= 64 || d <= -64 ? 0ull : (d >= 0 ? mask << d : mask >> -d);
}
__device__ __forceinline__ int second_slot(int begin, int pos) { return pos < begin ? 0 : 1; }
__device__ __forceinline__ float inverse(float sum) { return sum == 0.f ? 0.f : rcp_approx(sum); }

template <int D, int kQ>
struct Cta {
  using S = Shape<D, kQ>;
  using Ctl = Control<S::kStages>;
  using Walk = ::nvfp4mla::Walk<kTile, kUnitCost>;
  const Kv8TreeParams& p;
  uint8_t* stages;
  uint8_t* qimg;
  uint8_t* vimg;
  Ctl* ctl;

  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    return wait_long(ctl, p.status, bar, parity);
  }
  static __device__ __noinline__ bool wait_long(Ctl* ctl, int32_t* status, uint64_t* bar, uint32_t parity) {
    if (mbar_wait(bar, parity, &ctl->abort, kWaitTimeoutNs)) return true;
    if (atomicExch(&ctl->abort, 1) == 0 && status != nullptr) atomicAdd(status + NVFP4MLA_STAT_TIMEOUT, 1);
    return false;
  }
  __device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) { return __all_sync(kFull, wait(bar, parity)); }

  // Counts up to n and round again, with the phase that goes with it.
  template <int n>
  struct Ring {
    uint32_t st = 0, phase = 0;
    __device__ __forceinline__ void next() {
      if (++st == (uint32_t)n) {
        st = 0;
        phase ^= 1;
      }
    }
  };
  // ---------------------------------------------------------------- producer (warp 0)
  // Page numbers of 16 tiles from i on, a lane a page. -1: not needed, or none.
  __device__ __forceinline__ int load_pages(const Walk& w, int i) {
    const int lane = threadIdx.x & 31;
    if (i + lane / kHalves >= w.count) return -1;
    const int64_t col = kHalves * ((int64_t)w.first + w.at + i) + lane;
    if (col * kPageTokens >= w.len || col >= p.max_pages) return -1;   // behind the table: counted together
    const int page = p.page_table[(int64_t)w.b * p.max_pages + col];
    if (page >= 0 && page < p.num_pages) return page;
    if (w.ct == 0 && w.kvh == 0 && p.status != nullptr) atomicAdd(p.status + NVFP4MLA_STAT_BAD_PAGE, 1);
    return -1;
  }

  __device__ void producer(Walk w) {
    const int lane = threadIdx.x & 31;
    if (p.withhold) return;
    Ring<S::kStages> ring;
    uint32_t g = 0;
    int pages = w.left > 0 ? load_pages(w, 0) : -1;
    bool ok = true;
    while (ok && w.left > 0) {
      const int kvh = w.kvh;
      if (w.kvh == 0 && w.ct == 0 && w.at + w.count == w.n && lane == 0 && p.status != nullptr) {
        const int64_t need = ((int64_t)w.len + kPageTokens - 1) / kPageTokens;
        const int64_t from = max((int64_t)kHalves * w.first, p.max_pages);
        if (need > from) atomicAdd(p.status + NVFP4MLA_STAT_BAD_PAGE, (int)(need - from));
      }
      for (int i = 0; ok && i < w.count; i += 16) {
        const int mine = pages;
        if (i + 16 < w.count) {
          pages = load_pages(w, i + 16);
        } else {
          Walk nx = w;
          nx.next(p);
          pages = nx.left > 0 ? load_pages(nx, 0) : -1;
        }
        const int m = min(16, w.count - i);
        for (int k = 0; ok && k < m; ++k) {
          const int page = __shfl_sync(kFull, mine, kHalves * k + (lane & 1));
          const uint32_t have = __ballot_sync(kFull, page >= 0) & 3u;
          if (lane == 0) {
            ok = wait(&ctl->empty[ring.st], ring.phase ^ 1);
            if (ok) {
              ctl->pages_ok[ring.st] = (int)have;
              mbar_arrive_expect_tx(&ctl->full[ring.st], __popc(have) * 2 * S::kCodes);
            }
          }
          ok = __shfl_sync(kFull, ok ? 1 : 0, 0) != 0;
          if (ok && lane < kHalves) {
            if (page >= 0) {
              uint8_t* to = stages + ring.st * S::kStageBytes + lane * S::kCodes;
              const uint8_t* at = p.cache + page * p.page_bytes;
              tma_load_3d(to, &p.cache_map, 0, kvh * kPageTokens, page, &ctl->full[ring.st]);
              bulk_g2s(to + kHalves * S::kCodes, at + kv8_codes_off(p.kv_heads, D, 1, kvh), S::kCodes, &ctl->full[ring.st]);
              cp_async_16(&ctl->scales[ring.st][lane], at + kv8_scales_off(p.kv_heads, D, kvh & ~1));
            }
            cp_async_arrive(&ctl->full[ring.st]);
          }
          __syncwarp();
          if (ok) {
            ring.next();
            ++g;
          }
        }
      }
      if (ok) w.next(p);
    }
    if (lane == 0 && (!ok || *reinterpret_cast<volatile int*>(&ctl->abort) != 0)) {
      // a wait gave up: the copies that are still in flight land (bounded)
      const uint32_t n = min(g, (uint32_t)S::kStages);
      for (uint32_t i = 0; i < n; ++i) {
        const uint32_t t = g - 1 - i;
        mbar_wait(&ctl->full[t % S::kStages], (t / S::kStages) & 1, nullptr, kWaitTimeoutNs);
      }
    }
    __syncwarp();
  }

  // ---------------------------------------------------------------- what a unit's columns attend to (warp 2)
  __device__ __forceinline__ int node_of(int col) const { return (int)(((uint64_t)(uint32_t)col * p.group_inverse) >> 24); }   // col / group
  // Ahead of the others, by up to two units, as it waits for memory alone.
  __device__ void columns(Walk w) {
    const int lane = threadIdx.x & 31, ncols = p.Q * p.group;
    const uint64_t bits_of = p.Q == 64 ? ~0ull : (1ull << p.Q) - 1;
    for (uint32_t seg = 0; w.left > 0; ++seg, w.next(p)) {
      const uint32_t buf = seg & 1;
      if (!wait_warp(&ctl->done[buf], ((seg >> 1) & 1) ^ 1)) return;     // the unit before the last is written
      const int base = w.len - p.Q;
      const uint64_t* masks = p.masks + (int64_t)w.b * p.Q;
      uint64_t some = 0, all = ~0ull;
      int first = INT_MAX, last = 0;
#pragma unroll 1
      for (int j = lane; j < p.Q; j += 32) {
        const uint64_t mask = __ldg(masks + j);
        if (mask == 0) continue;
        some |= mask & bits_of;
        all &= mask & bits_of;
        const int lo = p.window > 0 ? max(0, base + max(1, __popcll(mask & bits_of)) - p.window) : 0;
        first = min(first, lo);
        last = max(last, lo);
      }
      const uint32_t some0 = __reduce_or_sync(kFull, (uint32_t)some), some1 = __reduce_or_sync(kFull, (uint32_t)(some >> 32));
      const uint32_t all0 = __reduce_and_sync(kFull, (uint32_t)all), all1 = __reduce_and_sync(kFull, (uint32_t)(all >> 32));
      first = __reduce_min_sync(kFull, first);
      last = __reduce_max_sync(kFull, last);
      if (lane == 0) {
        ctl->any_mask[buf] = (uint64_t)some1 << 32 | some0;
        ctl->all_mask[buf] = ((uint64_t)all1 << 32 | all0) & bits_of;
        ctl->any_lo[buf] = first;
        ctl->all_lo[buf] = last;
      }
#pragma unroll 1
      for (int c = lane; c < kCols; c += 32) {
        const int col = w.ct * kCols + c, j = node_of(col);
        const uint64_t mask = col < ncols ? __ldg(masks + j) : 0;
        const int place = base + max(1, __popcll(mask & bits_of)) - 1;
        ctl->mask[buf][c] = mask & bits_of;
        ctl->lo[buf][c] = mask == 0 ? INT_MAX : (p.window > 0 ? max(0, place - p.window + 1) : 0);
        // (the next unit's queries come from memory while this one's tiles are at work)
        if (col < ncols)
          for (int k = 0; k < D * 2; k += 128) prefetch_l2(reinterpret_cast<const uint8_t*>(p.q + ((int64_t)w.b * p.Q + j) * p.q_token_stride + (w.kvh * p.group + col - j * p.group) * p.q_head_stride) + k);
        ctl->row[buf][c] = col < ncols ? (w.b * p.Q + j) * p.H + w.kvh * p.group + (col - j * p.group) : -1;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->q_full[buf]);
    }
  }

  // ---------------------------------------------------------------- S = q K (warp 1, one thread)
  __device__ void issue_s(Walk w, uint32_t tmem) {
    constexpr uint32_t kId = idesc_e4m3(kCols, kTile, false, false);
    const uint64_t kd = sdesc(smem_u32(stages), 16, 8 * D, S::kSw), qd = sdesc(smem_u32(qimg), 16, 8 * D, S::kSw);
    Ring<S::kStages> ring;
    Ring<kBufs> buf;
    bool ok = true;
    for (uint32_t seg = 0; ok && w.left > 0; ++seg, w.next(p)) {
      ok = wait(&ctl->q_full[seg & 1], (seg >> 1) & 1);
      for (int i = 0; ok && i < w.count; ++i) {
        ok = wait(&ctl->full[ring.st], ring.phase);
        ok = ok && wait(&ctl->o_done[buf.st], buf.phase ^ 1);            // the buffer's last weights have been used
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + buf.st * kTile, k_lo = (uint32_t)kd + ((ring.st * S::kStageBytes) >> 4);
#pragma unroll
        for (int part = 0; part < kQ; ++part)
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            const uint32_t q_lo = (uint32_t)qd + ((part * S::kQImage) >> 4) + 2 * k;
            if (part == 0 && k == 0) umma_f8_ss_w<0>(d, q_lo, (uint32_t)(qd >> 32), k_lo + 2 * k, (uint32_t)(kd >> 32), kId);
            else umma_f8_ss_w<1>(d, q_lo, (uint32_t)(qd >> 32), k_lo + 2 * k, (uint32_t)(kd >> 32), kId);
          }
        umma_commit(&ctl->s_full[buf.st]);               // (the stage is given back by the softmax, which waits for this)
        ring.next();
        buf.next();
      }
      if (ok) umma_commit(&ctl->q_empty);
    }
    umma_commit(&ctl->drain[0]);
    mbar_wait(&ctl->drain[0], 0, nullptr, kWaitTimeoutNs);
  }

  // ---------------------------------------------------------------- O += w V (warp 3, one thread)
  __device__ void issue_o(Walk w, uint32_t tmem) {
    constexpr uint32_t kId = idesc_f16(kCols, D, false, true, false);
    const uint64_t vd = sdesc(smem_u32(vimg), kPageTokens * 128, 1024, SW_128B);
    Ring<kBufs> buf;
    Ring<2> vbuf;
    bool ok = true;
    for (; ok && w.left > 0; w.next(p)) {
      for (int i = 0; ok && i < w.count; ++i) {
        ok = wait(&ctl->v_full[vbuf.st], vbuf.phase);
        ok = ok && wait(&ctl->w_full[buf.st], buf.phase);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + S::kOCol, a = tmem + buf.st * kTile, v_lo = (uint32_t)vd + ((vbuf.st * kHalves * S::kVBytes) >> 4);
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k) {
          // (a page's weights lie in the first half of its scores' place)
          const uint32_t a_k = a + (k / 4) * kPageTokens + (k % 4) * 8, v_k = v_lo + (k / 4) * (S::kVBytes >> 4) + (k % 4) * 128;
          if (k == 0) umma_ts_w<-1>(d, a_k, v_k, (uint32_t)(vd >> 32), kId, i > 0 ? 1u : 0u);
          else umma_ts_w<1>(d, a_k, v_k, (uint32_t)(vd >> 32), kId);
        }
        umma_commit(&ctl->o_done[buf.st]);
        buf.next();
        vbuf.next();
      }
    }
    umma_commit(&ctl->drain[1]);
    mbar_wait(&ctl->drain[1], 0, nullptr, kWaitTimeoutNs);
  }

  // ---------------------------------------------------------------- feeders (warps 4-7)
  static constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kRounds = 32 / kAtOnce;    // of a row; rows of a load; loads of a lane
  // The unit's queries, on their way: a warp has 32 rows, a load's of every fourth, so that few rows are shared by all warps.
  __device__ __forceinline__ void fetch(const Walk& w, uint4 (&v)[kRounds]) {
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
    // a lane a column: where its row is
    const int col = w.ct * kCols + (lane / kAtOnce * 4 + warp) * kAtOnce + lane % kAtOnce, j = node_of(col);
    const int64_t mine = col < p.Q * p.group ? ((int64_t)w.b * p.Q + j) * p.q_token_stride + (w.kvh * p.group + col - j * p.group) * p.q_head_stride : -1;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int64_t at = __shfl_sync(kFull, mine, r * kAtOnce + lane / kLanes);
      v[r] = make_uint4(0u, 0u, 0u, 0u);
      if (at >= 0) v[r] = *reinterpret_cast<const uint4*>(p.q + at + (lane % kLanes) * 8);
    }
  }
  // And as parts.
  template <bool kHalf>
  __device__ __forceinline__ void queries(uint4 (&v)[kRounds], uint32_t buf, int rows) {
    constexpr int kTogether = 4;         // loads whose chains are under way together
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, sub = lane / kLanes, ch = lane % kLanes;
#pragma unroll 1
    for (int r0 = 0; r0 < kRounds; r0 += kTogether) {
      if (r0 * 4 * kAtOnce >= rows) {
        // no column: zeros, so that nothing rare comes of them
#pragma unroll 1
        for (int n = (r0 * 4 + warp) * kAtOnce + sub; n < kCols; n += 4 * kAtOnce) {
#pragma unroll
          for (int q = 0; q < kQ; ++q) *reinterpret_cast<uint2*>(qimg + q * S::kQImage + n * D + ch * 8) = make_uint2(0u, 0u);
          if (ch == 0) ctl->f[buf][n] = 0.f;
        }
        break;
      }
      uint4 x[kTogether];
      uint32_t top[kTogether / 2];       // of two rows
#pragma unroll
      for (int i = 0; i < kTogether; ++i) x[i] = v[i];
#pragma unroll
      for (int i = 0; i + kTogether < kRounds; ++i) v[i] = v[i + kTogether];
#pragma unroll
      for (int i = 0; i < kTogether; i += 2) {
        auto most = [&](const uint4& y) { return __vmaxu2(__vmaxu2(y.x & 0x7FFF7FFFu, y.y & 0x7FFF7FFFu), __vmaxu2(y.z & 0x7FFF7FFFu, y.w & 0x7FFF7FFFu)); };
        const uint32_t a = most(x[i]), b = most(x[i + 1]);
        top[i / 2] = __vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
      }
#pragma unroll
      for (int d = 1; d < kLanes; d <<= 1)
#pragma unroll
        for (int i = 0; i < kTogether / 2; ++i) top[i] = __vmaxu2(top[i], __shfl_xor_sync(kFull, top[i], d));
#pragma unroll
      for (int i = 0; i < kTogether; ++i) {
        const int n = ((r0 + i) * 4 + warp) * kAtOnce + sub;
        const uint32_t ws[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, most = (top[i / 2] >> (16 * (i & 1))) & 0xFFFFu;
        const bool finite = most < (kHalf ? 0x7C00u : 0x7F80u);
        // the largest magnitude goes to [128, 256): a power of two, exact
        const int e = (int)(__float_as_uint(widen2<kHalf>(most).x) >> 23) - 127;
        const int sh = most == 0 || !finite ? 0 : min(7 - e, 126);
        const float mul = __uint_as_float((uint32_t)(sh + 127) << 23);
        uint32_t part[4][kQ];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // (fp16 is off by 2^-25 at most, where the parts' last is off by 2^-10; a row with an infinity or a NaN has f)
          const float2 y = __fmul2_rn(widen2<kHalf>(ws[k]), make_float2(mul, mul));
          split(narrow2<true>(y.x, y.y), part[k]);
        }
        const int chunk = D == 128 ? ((ch >> 1) ^ (n & 7)) : ((ch >> 1) ^ ((n >> 1) & 3));
#pragma unroll
        for (int q = 0; q < kQ; ++q)
          *reinterpret_cast<uint2*>(qimg + q * S::kQImage + n * D + chunk * 16 + (ch & 1) * 8) =
              make_uint2(part[0][q] | (part[1][q] << 16), part[2][q] | (part[3][q] << 16));
        if (ch == 0) ctl->f[buf][n] = finite ? p.scale_log2 * __uint_as_float((uint32_t)(127 - sh) << 23) : __int_as_float(0x7fc00000);
      }
    }
  }

  // 16 codes of token t (row r of its page), dims 16 c .. 16 c + 15, as fp16 into the image.
  __device__ __forceinline__ void put_values(uint8_t* img, const uint4& x, int r, int c) {
    const uint2 a = codes4(x.x), b = codes4(x.y), d = codes4(x.z), e = codes4(x.w);
    const uint4 first = make_uint4(a.x, a.y, b.x, b.y), second = make_uint4(d.x, d.y, e.x, e.y);
    uint8_t* row = img + (c >> 2) * (kPageTokens * 128) + r * 128;
    const int at = (c & 3) * 2, swap = (c >> 2) & 1;           // (the halves of 64 dims in turn, for the banks' sake)
    *reinterpret_cast<uint4*>(row + (((at + swap) ^ (r & 7)) << 4)) = swap ? second : first;
    *reinterpret_cast<uint4*>(row + (((at + 1 - swap) ^ (r & 7)) << 4)) = swap ? first : second;
  }

  // Values of a row that only some columns attend to: a NaN is taken out and noted for those. (A row that none attends
  // to may hold anything, and becomes zeros.)
  static __device__ __forceinline__ bool nans_in(const uint4& x) {
    return (__vcmpeq4(x.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(x.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu) |
            __vcmpeq4(x.z & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(x.w & 0x7F7F7F7Fu, 0x7F7F7F7Fu)) != 0;
  }
  __device__ __noinline__ uint4 without_nans(uint4 x, int t, int c, uint32_t buf, int base) {
    uint8_t* byte = reinterpret_cast<uint8_t*>(&x);
#pragma unroll 1
    for (int k = 0; k < 16; ++k) {
      if ((byte[k] & 0x7F) != 0x7F) continue;
      byte[k] = 0;
      const int d = c * 16 + k;
#pragma unroll 1
      for (int n = 0; n < kCols; ++n) {
        const bool attends = t < base ? t >= ctl->lo[buf][n] : ((ctl->mask[buf][n] >> (t - base)) & 1) != 0;
        if (attends) atomicOr(&ctl->poison[buf][n][d >> 5], 1u << (d & 31));
      }
      ctl->any_poison[buf] = 1;
    }
    return x;
  }

  template <bool kHalf>
  __device__ void feed(Walk w) {
    constexpr int kChunks = D / 16, kLoads = kPageTokens * kChunks / kFeeders;
    const int tid = threadIdx.x & 127, lane = threadIdx.x & 31;
    Ring<S::kStages> ring;
    Ring<kBufs> used;                    // the tile before the last: its values' buffers are this one's
    Ring<2> vbuf;
    uint32_t t = 0;
    bool ok = true;
    for (uint32_t seg = 0; w.left > 0; ++seg, w.next(p)) {
      const uint32_t buf = seg & 1;
      uint4 q[kRounds];
      fetch(w, q);
      ok = ok && wait_warp(&ctl->q_empty, (seg & 1) ^ 1);              // the products with the last unit's queries are complete
      ok = ok && wait_warp(&ctl->done[buf], ((seg >> 1) & 1) ^ 1);     // and the unit's before that is written
      if (ok) {
        queries<kHalf>(q, buf, p.Q * p.group - w.ct * kCols);
        fence_proxy_async_smem();
      }
      if (bar_any(kBarFeeders, kFeeders, !ok)) return;
      if (lane == 0) mbar_arrive(&ctl->q_full[buf]);
      ok = wait_warp(&ctl->q_full[buf], (seg >> 1) & 1);                 // what the columns attend to
      const int base = w.len - p.Q, all_lo = ctl->all_lo[buf], any_lo = ctl->any_lo[buf];
      for (int i = 0; ok && i < w.count; ++i, ++t) {
        ok = wait_warp(&ctl->full[ring.st], ring.phase);
        if (t >= 2) ok = ok && wait_warp(&ctl->o_done[used.st], used.phase);
        if (!ok) break;
#pragma unroll 1
        for (int half = 0; half < kHalves; ++half) {
          const int t0 = (w.first + w.at + i) * kTile + half * kPageTokens;
          const uint8_t* from = stages + ring.st * S::kStageBytes + (kHalves + half) * S::kCodes;
          uint8_t* img = vimg + (vbuf.st * kHalves + half) * S::kVBytes;
          const bool page_ok = ((ctl->pages_ok[ring.st] >> half) & 1) != 0;
          if (page_ok && t0 >= all_lo && t0 + kPageTokens <= base) {
#pragma unroll 1
            for (int k0 = 0; k0 < kLoads; k0 += 2) {
              uint4 x[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) x[k] = *reinterpret_cast<const uint4*>(from + (tid + (k0 + k) * kFeeders) * 16);
#pragma unroll
              for (int k = 0; k < 2; ++k) put_values(img, x[k], (tid + (k0 + k) * kFeeders) / kChunks, (tid + (k0 + k) * kFeeders) % kChunks);
            }
          } else {
            const uint64_t any = page_ok ? bits(any_lo - t0, base - t0) | nodes_at(ctl->any_mask[buf], base, t0) : 0;
            const uint64_t all = page_ok ? bits(all_lo - t0, base - t0) | nodes_at(ctl->all_mask[buf], base, t0) : 0;
#pragma unroll 1
            for (int k = 0; k < kLoads; ++k) {
              const int r = (tid + k * kFeeders) / kChunks, c = (tid + k * kFeeders) % kChunks;
              uint4 y = make_uint4(0u, 0u, 0u, 0u);
              if ((any >> r) & 1) {
                y = *reinterpret_cast<const uint4*>(from + (tid + k * kFeeders) * 16);
                if (((all >> r) & 1) == 0 && nans_in(y)) y = without_nans(y, t0 + r, c, buf, base);
              }
              put_values(img, y, r, c);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ctl->v_full[vbuf.st]);
          mbar_arrive(&ctl->empty[ring.st]);
        }
        ring.next();
        vbuf.next();
        if (t >= 2) used.next();
      }
    }
  }

  // ---------------------------------------------------------------- softmax (warps 8-15)
  // References of a column's scores, and of its weights from there, and the sum that this thread has against the former.
  struct Refs {
    float m, w, l;
    __device__ __forceinline__ bool none() const { return w == kNone; }
  };
  // The first references of columns that have none, from a tile whose pages all columns attend to.
  __device__ __forceinline__ void start(Refs& refs, int half, uint32_t s_at, float f, uint2 sc) {
    const int warp = (threadIdx.x >> 5) & 3, r = threadIdx.x & 127;
    float mz = neg_inf(), mw = neg_inf();
#pragma unroll 1
    for (int b = 0; b < 4; ++b) {
      uint32_t s[16];
      tmem_ld16(s_at + 16 * b, s);
      tmem_wait_ld();
      float x = neg_inf();
#pragma unroll
      for (int k = 0; k < 16; k += 2) x = max3(x, __uint_as_float(s[k]), __uint_as_float(s[k + 1]));
      const float z = x == neg_inf() ? x : x * (f * __uint_as_float(((sc.x >> (8 * b)) & 0xFFu) << 23));
      mz = fmaxf(mz, z);
      mw = fmaxf(mw, z + (float)((int)((sc.y >> (8 * b)) & 0xFFu) - 127));
    }
    ctl->most[half][r] = make_float2(mz, mw);
    bar_sync(kBarQuarter + warp, 64);
    const float2 other = ctl->most[half ^ 1][r];
    const float top = fmaxf(mz, other.x);
    if (refs.none() && fabsf(top) < 1048576.f) {       // (none to speak of, or one beside which a scale would be rounded away: careful())
      refs.m = ceilf(top);
      refs.w = ceilf(fmaxf(mw, other.y)) - refs.m;
    }
    bar_sync(kBarQuarter + warp, 64);
  }

  // The scores of positions that a column does not attend to become -inf, and the scale bytes of a block that has no other,
  // which may be anything, those of 1. (Loops: code that runs a few times costs what its fetching costs.)
  static __device__ __noinline__ uint2 leave_out(uint32_t s_at, uint64_t mine, uint2 sc) {
#pragma unroll 1
    for (int b = 0; b < 4; ++b) {
      __syncwarp();
      uint32_t s[16];
      tmem_ld16(s_at + 16 * b, s);
      tmem_wait_ld();
      const uint32_t in = (uint32_t)(mine >> (16 * b)) & 0xFFFFu;
#pragma unroll
      for (int k = 0; k < 16; ++k) s[k] = (in >> k) & 1 ? s[k] : 0xFF800000u;
      tmem_st16(s_at + 16 * b, s);
      const uint32_t at = in == 0 ? 0xFFu << (8 * b) : 0u;
      sc.x = (sc.x & ~at) | (0x7F7F7F7Fu & at);
      sc.y = (sc.y & ~at) | (0x7F7F7F7Fu & at);
    }
    tmem_wait_st();
    return sc;
  }

  // A page's weights in the place of its scores, with whatever is rarer: new references, and scores or scales so
  // wide that sum and weights need an exponential each. Both halves' threads of a quarter of the columns come here together.
  // (at_rest: the barrier of the product before, or null; false: a wait gave up.)
  __device__ __noinline__ bool careful(Refs& refs, int half, uint32_t s_at, float f, uint2 sc, uint64_t mine, uint64_t* at_rest, uint32_t parity, uint32_t o_at) {
    Refs t = refs;
    const int warp = (threadIdx.x >> 5) & 3, r = threadIdx.x & 127;
    float z[4] = {}, mz = neg_inf();
    auto key_scale = [&](int b) { return f * __uint_as_float(((sc.x >> (8 * b)) & 0xFFu) << 23); };
    auto value_scale = [&](int b) { return (float)((int)((sc.y >> (8 * b)) & 0xFFu) - 127); };
    auto largest = [&](float m) {          // of the weights, against m
      float w = neg_inf();
#pragma unroll
      for (int b = 0; b < 4; ++b) w = fmaxf(w, (z[b] - m) + value_scale(b));
      return w;
    };
    // (kept as loops: code that runs a few times costs what its fetching costs)
#pragma unroll 1
    for (int b = 0; b < 4; ++b) {
      uint32_t s[16];
      tmem_ld16(s_at + 16 * b, s);
      tmem_wait_ld();
      const uint32_t in = (uint32_t)(mine >> (16 * b));
      float x = neg_inf();
#pragma unroll
      for (int k = 0; k < 16; ++k) x = fmaxf(x, (in >> k) & 1 ? __uint_as_float(s[k]) : neg_inf());
      x = x == neg_inf() ? x : x * key_scale(b);
      z[0] = b == 0 ? x : z[0];
      z[1] = b == 1 ? x : z[1];
      z[2] = b == 2 ? x : z[2];
      z[3] = b == 3 ? x : z[3];
      mz = fmaxf(mz, x);
    }
    ctl->most[half][r] = make_float2(mz, largest(t.m));
    bar_sync(kBarQuarter + warp, 64);
    const float2 other = ctl->most[half ^ 1][r];
    const float mz2 = fmaxf(mz, other.x), mw2 = fmaxf(largest(t.m), other.y);
    // (16 weights at the reference are 2^(9 + 4); the tile's own are at most 2^2 above it)
    const bool raise = t.none() ? mz2 > neg_inf() : mw2 > t.w + 2.f || mz2 > t.m + kSumHeadroom;
    float scale_o = 1.f;
    if (bar_any(kBarQuarter + warp, 64, raise)) {
      const float m1 = !raise ? t.m : (t.none() ? ceilf(mz2) : fmaxf(t.m, ceilf(mz2)));
      ctl->most[half][r].y = largest(m1);
      bar_sync(kBarQuarter + warp, 64);
      if (raise) {
        float w1 = ceilf(fmaxf(largest(m1), ctl->most[half ^ 1][r].y));
        if (!t.none()) {
          w1 = fmaxf(w1, t.w + (t.m - m1));
          scale_o = ex2_approx((t.m - m1) + (t.w - w1));
          t.l *= ratio(t.m, m1);
        }
        t.m = m1;
        t.w = w1;
      }
      if (at_rest != nullptr && __any_sync(kFull, scale_o != 1.f)) {
        if (!wait_warp(at_rest, parity)) return false;
        tc_fence_after();
#pragma unroll 1
        for (int k = half * (D / 2); k < (half + 1) * (D / 2); k += 32) {
          uint32_t o[32];
          tmem_ld32(o_at + k, o);
          tmem_wait_ld();
#pragma unroll
          for (int n = 0; n < 32; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * scale_o);
          tmem_st32(o_at + k, o);
        }
      }
    }
#pragma unroll 1
    for (int b = 0; b < 4; ++b) {
      uint32_t s[16], out[8];
      tmem_ld16(s_at + 16 * b, s);
      tmem_wait_ld();
      const uint32_t in = (uint32_t)(mine >> (16 * b));
      const float c = key_scale(b), less = value_scale(b) - t.w + kWeightScale;
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        float e[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float d = __fadd_rn(__fmul_rn(__uint_as_float(s[k + n]), c), -t.m);
          const bool is_in = ((in >> (k + n)) & 1) != 0;
          sum[n] += is_in ? ex2_approx(d) : 0.f;
          e[n] = is_in ? ex2_approx(d + less) : 0.f;
        }
        out[k / 2] = narrow2<true>(e[0], e[1]);
      }
      t.l += sum[0] + sum[1];
      tmem_st8(s_at + 8 * b, out);       // (in the place of scores that have been read)
    }
    refs = t;
    return true;
  }

  // A warpgroup a page of each tile. The two threads of a column have the same references, and agree on every tile whether
  // those will do.
  template <bool kHalf>
  __device__ void softmax(Walk w, uint32_t tmem, const Ranges& ranges, Shared* shared) {
    const int half = (threadIdx.x >> 7) - 2, warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, r = threadIdx.x & 127;
    const uint32_t quarter = tmem + ((uint32_t)(warp * 32) << 16), o_at = quarter + S::kOCol;
    const int t_first = ranges.begin(blockIdx.x);
    Ring<S::kStages> ring;
    Ring<kBufs> at;
    uint64_t* at_rest = nullptr;                         // the barrier of the product before
    uint32_t rest_phase = 0;
    for (uint32_t seg = 0; w.left > 0; ++seg, w.next(p)) {
      const uint32_t buf = seg & 1;
      bool ok = wait_warp(&ctl->q_full[buf], (seg >> 1) & 1);
      const int base = w.len - p.Q, all_lo = ctl->all_lo[buf];
      const float f = ctl->f[buf][r];
      const int row = ctl->row[buf][r], lo = ctl->lo[buf][r];
      const bool idle = __all_sync(kFull, row < 0);      // no column of this warp
      Refs refs{0.f, kNone, 0.f};
      // of the references: what a weight's exponent has beside its score and scale, what takes a block's weights to the
      // sum's units, and the smallest byte of a values' scale that one exponential will do for (256: none)
      float offset = 0.f, back = 0.f;
      int least_ev = 256;
      auto known = [&]() {
        offset = kWeightScale - refs.w - refs.m;
        back = ex2_approx(refs.w - kWeightScale);
        const bool plain = fabsf(refs.m) < 1048576.f && fabsf(refs.w) < 100.f;
        const float highest = redux_max(refs.w);
        least_ev = __all_sync(kFull, plain) ? (int)highest - 80 + 127 : 256;
      };
      int t0 = (w.first + w.at) * kTile + half * kPageTokens;
      bool there = false;                                // the next tile's scores, as far as is known
      for (int i = 0; ok && i < w.count; ++i, t0 += kTile) {
        if (!__all_sync(kFull, there)) ok = wait_warp(&ctl->full[ring.st], ring.phase) && wait_warp(&ctl->s_full[at.st], at.phase);
        tc_fence_after();
        if (!idle) {
          const bool page_ok = ((ctl->pages_ok[ring.st] >> half) & 1) != 0, whole = page_ok && t0 >= all_lo && t0 + kPageTokens <= base;
          uint2 sc = reinterpret_cast<const uint2*>(&ctl->scales[ring.st][half])[w.kvh & 1];
          const uint32_t s_at = quarter + at.st * kTile + half * kPageTokens;
          uint64_t mine = ~0ull;
          if (__builtin_expect(!whole, 0)) {
            // (what a padding node's column sums is not wanted: it attends to what any does, for references of the page's size)
            mine = page_ok ? (lo == INT_MAX ? bits(ctl->any_lo[buf] - t0, base - t0) | nodes_at(ctl->any_mask[buf], base, t0) : bits(lo - t0, base - t0) | nodes_at(ctl->mask[buf][r], base, t0)) : 0;
            sc = leave_out(s_at, mine, sc);
          }
          if (__builtin_expect(least_ev > 255, 0) && !bar_any(kBarQuarter + warp, 64, !ok)) {
            start(refs, half, s_at, f, sc);
            known();
          }
          const uint32_t ev2 = __vminu2(__byte_perm(sc.y, 0u, 0x4140), __byte_perm(sc.y, 0u, 0x4342));
          uint32_t out[32];
          float more = 0.f, most = 0.f;
          // (of the warp: its loads are made by all lanes together)
          const bool fits = __all_sync(kFull, ok && (int)min(ev2 & 0xFFu, ev2 >> 16) >= least_ev);
          // One exponential serves w and l where fp32 holds the one beside the other: the smallest that matters to l,
          // 2^-40, has a weight above 2^-120.
          if (fits) {
            uint2 left = sc;
#pragma unroll 1
            for (int part = 0; part < 64; part += 32) {
              uint32_t s[32];
              tmem_ld32(s_at + part, s);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) out[k] = out[16 + k];
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const uint32_t kb = (left.x >> (8 * b)) & 0xFFu, vb = (left.y >> (8 * b)) & 0xFFu;
                const float c = fmaf(f, __uint_as_float(kb << 23), 1e-37f);      // (not 0: -inf times it stays what it is)
                const float k0 = (__uint_as_float(0x4B000000u | vb) - 8388735.f) + offset;     // whole numbers: exact
                const float2 cc = make_float2(c, c), kk = make_float2(k0, k0);
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                  const float2 a = __ffma2_rn(pair_of(s, b * 16 + k), cc, kk);
                  const float2 e = make_float2(ex2_approx(a.x), ex2_approx(a.y));
                  sum = __fadd2_rn(sum, e);
                  out[16 + b * 8 + k / 2] = narrow2<true>(e.x, e.y);
                }
                const float both = sum.x + sum.y;
                most = fmaxf(most, both);
                more = fmaf(both * back, __uint_as_float((254u - vb) << 23), more);
              }
              left.x >>= 16;
              left.y >>= 16;
            }
          }
          if (__builtin_expect(!bar_any(kBarQuarter + warp, 64, !fits || most > kMostWeights), 1)) {
            refs.l += more;
            tmem_st32(s_at, out);
          } else if (bar_any(kBarQuarter + warp, 64, !ok)) {
            ok = false;
            break;
          } else {
            // (both halves' warps of a quarter go on together, or give up together)
            ok = !bar_any(kBarQuarter + warp, 64, !careful(refs, half, s_at, f, sc, mine, i > 0 ? at_rest : nullptr, rest_phase, o_at));
            known();
          }
        }
        uint64_t *const done = &ctl->w_full[at.st], *const free = &ctl->empty[ring.st];
        at_rest = &ctl->o_done[at.st];
        rest_phase = at.phase;
        ring.next();
        at.next();
        // (asked for here, the answer comes while the weights are stored)
        there = mbar_test(&ctl->full[ring.st], ring.phase) & mbar_test(&ctl->s_full[at.st], at.phase) & (i + 1 < w.count);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) {
          mbar_arrive(done);
          mbar_arrive(free);
        }
      }
      // ---- the segment's end: half of the dims each
      ok = ok && wait_warp(at_rest, rest_phase);
      ctl->l[half][r] = refs.l;
      tc_fence_before();
      if (bar_any(kBarSoftmax, kSoftmaxThreads, !ok)) return;
      tc_fence_after();
      const bool pad = lo == INT_MAX;                    // no node: whatever was summed is not wanted
      const float top = refs.none() || pad ? kNone : refs.m, sum = pad ? 0.f : ctl->l[0][r] + ctl->l[1][r];
      // what O is multiplied by makes it the weighted mean at once, in two factors that stay far from fp32's ends
      const int up = max(0, min(126, (int)((__float_as_uint(sum) >> 23) & 0xFFu) - 127));
      const float inv = inverse(sum * __uint_as_float((uint32_t)(127 - up) << 23));
      const float factor = ex2_approx(0.5f * ((refs.none() ? 0.f : refs.w) - kWeightScale - (float)up)), first = factor * inv;
      const bool poisoned = ctl->any_poison[buf] != 0, full_unit = w.whole();
      const int slot = 2 * (int)blockIdx.x + second_slot(t_first, w.pos);
      if (!idle) {
#pragma unroll 1
        for (int k0 = 0; k0 < D / 2; k0 += 16) {
          const int d0 = half * (D / 2) + k0;
          __syncwarp();
          uint32_t a[16];
          tmem_ld16(o_at + d0, a);
          tmem_wait_ld();
          float o[16];
          const uint32_t bad = poisoned ? ctl->poison[buf][r][d0 >> 5] >> (d0 & 31) : 0u;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            o[k] = pad ? 0.f : __uint_as_float(a[k]) * first * factor;
            if ((bad >> k) & 1) o[k] = __int_as_float(0x7fc00000);
          }
          if (row >= 0) {
            if (full_unit) {
              uint4* to = reinterpret_cast<uint4*>(p.out + (int64_t)row * D + d0);
#pragma unroll
              for (int k = 0; k < 2; ++k)
                to[k] = make_uint4(narrow2<kHalf>(o[8 * k], o[8 * k + 1]), narrow2<kHalf>(o[8 * k + 2], o[8 * k + 3]),
                                   narrow2<kHalf>(o[8 * k + 4], o[8 * k + 5]), narrow2<kHalf>(o[8 * k + 6], o[8 * k + 7]));
            } else {
              // four dims of all columns side by side: a warp writes 512 bytes in one piece
              float4* to = reinterpret_cast<float4*>(p.part_o) + ((int64_t)slot * (D / 4) + d0 / 4) * kCols + r;
#pragma unroll
              for (int k = 0; k < 4; ++k) to[k * kCols] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            }
          }
        }
        if (half == 0 && row >= 0) {
          if (full_unit) p.lse[row] = sum == 0.f ? neg_inf() : (top + log2f(sum)) * 0.69314718055994530942f;
          else reinterpret_cast<float2*>(p.part_ml)[slot * kCols + r] = make_float2(top, sum);
        }
      }
      tc_fence_before();
      bar_sync(kBarSoftmax, kSoftmaxThreads);            // all have read O, the notes of NaN and each other's sums
      if (poisoned) {
        if (half == 0)
          for (int k = 0; k < 4; ++k) ctl->poison[buf][r][k] = 0;
        if (threadIdx.x == 256) ctl->any_poison[buf] = 0;
        bar_sync(kBarSoftmax, kSoftmaxThreads);
      }
      if (lane == 0) mbar_arrive(&ctl->done[buf]);
      if (!full_unit && w.at == 0 && threadIdx.x == 256)
        *shared = Shared{ranges.of(w.pos + kUnitCost + w.n - 1), second_slot(t_first, w.pos), w.b, w.kvh, w.ct};
    }
  }
};

template <int D, bool kHalf>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_kernel(const __grid_constant__ Kv8TreeParams p) {
  constexpr int kQ = kHalf ? 3 : 2;
  using S = Shape<D, kQ>;
  using Ctl = Control<S::kStages>;
  static_assert(sizeof(Ctl) <= S::kControl, "the control block fits its share");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qimg = stages + S::kStages * S::kStageBytes;
  uint8_t* vimg = qimg + S::kQBytes;
  Ctl* ctl = reinterpret_cast<Ctl*>(vimg + S::kVBufs * S::kVBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 64) {
    prefetch_tensormap(&p.cache_map);
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&ctl->full[i], 1 + kHalves);           // the codes' bytes, every page's scale bytes
      mbar_init(&ctl->empty[i], (kFeeders + kSoftmaxThreads) / 32);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->q_full[i], kFeeders / 32 + 1);
      mbar_init(&ctl->done[i], kSoftmaxThreads / 32);
      mbar_init(&ctl->drain[i], 1);
      ctl->any_poison[i] = 0;
    }
    mbar_init(&ctl->q_empty, 1);
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->w_full[i], kSoftmaxThreads / 32);
      mbar_init(&ctl->o_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&ctl->v_full[i], kFeeders / 32);
    ctl->abort = 0;
    fence_barrier_init();
  }
  for (int i = tid; i < 2 * kCols * 4; i += kTreeThreads) (&ctl->poison[0][0][0])[i] = 0;
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, S::kTmem);
    tmem_relinquish();
  }

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Shared* shared = reinterpret_cast<Shared*>(p.arrived) + blockIdx.x;
  if (tid == 0) shared->last = -1;
  // the whole sequence: every thread sums a run of requests
  const int cts = (p.Q * p.group + kCols - 1) / kCols;
  const int per = (p.B + kTreeThreads - 1) / kTreeThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  int sum = 0;
  for (int b = b0; b < b1; ++b) {
    int first, n;
    unit_tiles<kTile>(p, max(0, p.seq_lens[b]), first, n);
    sum += n + kUnitCost;
  }
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(kFull, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) ctl->scan_sum[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int of_warp = lane < kTreeThreads / 32 ? ctl->scan_sum[lane] : 0;
  const int before = (__reduce_add_sync(kFull, lane < warp ? of_warp : 0) + incl - sum) * p.kv_heads;
  const int all = __reduce_add_sync(kFull, of_warp) * p.kv_heads;      // of one column tile
  const int units = p.B * p.kv_heads * cts, tiles = all * cts - kUnitCost * units;
  const Ranges ranges(all * cts, min((int)gridDim.x, max(units, (tiles + kMinTiles - 1) / kMinTiles)));
  const int cta = blockIdx.x;
  const int t_begin = ranges.begin(cta), t_end = cta < ranges.ctas ? ranges.begin(cta + 1) : t_begin;
  const int ct = t_begin / all, in_ct = t_begin - ct * all;
  if (t_begin < t_end && before <= in_ct && in_ct < before + sum * p.kv_heads) {
    int b = b0, at = before;
    for (;; ++b) {
      int first, n;
      unit_tiles<kTile>(p, max(0, p.seq_lens[b]), first, n);
      if (in_ct < at + (n + kUnitCost) * p.kv_heads) break;
      at += (n + kUnitCost) * p.kv_heads;
    }
    ctl->start_b = b;
    ctl->start_before = at;
  }
  __syncthreads();
  Walk<kTile, kUnitCost> w{};
  w.left = t_end - t_begin;
  if (w.left > 0) {
    w.ct = ct;
    w.b = ctl->start_b;
    w.load(p);
    const int in = in_ct - ctl->start_before, each = w.n + kUnitCost;
    w.kvh = in / each;
    w.pos = t_begin - (in - w.kvh * each);
    w.take(in - w.kvh * each);
    const uint32_t tmem = ctl->tmem_base;
    Cta<D, kQ> c{p, stages, qimg, vimg, ctl};
    if (warp == 0) {
      c.producer(w);
    } else if (warp == 1) {
      if (lane == 0) c.issue_s(w, tmem);
      __syncwarp();
    } else if (warp == 2) {
      c.columns(w);
    } else if (warp == 3) {
      if (lane == 0) c.issue_o(w, tmem);
      __syncwarp();
    } else if (warp >= 8) {
      c.template softmax<kHalf>(w, tmem, ranges, shared);
    } else if (warp >= 4) {
      c.template feed<kHalf>(w);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(ctl->tmem_base, S::kTmem);
  }
}

// Means of a shared unit's parts, added by the sums that they are of: a lane a column, eight dims a warp. (Four and 16 take
// as long where units are many, and 16 some 2 us more where one is long.)
template <int D, bool kHalf>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Kv8TreeParams p) {
  constexpr int kN = 2;                             // four dims each
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = 8 * blockIdx.z + (threadIdx.x >> 5), first = blockIdx.x, r = blockIdx.y * 32 + lane;
  const Shared s = reinterpret_cast<const Shared*>(p.arrived)[first];
  const int col = s.ct * kCols + r, j = (int)(((uint64_t)(uint32_t)col * p.group_inverse) >> 24);
  if (s.last < 0 || col >= p.Q * p.group) return;
  const int64_t row = ((int64_t)s.b * p.Q + j) * p.H + s.kvh * p.group + (col - j * p.group);
  auto slot = [&](int cta) { return (int64_t)(2 * cta + (cta == first ? s.slot : 0)); };
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  float m = kNone, sum = 0.f;
#pragma unroll 8
  for (int c = first; c <= s.last; ++c) m = fmaxf(m, ml[slot(c) * kCols + r].x);
#pragma unroll 8
  for (int c = first; c <= s.last; ++c) {
    const float2 x = ml[slot(c) * kCols + r];
    sum += x.y * ratio(x.x, m);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  float4 o[kN] = {};
#pragma unroll 4
  for (int c = first; c <= s.last; ++c) {
    const float2 x = ml[slot(c) * kCols + r];
    const float f = x.y * ratio(x.x, m) * inv;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const float4 v = reinterpret_cast<const float4*>(p.part_o)[(slot(c) * (D / 4) + warp * kN + k) * kCols + r];
      o[k].x = fmaf(v.x, f, o[k].x);
      o[k].y = fmaf(v.y, f, o[k].y);
      o[k].z = fmaf(v.z, f, o[k].z);
      o[k].w = fmaf(v.w, f, o[k].w);
    }
  }
  uint2* to = reinterpret_cast<uint2*>(p.out + row * D + warp * kN * 4);
#pragma unroll
  for (int k = 0; k < kN; ++k) to[k] = make_uint2(narrow2<kHalf>(o[k].x, o[k].y), narrow2<kHalf>(o[k].z, o[k].w));
  if (warp == 0) p.lse[row] = sum == 0.f ? neg_inf() : (m + log2f(sum)) * 0.69314718055994530942f;
}

template <int D, bool kHalf>
cudaError_t launch(const Kv8TreeParams& p, cudaStream_t stream) {
  using S = Shape<D, kHalf ? 3 : 2>;
  constexpr size_t smem = 1024 + (size_t)S::kStages * S::kStageBytes + S::kQBytes + S::kVBufs * S::kVBytes + S::kControl;
  static_assert(smem <= 232448, "exceeds the 227 KB shared-memory limit");
  static std::mutex mu;
  static bool allowed[64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 64 || !allowed[dev]) {
      err = cudaFuncSetAttribute(tree_kernel<D, kHalf>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (err != cudaSuccess) return err;
      if (dev < 64) allowed[dev] = true;
    }
  }
  // Dependent launches: a CTA sets itself up while the grid before it in the stream ends, and waits for all of that grid
  // before it reads or writes memory.
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.ctas, 1, 1);
  cfg.blockDim = dim3(kTreeThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, tree_kernel<D, kHalf>, p);
  if (err != cudaSuccess) return err;
  cfg.gridDim = dim3((unsigned)p.ctas, kCols / 32, D / 64);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_kernel<D, kHalf>, p);
}

}  // namespace

static_assert(sizeof(Shared) <= 3 * sizeof(uint64_t), "the workspace holds three words a CTA");
int kv8_tree_columns() { return kCols; }

cudaError_t launch_kv8_decode_tree(const Kv8TreeParams& p, int head_dim, bool fp16, cudaStream_t stream) {
  if (head_dim == 128) return fp16 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
  return fp16 ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
}

}  // namespace nvfp4mla
