// kv8_decode: attention of a step's queries over the 8-bit per-head cache.
//
// What it computes. For one request and key/value head, the columns c = (query, head of the group)
// share every key and value row, so the step is two products over a 128-token tile:
//   S[t, c] = K[t, :] . q_c            z = scale 2^(ek_t - 127) S        (ek, ev: scale bytes)
//   O[d, c] += sum_t V[t, d] w[t, c]   w = 2^(z log2e + ev_t - 127 - M_c)
// with M_c a running reference, at most 2^4 below the largest exponent so far, and beside it the
// softmax's own running sum l_c = sum_t 2^(z log2e - m_c). A value's block scale goes into the
// weight's exponent before the reference is taken.
//
// What bounds it. A token costs 2 D + 0.5 bytes per head and 4 D operations per column: below some
// 250 operations a byte the step is bound by memory, so the codes have to reach the tensor cores as
// they lie in the cache, without a conversion in between. 8-bit products do that: K and V are the A
// operands straight from where TMA put them (K K-major, V M-major), and the other operands, q and w,
// are written as sums of 8-bit parts, each a sixteenth of the one before:
//   x = x_0 + x_1/16 (+ x_2/256 (+ x_3/4096)),   x_i = 8 bits of (what is left x 16^i)
// The parts are further columns of the B operand (their products land in columns of their own and are
// added in fp32 afterwards), so that A is read from shared memory once.
//   q: E4M3. Two parts hold a bf16, three an fp16, with its row's largest element at 2^7 to 2^8, down to
//     the last part's half step: 2^-14 for two, 2^-18 for three. So an element is off by at most 2^-21
//     (2^-25) of its row's largest, and exact from 2^-13 of that on for bf16, 2^-14 for fp16.
//   w: E5M2, four parts: 2^-15 of the weight, whose largest is 2^11 to 2^15; the last part's half step is
//     2^-17/4096, 2^-40 of the largest. E4M3 parts hold one bit more of a weight near the largest, but
//     have 2^-26 in the place of that 2^-40, and what is below adds to l and not to O: one key as heavy
//     as 100,000 others together, whose value block had a scale 2^10 times theirs, took all of the
//     others' share.
//
// One CTA per SM, persistent. The tiles of all (request, key/value head, column tile) units form
// one sequence, found by every CTA from the lengths, and each CTA takes one contiguous range of it.
//   warp 0     producer: page numbers a group of tiles ahead, then per stage (128 rows of 128 bytes
//              of K and of V) the TMA boxes of its pages and their scale bytes into a ring
//   warp 1     issues S = K q;  warp 3: issues O += V w (two threads, so that neither waits for the other)
//   warp 2     queries of the next unit: scaling by a power of two, parts, two buffers
//   warps 4..  softmax: two streams of tiles, a warpgroup or two each (thread = token). Each stream has
//              its own S, w and O, and keeps its own M, m, l; they are added at the unit's end
// A stage is 128 rows of 128 bytes: a token each, or two tokens of 64 dims, which one softmax thread has.
// A unit that several CTAs share is joined by whichever of them finishes last: the others leave
// (m, l, O) in the workspace and count themselves.
//
// Measured (device time, inputs beyond L2, 152 SMs): 8 columns and 128 dims run at the memory's pace:
// 16 requests of 20-90K tokens, 8 key/value heads: 1.38 GB in 210 us, 6.6 TB/s, 97 % of the measured copy
// bandwidth; one request of 131K tokens: 269 MB in 51.5 us (77 %: 5 us until the first product, 5 from the
// last to the joined result). With 64 dims a byte brings twice the softmax work: 64 requests of 4-30K
// tokens: 871 MB in 152 us (85 %). With 16 columns the softmax's chain of a tile sets the pace, some 0.8 us
// a stage at 128 dims and 1.1 at 64 (32 requests of 4-16K, two queries of 8 heads: 595 MB in 109 us, 81 %;
// four queries, whose two column tiles read the codes twice, 181 us, 49 %; with 64 dims, four queries of 4
// heads, 105, 62 %). It is latency more than issue: in the four queries' step 57 % of the issue slots are
// taken, and loads (tensor memory's among them) are the largest stall. Fewer instructions and registers
// shorten it all the same: pairs of columns in one instruction took the first two from 117 and 202 to 115
// and 198 us, a join with few registers, beside which the compiler kept the tile loop's values in
// registers, to 109 and 179.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstddef>
#include <mutex>

#include "../../include/nvfp4mla.h"
#include "kv8.h"
#include "ptx.cuh"

namespace nvfp4mla {
namespace {

using namespace ptx;

constexpr int kRows = 128;             // 128-byte rows of K or V in a stage: a token each, or two of 64 dims
constexpr int kWParts = 4;
constexpr float kHeadroom = 4.f;       // log2: how far above the reference a weight's exponent may come
constexpr float kWeightScale = 11.f;   // log2: weights are held times 2^11: 2^4 above it, a part is at most 2^15 (E5M2: 57,344)
constexpr float kSumHeadroom = 60.f;   // log2: the same for the sum, which fp32 holds
constexpr unsigned kFull = 0xFFFFFFFFu;

// Sizes of the instance with D dims and NC columns.
template <int D, int NC, int kQ>
struct Shape {
  static constexpr int kQParts = kQ;                            // of a query element: 2 (bf16) or 3 (fp16)
  static constexpr bool kPair = D == 64;                        // a row is two tokens
  static constexpr int kHalves = kPair ? 2 : 1;                 // tokens of a row, and of a softmax thread
  // Two streams, that take the stages in turn. A softmax warpgroup has eight columns: it is bound by
  // latency, and with 16 columns two warpgroups took 0.6 of one's time.
  static constexpr int kStreams = 2;
  static constexpr int kGroups = NC / 8;
  static constexpr int kSoftmax = kStreams * kGroups * 128;     // its threads
  static constexpr int kThreads = 128 + kSoftmax;
  static constexpr int kTile = kPair ? 256 : 128;               // tokens of a stage
  static constexpr int kPages = kTile / kPageTokens;
  static constexpr int kPageRows = kRows / kPages;
  static constexpr int kGroup = 32 / kPages;                    // stages whose page numbers are read together
  static constexpr int kFewTiles = kPair ? 4 : 8;               // of a unit that is not worth splitting
  static constexpr int kMinTiles = kStreams;                    // of a CTA, on average: work for every stream
  static constexpr int kNS = (kQParts * NC + 15) / 16 * 16;     // columns of S
  static constexpr int kNO = kWParts * NC;                      // columns of O of a half
  static constexpr int kWRow = kHalves * kNO;                   // bytes of a row of w, columns of O
  static constexpr int kStageBytes = 2 * kRows * 128;           // groups of 8 rows of K and of V in turn
  static constexpr int kQBytes = (kNS * D + 1023) / 1024 * 1024;
  static constexpr int kWBytes = kRows * kWRow;
  static constexpr int kBudget = 232448 - 1024 - 6144;          // less alignment and the control block
  static constexpr int kFit = (kBudget - 2 * kQBytes - kStreams * kWBytes) / kStageBytes;
  static constexpr int kStages = kFit;
  // S of the next tile while this one's is read, where tensor memory holds it
  static constexpr int kBufs = kStreams * (2 * kHalves * kNS + kWRow) <= 512 ? 2 : 1;
  static constexpr int kSBuf = kHalves * kNS;                   // columns of a buffer of S
  static constexpr int kOCol = kStreams * kBufs * kSBuf;        // TMEM columns: S of the streams, then O
  static constexpr int kUsed = kOCol + kStreams * kWRow;
  static constexpr uint32_t kTmem = kUsed <= 256 ? 256 : 512;
  static constexpr uint32_t kSwQ = D == 128 ? SW_128B : SW_64B;
  static constexpr uint32_t kSwW = kWRow == 128 ? SW_128B : (kWRow == 64 ? SW_64B : SW_32B);
  static_assert(kUsed <= 512 && kStages >= 3, "fits");
};

template <int NC, int kStages, int kPages, int kStreams, int kWarps>
struct Control {
  uint64_t full[kStages], empty[kStages];    // empty: the product with V is complete
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[kStreams][2], w_full[kStreams][2];   // per buffer of S
  uint64_t drain[2];
  uint4 scales[kStages][kPages];       // per page: the scale bytes of two neighbouring heads
  uint32_t pages_ok[kStages];          // bit per page: it is one
  alignas(16) float f[2][NC];          // per query buffer: score of a column per unit of S, log2 units
  int hi[2][NC], lo[2][NC];            // positions that a column attends to
  int row[2][NC];                      // of out and lse, -1: no column
  int at0[2], at1[2], cols[2];         // positions of the tile's first and last column; its columns
  alignas(16) float top_w[kStreams][NC];   // the weights' reference: M less kWeightScale, less m (these four
                                           // are read four at a time)
  alignas(16) float top_s[kStreams][NC];   // m
  alignas(16) float scale_o[kStreams][NC];
  alignas(16) float scale_l[kStreams][NC];
  float part_max[kStreams][4][NC][2];  // of a warp: the largest score, and weight against that
  float part_l[kStreams][4][NC];
  uint32_t poison[kStreams][NC][4];    // dims that a NaN value reaches
  float join_m[NC], join_l[NC];
  alignas(8) float join_w[kStreams][NC][2];       // O's factor, in two
  int any_poison[kStreams];
  int scan_sum[kWarps];
  int start_before;                    // tiles before request start_b
  int start_b;
  int last;
  int abort;
  uint32_t tmem_base;
};

// Tiles of one unit of a request with `len` tokens: [first, first + n). A unit has at least one, so
// that a request without tokens is written too.
template <int kTile>
__device__ __forceinline__ void unit_tiles(const Kv8DecodeParams& p, int len, int& first, int& n) {
  constexpr int kPages = kTile / kPageTokens;
  const int64_t pages = min((int64_t)(len + (int64_t)kPageTokens - 1) / kPageTokens, p.max_pages);
  int last = len > 0 ? (int)((pages + kPages - 1) / kPages) : 1;
  first = 0;
  if (p.window > 0) {
    const int64_t from = (int64_t)len - p.Q - p.window + 1;
    if (from > 0) first = (int)(from / kTile);
  }
  if (first > last - 1) first = last - 1;
  n = last - first;
}

// The ranges of the CTAs: the first `more` of them are one tile longer. (The host refuses sizes whose
// tiles could leave 32 bits.)
struct Ranges {
  int ctas, each, more;
  __device__ __forceinline__ Ranges(int total, int n) : ctas(n), each(total / n), more(total - total / n * n) {}
  __device__ __forceinline__ int begin(int cta) const { return cta * each + min(cta, more); }
  __device__ __forceinline__ int of(int tile) const {
    const int longer = more * (each + 1);
    return tile < longer ? tile / (each + 1) : more + (tile - longer) / each;
  }
};

// What starting and ending a unit costs, in tiles: ranges count a unit of n tiles as kUnitCost + n, so
// that CTAs with many short units do not finish last. Measured with 0, 4, 8 and 12: 256 requests of
// 200-1,500 tokens 133, 99, 95 and 100 us; 64 of 4-30K with 64 dims 164, 148, 150 and 153; 32 of 900-9,000,
// four queries in a window, 59, 49, 50 and 52; 16 of 20-90K 208, 206, 206 and 207.
constexpr int kUnitCost = 8;

// A walk over the segments of this CTA: per unit, the tiles of it that the CTA has. Units go by column
// tile, request and key/value head; so the column tiles of one head's tokens run on different CTAs at
// about the same time, and all but one of them read the codes from L2.
template <int kTile>
struct Walk {
  int left;              // of the CTA's range, from this segment on
  int ct, b, kvh;        // the unit
  int len, first, n;     // the request's length and a unit's tiles
  int at, count;         // this segment: tiles at .. at + count - 1 of the unit
  int pos;               // of the unit's first tile, in the whole sequence

  __device__ __forceinline__ void load(const Kv8DecodeParams& p) {
    len = p.seq_lens[b];
    if (len < 0) len = 0;
    unit_tiles<kTile>(p, len, first, n);
  }
  // From `in` of the unit on, of which the first kUnitCost are no tiles.
  __device__ __forceinline__ void take(int in) {
    const int skip = in < kUnitCost ? kUnitCost - in : 0;
    left -= skip;
    at = in + skip - kUnitCost;
    count = min(n - at, left);
  }
  __device__ __forceinline__ void next(const Kv8DecodeParams& p) {
    left -= count;
    if (left <= 0) return;
    pos += n + kUnitCost;
    if (++kvh == p.kv_heads) {
      kvh = 0;
      if (++b == p.B) {
        b = 0;
        ++ct;
      }
      load(p);
    }
    take(0);
  }
  __device__ __forceinline__ bool whole() const { return count == n; }
};

__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
__device__ __forceinline__ bool bar_any(int id, int threads, bool v) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %3, 0;\n\tbarrier.cta.red.or.pred q, %1, %2, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(v ? 1 : 0)
      : "memory");
  return r != 0;
}

template <bool kHalf>
__device__ __forceinline__ float2 widen2(uint32_t w) {
  if constexpr (kHalf) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// (a, b) as kParts pairs of E4M3 parts: part[i] holds two bytes, a's in the low one. |a|, |b| <= 448.
template <int kParts>
__device__ __forceinline__ void split_parts(float a, float b, uint32_t (&part)[kParts]) {
  part[0] = f32x2_to_e4m3x2(a, b);
  uint32_t h = e4m3x2_to_f16x2(part[0]);
  const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&h));
  // (an element of q has at most 11 significant bits: what the first part leaves is an fp16, but for its last
  // subnormal bits, below what the other parts hold)
  const float2 left = __ffma2_rn(c, make_float2(-1.f, -1.f), make_float2(a, b));
  __half2 r = __floats2half2_rn(left.x, left.y);
  const __half2 sixteen = __floats2half2_rn(16.f, 16.f);
#pragma unroll
  for (int i = 1; i < kParts; ++i) {
    r = __hmul2(r, sixteen);
    part[i] = f16x2_to_e4m3x2(*reinterpret_cast<const uint32_t*>(&r));
    if (i + 1 < kParts) {
      h = e4m3x2_to_f16x2(part[i]);
      r = __hsub2(r, *reinterpret_cast<const __half2*>(&h));
    }
  }
}

// (a, b) as four pairs of E5M2 parts, 0 <= a, b <= 2^15. A part leaves at most 2^-3 of the power of two below
// its value, the next ones 2^-4 each: 2^-15 after four. The first two are taken off in fp32 (exactly); of what they
// leave the fp16 keeps 11 bits, more than the others hold.
__device__ __forceinline__ void split_weight(float a, float b, uint32_t (&part)[kWParts]) {
  auto wide = [](uint32_t two) {
    const uint32_t h = e5m2x2_to_f16x2(two);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
  };
  const float2 minus = make_float2(-1.f, -1.f), sixteen = make_float2(16.f, 16.f);
  part[0] = f32x2_to_e5m2x2(a, b);
  float2 left = __fmul2_rn(__ffma2_rn(wide(part[0]), minus, make_float2(a, b)), sixteen);
  part[1] = f32x2_to_e5m2x2(left.x, left.y);
  left = __fmul2_rn(__ffma2_rn(wide(part[1]), minus, left), sixteen);
  const __half2 r = __floats2half2_rn(left.x, left.y);
  part[2] = f16x2_to_e5m2x2(*reinterpret_cast<const uint32_t*>(&r));
  const uint32_t h = e5m2x2_to_f16x2(part[2]);
  const __half2 last = __hmul2(__hsub2(r, *reinterpret_cast<const __half2*>(&h)), __floats2half2_rn(16.f, 16.f));
  part[3] = f16x2_to_e5m2x2(*reinterpret_cast<const uint32_t*>(&last));
}

// The largest of three; a NaN counts as none.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// The largest over the warp; a NaN counts as none.
__device__ __forceinline__ float redux_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
template <int N>
__device__ __forceinline__ float2 pair_of(const uint32_t (&v)[N], int i) {
  return make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
}
__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
// A reference before any position: below every exponent that fp32 holds but the last few, and finite, so that
// what is left out (an exponent of -inf) stays 0 against it.
constexpr float kNone = -3e38f;
// 2^(a - b), 1 where the two are equal.
__device__ __forceinline__ float ratio(float a, float b) { return a == b ? 1.f : ex2_approx(a - b); }

template <int D, int NC, int kQ>
struct Cta {
  using S = Shape<D, NC, kQ>;
  static constexpr int kQParts = kQ;
  using Ctl = Control<NC, S::kStages, S::kPages, S::kStreams, S::kThreads / 32>;
  using Walk = ::nvfp4mla::Walk<S::kTile>;
  const Kv8DecodeParams& p;
  uint8_t* stages;
  uint8_t* qbuf;
  uint8_t* wbuf;
  Ctl* ctl;

  // The waiting, its limit and the error are a function of their own: the loops of five roles run from
  // one instruction cache, and with the long wait inlined at each call, and the rare branches of the
  // softmax in line, the 16-column steps took 6 to 8 % longer (32 requests of 4-16K, two queries of 8
  // heads: 117 us against 124) and 256 short requests 111 us against 123.
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    return wait_long(ctl, p.status, bar, parity);
  }
  static __device__ __noinline__ bool wait_long(Ctl* ctl, int32_t* status, uint64_t* bar, uint32_t parity) {
    if (mbar_wait(bar, parity, &ctl->abort, kWaitTimeoutNs)) return true;
    if (atomicExch(&ctl->abort, 1) == 0 && status != nullptr) atomicAdd(status + NVFP4MLA_STAT_TIMEOUT, 1);
    return false;
  }
  // The product with V of the stage number g is complete. Not for a stage that may have been filled
  // again and read since.
  __device__ __forceinline__ bool product_done(uint32_t g) { return wait(&ctl->empty[g % S::kStages], (g / S::kStages) & 1); }
  // First position that a query at `at` attends to.
  __device__ __forceinline__ int window_start(int at) const { return p.window > 0 && at + 1 > p.window ? at + 1 - p.window : 0; }

  // ---------------------------------------------------------------- producer (warp 0)
  // Page numbers of a group of tiles from i on: a lane a page. -1: not needed, or none.
  __device__ __forceinline__ int load_pages(const Walk& w, int i) {
    const int lane = threadIdx.x & 31;
    const int tile = i + lane / S::kPages;
    if (tile >= w.count) return -1;
    const int64_t col = S::kPages * ((int64_t)w.first + w.at + tile) + lane % S::kPages;
    const int64_t from = p.window > 0 ? (int64_t)w.len - p.Q - p.window + 1 : 0;
    if (col * kPageTokens >= w.len || (col + 1) * kPageTokens <= from) return -1;
    int page = -1;
    if (col < p.max_pages) {
      page = p.page_table[(int64_t)w.b * p.max_pages + col];
      if (page >= 0 && page < p.num_pages) return page;
      page = -1;
    } else {
      return -1;                       // counted with the pages behind the table
    }
    if (w.ct == 0 && w.kvh == 0 && p.status != nullptr) atomicAdd(p.status + NVFP4MLA_STAT_BAD_PAGE, 1);
    return page;
  }

  __device__ void producer(Walk w) {
    const int lane = threadIdx.x & 31;
    uint32_t g = 0;
    if (p.withhold) return;
    int pages = w.left > 0 ? load_pages(w, 0) : -1;
    while (w.left > 0) {
      const int kvh = w.kvh;
      if (w.kvh == 0 && w.ct == 0 && w.at + w.count == w.n && lane == 0 && p.status != nullptr) {
        const int64_t need = ((int64_t)w.len + kPageTokens - 1) / kPageTokens;
        int64_t from = p.window > 0 ? ((int64_t)w.len - p.Q - p.window + 1) / kPageTokens : 0;
        if (from < p.max_pages) from = p.max_pages;
        if (need > from) atomicAdd(p.status + NVFP4MLA_STAT_BAD_PAGE, (int)(need - from));
      }
      for (int i = 0; i < w.count; i += S::kGroup) {
        const int mine = pages;
        if (i + S::kGroup < w.count) {
          pages = load_pages(w, i + S::kGroup);
        } else {
          Walk nx = w;
          nx.next(p);
          pages = nx.left > 0 ? load_pages(nx, 0) : -1;
        }
        const int m = min(S::kGroup, w.count - i);
        for (int k = 0; k < m; ++k, ++g) {
          // a lane a page: one box of its codes (a page that is none reads from behind the cache:
          // zeros) and its scale bytes
          const int page = __shfl_sync(kFull, mine, S::kPages * k + lane % S::kPages);
          const uint32_t have = __ballot_sync(kFull, page >= 0) & ((1u << S::kPages) - 1);
          const uint32_t st = g % S::kStages, round = g / S::kStages;
          bool ok = true;
          if (lane == 0) {
            ok = wait(&ctl->empty[st], (round & 1) ^ 1);
            if (ok) {
              ctl->pages_ok[st] = have;
              mbar_arrive_expect_tx(&ctl->full[st], S::kStageBytes);
            }
          }
          ok = __shfl_sync(kFull, ok ? 1 : 0, 0) != 0;
          if (ok && lane < S::kPages) {
            tma_load_5d(stages + st * S::kStageBytes + lane * 2 * kPageTokens * D, &p.cache_map, 0, 0, 0, kvh * (kPageTokens * D / 1024),
                        page >= 0 ? page : (int)p.num_pages, &ctl->full[st]);
            // (a TMA copy takes the warp some 80 ns, a load-store copy by all lanes at once a few)
            if (page >= 0) cp_async_16(&ctl->scales[st][lane], p.cache + page * p.page_bytes + kv8_scales_off(p.kv_heads, D, kvh & ~1));
            cp_async_arrive(&ctl->full[st]);
          }
          __syncwarp();
          if (!ok) {
            drain_copies(g);
            return;
          }
        }
      }
      w.next(p);
    }
    if (ctl_aborted()) drain_copies(g);
  }
  __device__ __forceinline__ bool ctl_aborted() { return *reinterpret_cast<volatile int*>(&ctl->abort) != 0; }

  // After a wait gave up: the copies of tiles before g that are still in flight land (bounded).
  __device__ void drain_copies(uint32_t g) {
    if ((threadIdx.x & 31) != 0) return;
    const uint32_t n = g < (uint32_t)S::kStages ? g : (uint32_t)S::kStages;
    for (uint32_t i = 0; i < n; ++i) {
      const uint32_t t = g - 1 - i;
      mbar_wait(&ctl->full[t % S::kStages], (t / S::kStages) & 1, nullptr, kWaitTimeoutNs);
    }
  }

  // The two issuing threads. What bounds them is their own instructions (an MMA takes its issuer some
  // 80 cycles, a commit as much), so each tile has one commit of each, descriptors differ in their low
  // words alone, and stages and phases are counted instead of divided.
  struct Ring {
    uint32_t st = 0, phase = 0;
    __device__ __forceinline__ void next() {
      if (++st == (uint32_t)S::kStages) {
        st = 0;
        phase ^= 1;
      }
    }
  };

  // ---------------------------------------------------------------- S = K q (warp 1, one thread)
  __device__ void issue_s(Walk w, uint32_t tmem) {
    constexpr uint32_t kId = idesc_e4m3(128, S::kNS, false, false);
    const uint64_t kd = sdesc(smem_u32(stages), 16, 2048, SW_128B), qd = sdesc(smem_u32(qbuf), 16, 8 * D, S::kSwQ);
    Ring ring;
    uint32_t uses[2] = {0, 0};             // tiles that the streams have had
    bool ok = true;
    for (uint32_t seg = 0; ok && w.left > 0; ++seg, w.next(p)) {
      const uint32_t buf = seg & 1;
      ok = wait(&ctl->q_full[buf], (seg >> 1) & 1);
      const uint32_t q_lo = (uint32_t)qd + ((buf * S::kQBytes) >> 4);
      for (int i = 0; ok && i < w.count; ++i) {
        const int stream = i & 1;
        const uint32_t u = stream == 0 ? uses[0]++ : uses[1]++, sb = u % S::kBufs;
        ok = wait(&ctl->full[ring.st], ring.phase);
        // this buffer's last S has been read once its weights are written (before the first, parity 1 is
        // that of the phase before any)
        ok = ok && wait(&ctl->w_full[stream][sb], ((u / S::kBufs) & 1) ^ 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int half = 0; half < S::kHalves; ++half) {
          const uint32_t d = tmem + (stream * S::kBufs + sb) * S::kSBuf + half * S::kNS;
          const uint32_t k_lo = (uint32_t)kd + ((ring.st * S::kStageBytes + half * 64) >> 4);   // a row's first or second token
          umma_f8_ss_w<0>(d, k_lo, (uint32_t)(kd >> 32), q_lo, (uint32_t)(qd >> 32), kId);
#pragma unroll
          for (int k = 1; k < D / 32; ++k)
            umma_f8_ss_w<1>(d, k_lo + 2 * k, (uint32_t)(kd >> 32), q_lo + 2 * k, (uint32_t)(qd >> 32), kId);
        }
        umma_commit(&ctl->s_full[stream][sb]);
        ring.next();
      }
      if (ok) umma_commit(&ctl->q_empty[buf]);
    }
    umma_commit(&ctl->drain[0]);
    mbar_wait(&ctl->drain[0], 0, nullptr, kWaitTimeoutNs);
  }

  // ---------------------------------------------------------------- O += V w (warp 3, one thread)
  // With 64 dims the rows of V are 128 values, of two tokens, and those of w the weights of either: one
  // product takes both. Of its 128 x 2 kNO results the even token's dims with the even token's weights
  // are wanted, and the odd one's with the odd one's; the other half of the work costs less than twice
  // as many instructions of this thread would.
  __device__ void issue_o(Walk w, uint32_t tmem) {
    constexpr uint32_t kId = idesc_e4m3(128, S::kWRow, true, true, true);
    const uint64_t vd = sdesc(smem_u32(stages + 1024), 16, 2048, SW_128B), wd = sdesc(smem_u32(wbuf), 16, 8 * S::kWRow, S::kSwW);
    Ring ring;
    uint32_t uses[2] = {0, 0};             // tiles that the streams have had
    bool ok = true;
    for (; ok && w.left > 0; w.next(p)) {
      for (int i = 0; ok && i < w.count; ++i) {
        const int stream = i & 1;
        const uint32_t u = stream == 0 ? uses[0]++ : uses[1]++;
        ok = wait(&ctl->w_full[stream][u % S::kBufs], (u / S::kBufs) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + S::kOCol + stream * S::kWRow;
        const uint32_t v_lo = (uint32_t)vd + ((ring.st * S::kStageBytes) >> 4), w_lo = (uint32_t)wd + ((stream * S::kWBytes) >> 4);
        umma_f8_ss_w<-1>(d, v_lo, (uint32_t)(vd >> 32), w_lo, (uint32_t)(wd >> 32), kId, i >= S::kStreams ? 1u : 0u);
#pragma unroll
        for (int k = 1; k < kRows / 32; ++k)
          umma_f8_ss_w<1>(d, v_lo + k * 512, (uint32_t)(vd >> 32), w_lo + k * 2 * S::kWRow, (uint32_t)(wd >> 32), kId);
        umma_commit(&ctl->empty[ring.st]);
        ring.next();
      }
    }
    umma_commit(&ctl->drain[1]);
    mbar_wait(&ctl->drain[1], 0, nullptr, kWaitTimeoutNs);
  }

  // ---------------------------------------------------------------- queries (warp 2)
  template <bool kHalf>
  __device__ void queries(Walk w) {
    constexpr int kLanes = D / 8, kCols = 32 / kLanes;    // lanes a column, columns a round
    const int lane = threadIdx.x & 31, sub = lane / kLanes, ch = lane % kLanes;
    const int ncols = p.Q * p.group;
    for (uint32_t seg = 0; w.left > 0; ++seg, w.next(p)) {
      const uint32_t buf = seg & 1;
      const int kvh = w.kvh, ct = w.ct;
      uint8_t* img = qbuf + buf * S::kQBytes;
      constexpr int kRounds = NC / kCols, kAhead = kRounds < 4 ? kRounds : 4;
      auto load = [&](int round) {
        const int col = ct * NC + round * kCols + sub;
        if (round >= kRounds || col >= ncols) return make_uint4(0u, 0u, 0u, 0u);
        const int j = col / p.group, h = kvh * p.group + col - j * p.group;
        return *reinterpret_cast<const uint4*>(p.q + ((int64_t)w.b * p.Q + j) * p.q_token_stride + h * p.q_head_stride + ch * 8);
      };
      // four rounds' loads in flight, one round's code
      uint4 v[kAhead];
#pragma unroll
      for (int r = 0; r < kAhead; ++r) v[r] = load(r);
      const bool ok = wait(&ctl->q_empty[buf], ((seg >> 1) & 1) ^ 1);
      if (__any_sync(kFull, !ok)) return;
#pragma unroll 1
      for (int r = 0; r < kRounds; ++r) {
        const uint4 x4 = v[0];
#pragma unroll
        for (int k = 0; k + 1 < kAhead; ++k) v[k] = v[k + 1];
        v[kAhead - 1] = load(r + kAhead);
        {
          const int c = r * kCols + sub, col = ct * NC + c;
          const uint32_t ws[4] = {x4.x, x4.y, x4.z, x4.w};
          uint32_t top = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) top = __vmaxu2(top, ws[k] & 0x7FFF7FFFu);
          top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
          for (int d = 1; d < kLanes; d <<= 1) top = max(top, __shfl_xor_sync(kFull, top, d));
          const bool finite = top < (kHalf ? 0x7C00u : 0x7F80u);
          // the largest magnitude goes to [128, 256): a power of two, exact
          const int e = (int)(__float_as_uint(widen2<kHalf>(top).x) >> 23) - 127;
          const int sh = top == 0 || !finite ? 0 : min(7 - e, 126);
          const float mul = finite ? __uint_as_float((uint32_t)(sh + 127) << 23) : 0.f;
          uint32_t part[4][kQParts];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 x = widen2<kHalf>(ws[k]);
            split_parts(finite ? x.x * mul : 0.f, finite ? x.y * mul : 0.f, part[k]);
          }
#pragma unroll
          for (int i = 0; i < kQParts; ++i) {
            const int n = i * NC + c;
            const int chunk = D == 128 ? ((ch >> 1) ^ (n & 7)) : ((ch >> 1) ^ ((n >> 1) & 3));
            *reinterpret_cast<uint2*>(img + n * D + chunk * 16 + (ch & 1) * 8) =
                make_uint2(part[0][i] | (part[1][i] << 16), part[2][i] | (part[3][i] << 16));
          }
          if (ch == 0) {
            const float back = __uint_as_float((uint32_t)(127 - sh) << 23);
            ctl->f[buf][c] = col < ncols ? (finite ? p.scale_log2 * back : __int_as_float(0x7fc00000)) : 0.f;
            const int j = col / p.group, at = w.len - p.Q + j;
            ctl->row[buf][c] = col < ncols ? (w.b * p.Q + j) * p.H + kvh * p.group + (col - j * p.group) : -1;
            const int cols = min(NC, ncols - ct * NC);
            if (c == 0) ctl->at0[buf] = at;
            if (c == cols - 1) {
              ctl->at1[buf] = at;
              ctl->cols[buf] = cols;
            }
            ctl->hi[buf][c] = col < ncols ? at : -1;
            ctl->lo[buf][c] = window_start(at);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->q_full[buf]);
    }
  }

  // ---------------------------------------------------------------- softmax (warps 4-11, with 16 columns 4-19)
  // A token's row of V that no column attends to becomes zeros (it may hold anything), and a NaN in
  // one that only some columns attend to is taken out and noted for those.
  static __device__ __forceinline__ uint32_t nans_in(const uint4& x) {
    return __vcmpeq4(x.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(x.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu) |
           __vcmpeq4(x.z & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(x.w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
  }
  __device__ __forceinline__ void take_out(uint8_t* bytes, int d0, int t, uint32_t buf, int stream) {
    for (int k = 0; k < 16; ++k) {
      if ((bytes[k] & 0x7F) != 0x7F) continue;
      bytes[k] = 0;
      const int d = d0 + k;
      for (int c = 0; c < ctl->cols[buf]; ++c)
        if (t <= ctl->hi[buf][c] && t >= ctl->lo[buf][c]) atomicOr(&ctl->poison[stream][c][d >> 5], 1u << (d & 31));
      ctl->any_poison[stream] = 1;
    }
  }
  __device__ void clean_row(uint8_t* row, int r, int half, int t, bool any, uint32_t buf, int stream) {
    constexpr int kChunks = D / 16;
    auto chunk = [&](int i) { return reinterpret_cast<uint4*>(row + (((half * kChunks + i) ^ (r & 7)) * 16)); };
    if constexpr (S::kPair) {
      // the loads of a row of 64 dims all in flight: 32 requests' four queries in a window 58 us instead of
      // 60 (with 128 dims, more code than it saves: 256 short requests 99 instead of 95)
      uint4 x[kChunks];
      uint32_t nan = 0;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (any) x[i] = *chunk(i);
        else *chunk(i) = x[i];
      }
#pragma unroll
      for (int i = 0; i < kChunks; ++i) nan |= nans_in(x[i]);
      if (nan == 0) return;
#pragma unroll 1
      for (int i = 0; i < kChunks; ++i) take_out(reinterpret_cast<uint8_t*>(chunk(i)), i * 16, t, buf, stream);
    } else {
#pragma unroll 1
      for (int i = 0; i < kChunks; ++i) {
        if (!any) *chunk(i) = make_uint4(0u, 0u, 0u, 0u);
        else if (nans_in(*chunk(i)) != 0) take_out(reinterpret_cast<uint8_t*>(chunk(i)), i * 16, t, buf, stream);
      }
    }
  }

  // Counts this CTA among those that have left their partial results of a unit; true for the last to
  // come. A count of another call, or whatever the workspace held before, is replaced by the first to
  // come; the last leaves this call's count at none, as a replay of a captured call expects it.
  __device__ bool arrive(int c_lo, int c_hi) {
    uint64_t* at = p.arrived + c_lo;
    uint64_t old = add_acq_rel_gpu_u64(at, 1);
    for (;;) {
      if ((old & ~(uint64_t)0xFFFF) == p.tag) {
        if ((int)(old & 0xFFFF) != c_hi - c_lo) return false;
        st_relaxed_gpu_u64(at, p.tag);
        return true;
      }
      const uint64_t now = cas_acq_rel_gpu_u64(at, old + 1, p.tag | 1);
      if (now == old + 1) return false;      // two CTAs at least share a unit that is counted
      old = (now & ~(uint64_t)0xFFFF) == p.tag ? add_acq_rel_gpu_u64(at, 1) : now - 1;
    }
  }

  // A CTA's partial results go to its first slot for the unit that its range begins in, else to its
  // second: there are at most two such units.
  static __device__ __forceinline__ int second_slot(int begin, int pos) { return pos < begin ? 0 : 1; }

  template <bool kHalf>
  __device__ __forceinline__ void put(int64_t at, float v) {
    if constexpr (kHalf) p.out[at] = __half_as_ushort(__float2half_rn(v));
    else p.out[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }

  __device__ __forceinline__ void put_lse(int row, float m, float sum) {
    if (row >= 0) p.lse[row] = sum == 0.f ? neg_inf() : (m + log2f(sum)) * 0.69314718055994530942f;
  }
  // 1 / sum (to 2^-23), 0 where there was no position. A sum is 0, or at least 1 and far from fp32's end.
  static __device__ __forceinline__ float inverse(float sum) { return sum == 0.f ? 0.f : rcp_approx(sum); }

  // Joins the partial means that CTAs c_lo .. c_hi left of a unit, for dim d of this warpgroup's
  // columns, 32 at a time: a lane has the maxima and sums of one, and the outputs of kSlots are in flight
  // together, the first of them beside the maxima. (It has few registers on purpose: with every part's
  // maxima and sums in each thread, the compiler spilled: with 16 columns 197 us instead of 178, 32 requests
  // of 4-16K, four queries of 8 heads, and 120 instead of 106 with 64 dims. Of the eight instances one still
  // spills, 4 bytes: 64 dims, 16 columns, fp16.)
  template <bool kHalf>
  __device__ void join(const int* row, int c, int d, int c_lo, int c_hi, int first) {
    constexpr int kN = NC / (S::kSoftmax / 128), kSlots = S::kThreads == 384 ? 8 : 4;
    const int lane = threadIdx.x & 31;
    float m[kN], sum[kN], acc[kN];
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      m[k] = kNone;
      sum[k] = acc[k] = 0.f;
    }
    auto at = [&](int cta) { return (2 * cta + (cta == c_lo ? first : 0)) * NC + c; };
#pragma unroll 1
    for (int s0 = c_lo; s0 <= c_hi; s0 += 32) {
      const int n = min(32, c_hi - s0 + 1);
      float o[kSlots][kN], w[kN], l[kN];
      auto load = [&](int from) {
#pragma unroll
        for (int i = 0; i < kSlots; ++i)
#pragma unroll
          for (int k = 0; k < kN; ++k) o[i][k] = from + i < n ? __ldcg(p.part_o + (int64_t)(at(s0 + from + i) + k) * D + d) : 0.f;
      };
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const float2 ml = lane < n ? __ldcg(reinterpret_cast<const float2*>(p.part_ml) + at(s0 + lane) + k) : make_float2(kNone, 0.f);
        w[k] = ml.x;
        l[k] = ml.y;
      }
      load(0);
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const float m_new = fmaxf(m[k], redux_max(w[k])), keep = ratio(m[k], m_new);
        w[k] = l[k] * ratio(w[k], m_new);
        float all = w[k];
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) all += __shfl_xor_sync(kFull, all, x);
        all += sum[k] * keep;
        const float inv = inverse(all);      // acc, too, is a mean all the way
        acc[k] *= sum[k] * keep * inv;
        w[k] *= inv;
        sum[k] = all;
        m[k] = m_new;
      }
#pragma unroll 1
      for (int from = 0; from < n; from += kSlots) {
        if (from > 0) load(from);
#pragma unroll
        for (int i = 0; i < kSlots; ++i)
#pragma unroll
          for (int k = 0; k < kN; ++k) acc[k] = fmaf(o[i][k], __shfl_sync(kFull, w[k], (from + i) & 31), acc[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      if (row[c + k] < 0) break;
      put<kHalf>((int64_t)row[c + k] * D + d, acc[k]);
      if (d == 0) put_lse(row[c + k], m[k], sum[k]);
    }
  }

  template <bool kHalf>
  __device__ void softmax(Walk w, uint32_t tmem, const Ranges& ranges) {
    // the warpgroup's stream, and which of the columns are its own: own .. own + 7
    constexpr int kCols = 8, kStreams = S::kStreams;
    const int wi = (threadIdx.x >> 7) - 1, stream = wi % kStreams, grp = wi / kStreams, own = grp * kCols;
    constexpr int kAll = S::kSoftmax, kAllBar = kAll / 128 + 1;   // threads of the softmax, and their barrier
    const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, r = threadIdx.x & 127;
    const uint32_t quarter = tmem + ((uint32_t)(warp * 32) << 16);
    // its own S and O; with 64 dims the lower lanes of O hold the even tokens' dims, the upper the odd ones'
    const uint32_t s_at = quarter + stream * S::kBufs * S::kSBuf + own;
    const uint32_t o_half = S::kPair && warp >= 2 ? S::kNO : 0, o_at = quarter + S::kOCol + stream * S::kWRow + o_half + own;
    const int t_first = ranges.begin(blockIdx.x);
    uint32_t g = 0, uses = 0;                             // stages before this segment; this stream's tiles
    float l[kCols];
    for (uint32_t seg = 0; w.left > 0; ++seg, w.next(p)) {
      const uint32_t buf = seg & 1;
      bool ok = wait(&ctl->q_full[buf], (seg >> 1) & 1);
      // positions that every column attends to, and that any does
      const int at0 = ctl->at0[buf], at1 = ctl->at1[buf], all_lo = window_start(at1), any_lo = window_start(at0);
#pragma unroll
      for (int c = 0; c < kCols; ++c) l[c] = 0.f;
      bool stop = false;
      for (int i = stream; i < w.count; i += S::kStreams) {
        const uint32_t gt = g + i, st = gt % S::kStages, sb = uses % S::kBufs;
        const int t0 = (w.first + w.at + i) * S::kTile, t = t0 + S::kHalves * r;
        const int h = r / S::kPageRows;
        ok = ok && wait(&ctl->full[st], (gt / S::kStages) & 1);
        const uint32_t pages = ctl->pages_ok[st];
        const uint8_t* sc = reinterpret_cast<const uint8_t*>(&ctl->scales[st][h]) + (w.kvh & 1) * 8 + (t % kPageTokens) / kBlockTokens;
        const float ks = __uint_as_float((uint32_t)sc[0] << 23);
        const float ev = (float)((int)sc[4] - 127);
        ok = ok && wait(&ctl->s_full[stream][sb], (uses / S::kBufs) & 1);
        __syncwarp();
        tc_fence_after();
        // the positions that columns attend to end or begin in some tiles: most rows are in for all of
        // the columns or for none
        const bool whole = pages == (1u << S::kPages) - 1 && t0 + S::kTile - 1 <= at0 && t0 >= all_lo;
        const bool page_ok = (pages >> h) & 1;
        // exponents (log2 units) of the scores of a half's token; two columns an instruction here and below,
        // and four columns' parts at a time, as registers are short (eight: 182 us instead of 179, as below)
        auto scores = [&](int half, float (&z)[kCols]) {
#pragma unroll
          for (int k = 0; k < kCols; k += 4) {
            uint32_t part[kQParts][4];
#pragma unroll
            for (int q = 0; q < kQParts; ++q) tmem_ld4(s_at + sb * S::kSBuf + half * S::kNS + q * NC + k, part[q]);
            tmem_wait_ld();
            const float4 f = *reinterpret_cast<const float4*>(&ctl->f[buf][own + k]);
            const float2 fs[2] = {make_float2(f.x, f.y), make_float2(f.z, f.w)};
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              float2 s = pair_of(part[kQParts - 1], 2 * n);
#pragma unroll
              for (int q = kQParts - 2; q >= 0; --q) s = __ffma2_rn(s, make_float2(1.f / 16.f, 1.f / 16.f), pair_of(part[q], 2 * n));
              s = __fmul2_rn(s, __fmul2_rn(fs[n], make_float2(ks, ks)));
              z[k + 2 * n] = s.x;
              z[k + 2 * n + 1] = s.y;
            }
          }
          if (__builtin_expect(!whole, 0)) {
#pragma unroll
            for (int c = 0; c < kCols; ++c)
              if (!page_ok || t + half > ctl->hi[buf][own + c] || t + half < ctl->lo[buf][own + c]) z[c] = neg_inf();
          }
        };
        // and against the references: of the sum, and from there of the weights (scores may be so large that a
        // block's scale added to one would be rounded away)
        auto refs = [&](const float* top, int k, float2 (&r)[2]) {
          const float4 t = *reinterpret_cast<const float4*>(top + own + k);
          r[0] = make_float2(t.x, t.y);
          r[1] = make_float2(t.z, t.w);
        };
        auto less = [&](float2 z, float2 r) { return __ffma2_rn(r, make_float2(-1.f, -1.f), z); };
        // (z becomes the sum's; taking both from the scores again later, for fewer registers, took 182 us
        // instead of 179: 32 requests of 4-16K, four queries of 8 heads)
        float z[S::kHalves][kCols], zw[S::kHalves][kCols];
        auto against = [&](float (&zw)[kCols], float (&z)[kCols]) {
          float most_w = neg_inf(), most_s = neg_inf();
#pragma unroll
          for (int k = 0; k < kCols; k += 4) {
            float2 rw[2], rs[2];
            refs(ctl->top_w[stream], k, rw);
            refs(ctl->top_s[stream], k, rs);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const int c = k + 2 * n;
              const float2 x = make_float2(z[c], z[c + 1]);
              const float2 s = less(x, rs[n]), w = __fadd2_rn(s, less(make_float2(ev, ev), rw[n]));
              zw[c] = w.x;
              zw[c + 1] = w.y;
              z[c] = s.x;
              z[c + 1] = s.y;
              most_w = max3(most_w, w.x, w.y);
              most_s = max3(most_s, s.x, s.y);
            }
          }
          return most_w > kWeightScale + kHeadroom || most_s > kSumHeadroom;
        };
        bool raise = false;
#pragma unroll
        for (int half = 0; half < S::kHalves; ++half) {
          scores(half, z[half]);
          raise |= against(zw[half], z[half]);
        }
        if (__builtin_expect(!whole && ok && grp == 0, 0)) {
          for (int half = 0; half < S::kHalves; ++half) {
            const int at = t + half;
            const bool any = page_ok && at <= at1 && at >= any_lo, all = page_ok && at <= at0 && at >= all_lo;
            if (!all) clean_row(stages + st * S::kStageBytes + 1024 + (r >> 3) * 2048 + (r & 7) * 128, r, half, at, any, buf, stream);
          }
        }
        // the stream's weights before these have been read, and its O is at rest (those of earlier segments
        // are: a segment ends when all its products are complete, and the stages may have gone round since)
        if (i >= S::kStreams) ok = ok && product_done(gt - S::kStreams);
        __syncwarp();
        tc_fence_after();
        if (__builtin_expect(bar_any(1 + wi, 128, raise || !ok), 0)) {
          // rare after the first tiles: new references, the tile's own maxima where those are larger (the
          // scores are read again rather than kept in registers all the time)
          float top[kCols];
#pragma unroll
          for (int half = 0; half < S::kHalves; ++half) {
            scores(half, z[half]);
#pragma unroll
            for (int c = 0; c < kCols; ++c) top[c] = half == 0 ? z[0][c] : fmaxf(top[c], z[half][c]);
          }
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            const float ms = fmaxf(redux_max(top[c]), kNone), mw = redux_max(top[c] - ms + ev);
            if (lane == 0) *reinterpret_cast<float2*>(ctl->part_max[stream][warp][own + c]) = make_float2(ms, mw);
          }
          if (bar_any(1 + wi, 128, !ok)) {
            stop = true;
            break;
          }
          if (r < kCols) {
            const int c = own + r;
            const float w0 = ctl->top_w[stream][c], s0 = ctl->top_s[stream][c];
            float s1 = s0;
            for (int k = 0; k < 4; ++k) s1 = fmaxf(s1, ctl->part_max[stream][k][c][0]);
            float w1 = s0 - s1 + w0;
            for (int k = 0; k < 4; ++k) {
              const float2 most = *reinterpret_cast<const float2*>(ctl->part_max[stream][k][c]);
              w1 = fmaxf(w1, most.x - s1 + most.y - kWeightScale);
            }
            ctl->top_w[stream][c] = w1;
            ctl->top_s[stream][c] = s1;
            ctl->scale_o[stream][c] = ex2_approx(s0 - s1 + w0 - w1);
            ctl->scale_l[stream][c] = ratio(s0, s1);
          }
          bar_sync(1 + wi, 128);
#pragma unroll
          for (int c = 0; c < kCols; ++c) l[c] *= ctl->scale_l[stream][own + c];
#pragma unroll
          for (int half = 0; half < S::kHalves; ++half) against(zw[half], z[half]);
          if (i >= S::kStreams) {
            __syncwarp();
#pragma unroll 1
            for (int k = 0; k < kWParts; ++k) {
              uint32_t o[kCols];
              tmem_ld8(o_at + k * NC, o);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < kCols; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * ctl->scale_o[stream][own + c]);
              tmem_st8(o_at + k * NC, o);
            }
            tmem_wait_st();
          }
        }
        // weights, as parts, into the row of the B operand, whose 16-byte chunks are in swizzled order
        ++uses;
        uint8_t* wrow = wbuf + stream * S::kWBytes + r * S::kWRow;
        const int swizzle = S::kWRow == 128 ? r & 7 : (S::kWRow == 64 ? (r >> 1) & 3 : (r >> 2) & 1);
#pragma unroll
        for (int half = 0; half < S::kHalves; ++half) {
          uint32_t out[kWParts][2];
#pragma unroll
          for (int k = 0; k < kCols; k += 4) {
            float e[4];
#pragma unroll
            for (int n = 0; n < 4; n += 2) {
              const int c = k + n;
              e[n] = ex2_approx(zw[half][c]);
              e[n + 1] = ex2_approx(zw[half][c + 1]);
              const float2 sum = __fadd2_rn(make_float2(l[c], l[c + 1]), make_float2(ex2_approx(z[half][c]), ex2_approx(z[half][c + 1])));
              l[c] = sum.x;
              l[c + 1] = sum.y;
            }
            uint32_t p01[kWParts], p23[kWParts];
            split_weight(e[0], e[1], p01);
            split_weight(e[2], e[3], p23);
#pragma unroll
            for (int n = 0; n < kWParts; ++n) out[n][k / 4] = p01[n] | (p23[n] << 16);
          }
          if constexpr (NC == 8) {
            *reinterpret_cast<uint4*>(wrow + 16 * ((2 * half) ^ swizzle)) = make_uint4(out[0][0], out[0][1], out[1][0], out[1][1]);
            *reinterpret_cast<uint4*>(wrow + 16 * ((2 * half + 1) ^ swizzle)) = make_uint4(out[2][0], out[2][1], out[3][0], out[3][1]);
          } else {
#pragma unroll
            for (int n = 0; n < kWParts; ++n)
              *reinterpret_cast<uint2*>(wrow + 16 * ((4 * half + n) ^ swizzle) + 8 * grp) = make_uint2(out[n][0], out[n][1]);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->w_full[stream][sb]);
      }
      // ---- the segment's end: all streams, this warpgroup's share of the columns
      const int n = w.count;
      if (!stop) {
#pragma unroll
        for (int k = 0; k < kStreams; ++k) {
          if (n > k) ok = ok && product_done(g + k + (n - 1 - k) / kStreams * kStreams);   // the stream's last stage
        }
        __syncwarp();
        tc_fence_after();
        // sums over the warp's tokens: halves of the columns go to halves of the lanes, until a lane has one
#pragma unroll
        for (int step = 0; step < 5; ++step) {
          const int part = kCols >> (step + 1), d = 16 >> step;
#pragma unroll
          for (int c = 0; c < part; ++c) {
            const bool up = (lane & d) != 0;
            const float give = up ? l[c] : l[c + part], keep = up ? l[c + part] : l[c];
            l[c] = keep + __shfl_xor_sync(kFull, give, d);
          }
          if (part == 0) l[0] += __shfl_xor_sync(kFull, l[0], d);
        }
        // the lane's highest bits say which column: bit 4 halves them, bit 3 quarters, ...
        if (lane % (32 / kCols) == 0) ctl->part_l[stream][warp][own + lane / (32 / kCols)] = l[0];
      }
      if (bar_any(kAllBar, kAll, stop || !ok)) {
        // gave up: the counts of the units that this CTA shares still come out even
        if (wi == 0 && r == 0)
          for (; w.left > 0; w.next(p))
            if (!w.whole()) arrive(ranges.of(w.pos + kUnitCost), ranges.of(w.pos + kUnitCost + w.n - 1));
        return;
      }
      g += n;
      constexpr int kN = NC / (kAll / 128);               // columns whose streams this warpgroup adds
      const int c0 = wi * kN;
      if (r < kN) {
        const int c = c0 + r;
        float m = kNone, sum = 0.f;
#pragma unroll
        for (int k = 0; k < kStreams; ++k) m = fmaxf(m, ctl->top_s[k][c]);
#pragma unroll
        for (int k = 0; k < kStreams; ++k) {
          float part = 0.f;
          for (int q = 0; q < 4; ++q) part += ctl->part_l[k][q][c];
          sum += part * ratio(ctl->top_s[k][c], m);
        }
        // What O is multiplied by makes it the weighted mean at once, which fp32 holds wherever it holds the
        // values (m may lie 2^60 below the largest weight, so that the weighted sum need not fit). It is
        // taken in two factors beside 1 / (the sum's 1 to 2), which stay far from fp32's ends.
        const int up = max(0, min(126, (int)((__float_as_uint(sum) >> 23) & 0xFFu) - 127));
        const float inv = inverse(sum * __uint_as_float((uint32_t)(127 - up) << 23));
#pragma unroll
        for (int k = 0; k < kStreams; ++k) {
          const float half = ex2_approx(0.5f * (ctl->top_s[k][c] - m + ctl->top_w[k][c] - (float)up));
          *reinterpret_cast<float2*>(ctl->join_w[k][c]) = make_float2(half * inv, half);
        }
        ctl->join_m[c] = m;
        ctl->join_l[c] = sum;
        if (w.whole()) put_lse(ctl->row[buf][c], m, sum);
      }
      bar_sync(1 + wi, 128);
      __syncwarp();
      int d = S::kPair ? r & 63 : r;
      const bool full_unit = w.whole();
      const int slot = 2 * (int)blockIdx.x + second_slot(t_first, w.pos);
      bool poisoned = false;
#pragma unroll
      for (int k = 0; k < kStreams; ++k) poisoned |= ctl->any_poison[k] != 0;
      float acc[kN] = {};
      // kept as a loop, as code that runs once costs what its fetching costs
#pragma unroll 1
      for (int k = 0; k < min(kStreams, n); ++k) {
        uint32_t o[kWParts][kN];
#pragma unroll
        for (int q = 0; q < kWParts; ++q) {
          tmem_ld4(quarter + S::kOCol + k * S::kWRow + o_half + q * NC + c0, o[q]);
        }
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < kN; ++c) {
          float x = __uint_as_float(o[3][c]);
          x = fmaf(x, 1.f / 16.f, __uint_as_float(o[2][c]));
          x = fmaf(x, 1.f / 16.f, __uint_as_float(o[1][c]));
          x = fmaf(x, 1.f / 16.f, __uint_as_float(o[0][c]));
          if (poisoned && ((ctl->poison[k][c0 + c][d >> 5] >> (d & 31)) & 1)) x = __int_as_float(0x7fc00000);
          const float2 f = *reinterpret_cast<const float2*>(ctl->join_w[k][c0 + c]);
          acc[c] = fmaf(x * f.x, f.y, acc[c]);
        }
      }
      if constexpr (S::kPair) {
        // the odd tokens' sums to the threads of the even ones', through the weights' memory, which is free
        float* other = reinterpret_cast<float*>(wbuf) + (wi * 64 + d) * kN;
        if (r >= 64) {
#pragma unroll
          for (int c = 0; c < kN; ++c) other[c] = acc[c];
        }
        bar_sync(1 + wi, 128);
        if (r < 64) {
#pragma unroll
          for (int c = 0; c < kN; ++c) acc[c] += other[c];
        } else {
          d = -1;
        }
      }
      if (full_unit) {
#pragma unroll
        for (int c = 0; c < kN; ++c)
          if (d >= 0 && ctl->row[buf][c0 + c] >= 0) put<kHalf>((int64_t)ctl->row[buf][c0 + c] * D + d, acc[c]);
      } else {
#pragma unroll
        for (int c = 0; c < kN; ++c)
          if (d >= 0) p.part_o[(int64_t)(slot * NC + c0 + c) * D + d] = acc[c];
        if (r < kN) reinterpret_cast<float2*>(p.part_ml)[slot * NC + c0 + r] = make_float2(ctl->join_m[c0 + r], ctl->join_l[c0 + r]);
        const int base = w.pos + kUnitCost, c_lo = ranges.of(base), c_hi = ranges.of(base + w.n - 1);
        bar_sync(kAllBar, kAll);
        if (wi == 0 && r == 0) ctl->last = arrive(c_lo, c_hi) ? 1 : 0;
        bar_sync(kAllBar, kAll);
        if (ctl->last && d >= 0) join<kHalf>(ctl->row[buf], c0, d, c_lo, c_hi, second_slot(ranges.begin(c_lo), w.pos));
      }
      // the next segment starts from nothing
      bar_sync(kAllBar, kAll);
      if (r < kCols) {
        ctl->top_w[stream][own + r] = 0.f;
        ctl->top_s[stream][own + r] = kNone;
      }
      // (a stream's notes of NaN, of all columns, by the warpgroup that makes them: no barrier of both its
      // warpgroups comes before the next segment's first)
      if (poisoned && grp == 0 && r < NC)
        for (int k = 0; k < 4; ++k) ctl->poison[stream][r][k] = 0;
      if (r == 0 && grp == 0) ctl->any_poison[stream] = 0;
      bar_sync(1 + wi, 128);
      if (lane == 0) mbar_arrive(&ctl->q_empty[buf]);
    }
  }
};

template <int D, int NC, bool kHalf>
__global__ void __launch_bounds__(Shape<D, NC, kHalf ? 3 : 2>::kThreads, 1) kv8_decode_kernel(const __grid_constant__ Kv8DecodeParams p) {
  using S = Shape<D, NC, kHalf ? 3 : 2>;
  using Ctl = Control<NC, S::kStages, S::kPages, S::kStreams, S::kThreads / 32>;
  static_assert(offsetof(Ctl, scales) % 16 == 0 && offsetof(Ctl, f) % 16 == 0 && offsetof(Ctl, top_w) % 16 == 0 &&
                offsetof(Ctl, top_s) % 16 == 0 && offsetof(Ctl, part_max) % 8 == 0 && offsetof(Ctl, join_w) % 8 == 0 && NC % 8 == 0, "vector accesses are aligned");
  static_assert(sizeof(Ctl) <= 6144, "the control block fits its share");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stages = base;
  uint8_t* qbuf = stages + S::kStages * S::kStageBytes;
  uint8_t* wbuf = qbuf + 2 * S::kQBytes;
  Ctl* ctl = reinterpret_cast<Ctl*>(wbuf + S::kStreams * S::kWBytes);
  constexpr int kThreads = S::kThreads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 64) {
    prefetch_tensormap(&p.cache_map);
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&ctl->full[i], 1 + S::kPages);       // the codes' bytes, every page's scale bytes
      mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->q_full[i], 1);
      mbar_init(&ctl->q_empty[i], 1 + S::kSoftmax / 32);           // the issuer of S and the softmax warps
      mbar_init(&ctl->drain[i], 1);
    }
    for (int i = 0; i < S::kStreams; ++i) {
      for (int k = 0; k < 2; ++k) {
        mbar_init(&ctl->s_full[i][k], 1);
        mbar_init(&ctl->w_full[i][k], 4 * S::kGroups);
      }
      ctl->any_poison[i] = 0;
    }
    ctl->abort = 0;
    fence_barrier_init();
  }
  for (int i = tid; i < S::kStreams * NC; i += kThreads) {
    ctl->top_w[i / NC][i % NC] = 0.f;
    ctl->top_s[i / NC][i % NC] = kNone;
    for (int k = 0; k < 4; ++k) ctl->poison[i / NC][i % NC][k] = 0;
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, S::kTmem);
    tmem_relinquish();
  }

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the whole sequence: every thread sums a run of requests
  const int cts = (p.Q * p.group + NC - 1) / NC;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  int sum = 0;
  for (int b = b0; b < b1; ++b) {
    int first, n;
    unit_tiles<S::kTile>(p, max(0, p.seq_lens[b]), first, n);
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
  const int of_warp = lane < kThreads / 32 ? ctl->scan_sum[lane] : 0;
  const int before = (__reduce_add_sync(kFull, lane < warp ? of_warp : 0) + incl - sum) * p.kv_heads;
  const int all = __reduce_add_sync(kFull, of_warp) * p.kv_heads;      // of one column tile
  // no more CTAs than leave each a tile for each of its streams on average, and where units have few tiles, no
  // more than units: joining partial results costs some 4 us, a tile 0.6 (one request of 1,000 tokens: 10.6
  // us, and 12.7 when its eight units are split). Ranges divide positions, of which a unit's first kUnitCost
  // are no tiles, so where few CTAs share one unit the first may have no tile and the others more than that
  // average: of 16 tiles of one unit, cut in eight, two have none, one has one, and five have three.
  const int units = p.B * p.kv_heads * cts, tiles = all * cts - kUnitCost * units;
  // Where a unit would be cut into very many, a part less saves more of the joining (some 0.1 us each) than
  // it adds to the others' tiles: of t tiles, 2 sqrt(t) parts at most (one request, one key/value head of 8
  // query heads: 16K tokens 15 us, 32K 15; with the join as it was then 16.5 and 17.3 instead of 22 and 31;
  // with sqrt(t) parts 16.0 and 18.5, but 2K tokens 12.9 instead of 11.9)
  const int parts = (int)ceilf(2.f * sqrtf((float)tiles / (float)units)), grid = (int)gridDim.x;
  const int most = tiles <= S::kFewTiles * units ? units
                                                 : min((tiles + S::kMinTiles - 1) / S::kMinTiles, min(units, grid) * min(parts, grid));
  const Ranges ranges(all * cts, min(grid, most));
  const int cta = blockIdx.x;
  const int t_begin = ranges.begin(cta), t_end = cta < ranges.ctas ? ranges.begin(cta + 1) : t_begin;
  const int ct = t_begin / all, in_ct = t_begin - ct * all;
  if (t_begin < t_end && before <= in_ct && in_ct < before + sum * p.kv_heads) {
    int b = b0, at = before;
    for (;; ++b) {
      int first, n;
      unit_tiles<S::kTile>(p, max(0, p.seq_lens[b]), first, n);
      if (in_ct < at + (n + kUnitCost) * p.kv_heads) break;
      at += (n + kUnitCost) * p.kv_heads;
    }
    ctl->start_b = b;
    ctl->start_before = at;
  }
  __syncthreads();
  Walk<S::kTile> w{};
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
    Cta<D, NC, kHalf ? 3 : 2> c{p, stages, qbuf, wbuf, ctl};
    if (warp == 0) {
      c.producer(w);
    } else if (warp == 1) {
      if (lane == 0) c.issue_s(w, tmem);
      __syncwarp();
    } else if (warp == 2) {
      c.template queries<kHalf>(w);
    } else if (warp == 3) {
      if (lane == 0) c.issue_o(w, tmem);
      __syncwarp();
    } else {
      c.template softmax<kHalf>(w, tmem, ranges);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(ctl->tmem_base, S::kTmem);
  }
}

template <class S, int NC>
constexpr size_t smem_bytes() {
  return 1024 + (size_t)S::kStages * S::kStageBytes + 2 * S::kQBytes + S::kStreams * S::kWBytes +
         sizeof(Control<NC, S::kStages, S::kPages, S::kStreams, S::kThreads / 32>);
}

template <int D, int NC, bool kHalf>
cudaError_t launch(const Kv8DecodeParams& p, cudaStream_t stream) {
  using S = Shape<D, NC, kHalf ? 3 : 2>;
  constexpr size_t smem = smem_bytes<S, NC>();
  static_assert(smem <= 232448, "exceeds the 227 KB shared-memory limit");
  static std::mutex mu;
  static bool allowed[64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 64 || !allowed[dev]) {
      err = cudaFuncSetAttribute(kv8_decode_kernel<D, NC, kHalf>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (err != cudaSuccess) return err;
      if (dev < 64) allowed[dev] = true;
    }
  }
  // A dependent launch: a CTA sets itself up while the grid before it in the stream ends, and waits for
  // all of that grid before it reads or writes memory.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.ctas, 1, 1);
  cfg.blockDim = dim3(S::kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_decode_kernel<D, NC, kHalf>, p);
}

template <int D, bool kHalf>
cudaError_t launch_columns(const Kv8DecodeParams& p, cudaStream_t stream) {
  if (kv8_decode_columns(p.Q, p.group) == 8) return launch<D, 8, kHalf>(p, stream);
  return launch<D, 16, kHalf>(p, stream);
}

}  // namespace

// Columns of a tile. 8 where they hold all of a key/value head's: with 16 such steps took 219 us instead
// of 210 (16 requests of 20-90K tokens, 128 dims) and 187 instead of 151 (64 of 4-30K, 64 dims), as the
// softmax's work grows with them. From 9 columns on 16: two tiles of 8 would read every key twice and
// take as many instructions. (32 columns in one tile spilled registers, and took 82 ns a column and
// tile where 16 took 62.)
int kv8_decode_columns(int Q, int group) {
  return Q * group <= 8 ? 8 : 16;
}

cudaError_t launch_kv8_decode(const Kv8DecodeParams& p, int head_dim, bool fp16, cudaStream_t stream) {
  if (head_dim == 128) return fp16 ? launch_columns<128, true>(p, stream) : launch_columns<128, false>(p, stream);
  return fp16 ? launch_columns<64, true>(p, stream) : launch_columns<64, false>(p, stream);
}

}  // namespace nvfp4mla
