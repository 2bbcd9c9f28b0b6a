// Page operators: copy, free, trim, fork, extend and compact the pages of a paged cache.
//
// The tables are small and the pages large, so each call is a planning kernel over the counts and
// tables and, where pages move, a copy grid over their bytes that follows it as a dependent launch.
//
// Planning is one thread-block cluster of eight CTAs. The lowest-numbered free pages are found by
// two passes over the counts, cut into eight pieces: every CTA counts the free pages of its piece,
// the counts are exchanged through distributed shared memory, and the second pass (from cache)
// numbers the free pages from there. The page with number g goes to the request whose range of the
// needs' running sum holds g, so the result does not depend on the order in which threads run.
//
// Copies are bound by memory, planning by the latency of a few dependent passes and exchanges (1.5 us
// each; one CTA alone took 22 us for a plan that eight take 17 for, and 10 since moves are left to the
// copy grid). Measured (device time): 3,001 pages of 131 KB 787 MB in 117 us, 99 % of the measured copy
// bandwidth; compaction of 40,000 pages of 22.5 KB, 9,600 of which move: 85 us, of which the copy's 432 MB
// 70; free, fork and extend of 64 sequences over 4,096 pages together 16 us.
#include <climits>
#include <mutex>

#include "../../include/nvfp4mla.h"
#include "kv8.h"
#include "ptx.cuh"

namespace nvfp4mla {
namespace {

using namespace ptx;

constexpr int kPlanCtas = 8;           // one portable cluster
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kCopyThreads = 256;
constexpr int kChunkBytes = 16384;     // of a page that a copy block moves: four 16-byte loads a thread, all in flight
constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ void count_bad(int32_t* status, int word, int n = 1) {
  if (status != nullptr) atomicAdd(status + word, n);
}
__device__ __forceinline__ void wait_for_planner() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_dependents_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// One chunk of one page, 16 bytes a load; page_bytes is a multiple of 16.
__device__ __forceinline__ void copy_chunk(const PageStore& c, int64_t layer, int64_t from, int64_t to, int64_t chunk) {
  const uint8_t* src = c.base + layer * c.layer_stride + from * c.page_bytes;
  uint8_t* dst = c.base + layer * c.layer_stride + to * c.page_bytes;
  constexpr int kLoads = kChunkBytes / (16 * kCopyThreads);
  const int64_t at = chunk * kChunkBytes + (int64_t)threadIdx.x * 16;
  uint4 v[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i)
    if (at + i * kCopyThreads * 16 < c.page_bytes) v[i] = *reinterpret_cast<const uint4*>(src + at + i * kCopyThreads * 16);
#pragma unroll
  for (int i = 0; i < kLoads; ++i)
    if (at + i * kCopyThreads * 16 < c.page_bytes) *reinterpret_cast<uint4*>(dst + at + i * kCopyThreads * 16) = v[i];
}
__host__ __device__ __forceinline__ int64_t chunks_of(const PageStore& c) { return (c.page_bytes + kChunkBytes - 1) / kChunkBytes; }

// ------------------------------------------------------------------ copy
__global__ void __launch_bounds__(kCopyThreads)
copy_kernel(const PageStore c, int64_t num_pages, const int32_t* src, const int32_t* dst, int32_t* status) {
  const int64_t chunks = chunks_of(c), per = chunks * c.layers;
  const int64_t i = blockIdx.x / per, rest = blockIdx.x % per;
  const int64_t from = src[i], to = dst[i];
  if (from == -1 || to == -1) return;
  if (from < 0 || from >= num_pages || to < 0 || to >= num_pages) {
    if (rest == 0 && threadIdx.x == 0) count_bad(status, NVFP4MLA_STAT_BAD_PAGE);
    return;
  }
  if (from != to) copy_chunk(c, rest / chunks, from, to, rest % chunks);
}

// ------------------------------------------------------------------ free
// Entries are taken out of the row by an exchange, so that a sequence listed twice gives each page
// up once whichever of its blocks comes first.
__global__ void __launch_bounds__(256) free_kernel(const PageState s, const int32_t* seqs) {
  const int seq = seqs[blockIdx.x];
  if (seq == -1) return;
  if (seq < 0 || seq >= s.num_seqs) {
    if (blockIdx.y == 0 && threadIdx.x == 0) count_bad(s.status, NVFP4MLA_STAT_BAD_SLOT);
    return;
  }
  int32_t* row = s.table + (int64_t)seq * s.max_pages;
  if (blockIdx.y == 0 && threadIdx.x == 0) s.lens[seq] = 0;
  for (int64_t i = (int64_t)blockIdx.y * 256 + threadIdx.x; i < s.max_pages; i += (int64_t)gridDim.y * 256) {
    if (row[i] == -1) continue;
    const int32_t page = atomicExch(row + i, -1);
    if (page == -1) continue;
    if (page < 0 || page >= s.num_pages) {
      count_bad(s.status, NVFP4MLA_STAT_BAD_PAGE);
    } else if (atomicSub(s.refs + page, 1) <= 0) {
      atomicAdd(s.refs + page, 1);
      count_bad(s.status, NVFP4MLA_STAT_BAD_PAGE);
    }
  }
}

// ------------------------------------------------------------------ trim
// A warp a sequence, an entry a lane: a chain of two reads and an atomic, some 3 us of a step's end.
__global__ void __launch_bounds__(32) trim_kernel(const PageState s, const int32_t* new_lens) {
  const int seq = blockIdx.x;
  const int len = s.lens[seq], now = new_lens[seq];
  if (now < 0 || now > len) {
    if (threadIdx.x == 0) count_bad(s.status, NVFP4MLA_STAT_BAD_SLOT);
    return;
  }
  if (now == len) return;
  __syncwarp();                        // (new_lens may be lens itself)
  if (threadIdx.x == 0) s.lens[seq] = now;
  int32_t* row = s.table + (int64_t)seq * s.max_pages;
  const int64_t end = min(((int64_t)len + kPageTokens - 1) / kPageTokens, s.max_pages);
  for (int64_t i = ((int64_t)now + kPageTokens - 1) / kPageTokens + threadIdx.x; i < end; i += 32) {
    const int32_t page = row[i];
    row[i] = -1;
    if (page < 0 || page >= s.num_pages) {
      count_bad(s.status, NVFP4MLA_STAT_BAD_PAGE);
    } else if (atomicSub(s.refs + page, 1) <= 0) {
      atomicAdd(s.refs + page, 1);
      count_bad(s.status, NVFP4MLA_STAT_BAD_PAGE);
    }
  }
}

// ------------------------------------------------------------------ planning
struct PlanShared {
  int2 piece[2];               // this CTA's counts, by exchange, read by the others
  int4 sums;                   // of an exchange: before, all; of the first count and of the second
  int warp[kPlanWarps];
  int2 warp2[kPlanWarps];
  int64_t running;
};

// Exclusive prefix over the block's warps of a per-warp value, which is not negative (32 of which may leave 32 bits).
__device__ int64_t warp_prefix(PlanShared* sh, int v) {
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh->warp[threadIdx.x >> 5] = v;
  __syncthreads();
  const int w = (int)(threadIdx.x & 31) < (int)(threadIdx.x >> 5) ? sh->warp[threadIdx.x & 31] : 0;
  return ((int64_t)__reduce_add_sync(kFull, w >> 16) << 16) + __reduce_add_sync(kFull, w & 0xFFFF);
}

// Two counts of every warp of the cluster: their sums over the warps before this one (of this and of
// earlier CTAs) and over all. A warp of each CTA reads the others' sums; round: 0 and 1 in turn. Global
// writes of the cluster before it are visible after it.
struct Counts {
  int before, all;
};
__device__ void exchange(PlanShared* sh, int round, int2 mine, Counts& first, Counts& second) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) sh->warp2[warp] = mine;
  __syncthreads();
  const int2 w = sh->warp2[lane];
  if (warp == 0) {
    const int2 sum = make_int2(__reduce_add_sync(kFull, w.x), __reduce_add_sync(kFull, w.y));
    if (lane == 0) sh->piece[round] = sum;
  }
  cluster_sync_all();
  if (warp == 0) {
    const int rank = (int)cluster_ctarank();
    int2 v = make_int2(0, 0);
    if (lane < kPlanCtas) {
      const uint32_t at = map_shared_rank(smem_u32(&sh->piece[round]), (uint32_t)lane);
      v = make_int2((int)ld_dsmem_u32(at), (int)ld_dsmem_u32(at + 4));
    }
    const int4 sums = make_int4(__reduce_add_sync(kFull, lane < rank ? v.x : 0), __reduce_add_sync(kFull, v.x),
                                __reduce_add_sync(kFull, lane < rank ? v.y : 0), __reduce_add_sync(kFull, v.y));
    if (lane == 0) sh->sums = sums;
  }
  __syncthreads();
  const int4 sums = sh->sums;
  first = {sums.x + __reduce_add_sync(kFull, lane < warp ? w.x : 0), sums.y};
  second = {sums.z + __reduce_add_sync(kFull, lane < warp ? w.y : 0), sums.w};
}

// This CTA's piece of n items, and within it this warp's: multiples of 128, so that a lane's four
// are one 16-byte load (refcounts are 16-byte aligned).
__device__ __forceinline__ void piece_of(int64_t n, int64_t& lo, int64_t& hi) {
  constexpr int kAll = kPlanCtas * kPlanWarps * 128;
  const int64_t per_warp = (n + kAll - 1) / kAll * 128;
  const int64_t w = (int64_t)cluster_ctarank() * kPlanWarps + (threadIdx.x >> 5);
  lo = w * per_warp < n ? w * per_warp : n;
  hi = lo + per_warp < n ? lo + per_warp : n;
}

// The four counts at i (items behind n read as `fill`).
__device__ __forceinline__ int4 four_at(const int32_t* a, int64_t i, int64_t n, int fill) {
  if (i + 3 < n) return *reinterpret_cast<const int4*>(a + i);
  return make_int4(i < n ? a[i] : fill, i + 1 < n ? a[i + 1] : fill, i + 2 < n ? a[i + 2] : fill, fill);
}

// Items of [lo, hi) that `is` holds for, over the warp, in every lane.
template <class F>
__device__ int warp_count(const int32_t* a, int64_t lo, int64_t hi, int64_t n, int fill, F is) {
  const int lane = threadIdx.x & 31;
  int c = 0;
#pragma unroll 4
  for (int64_t i = lo; i < hi; i += 128) {
    const int4 v = four_at(a, i + lane * 4, n, fill);
    c += is(i + lane * 4, v.x) + is(i + lane * 4 + 1, v.y) + is(i + lane * 4 + 2, v.z) + is(i + lane * 4 + 3, v.w);
  }
  return __reduce_add_sync(kFull, c);
}

// do_(item, value, number) for every item of [lo, hi) that `is` holds for, numbered from `from`.
template <class F, class G>
__device__ void warp_number(const int32_t* a, int64_t lo, int64_t hi, int64_t n, int fill, int64_t from, int64_t stop, F is, G do_) {
  const int lane = threadIdx.x & 31;
  for (int64_t i = lo; i < hi && from < stop; i += 128) {
    const int64_t at = i + lane * 4;
    const int4 v = four_at(a, at, n, fill);
    const int vs[4] = {v.x, v.y, v.z, v.w};
    int c = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) c += is(at + k, vs[k]) ? 1 : 0;
    int before = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(kFull, before, d);
      if (lane >= d) before += o;
    }
    const int total = __shfl_sync(kFull, before, 31);
    int64_t g = from + before - c;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (is(at + k, vs[k])) do_(at + k, vs[k], g++);
    from += total;
  }
}

// Running sums of the needs: sum[i] = those of the requests before i, sum[n] = all. (A need is at most the pages
// of 2^31 tokens, 2^25, so a warp's sum is one of 32 bits.)
template <class F>
__device__ int64_t sum_needs(PlanShared* sh, int32_t* sum, int n, F need) {
  if (threadIdx.x == 0) sh->running = 0;
  __syncthreads();
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    const int c = i < n ? need(i) : 0;
    const int lane = threadIdx.x & 31;
    int incl = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(kFull, incl, d);
      if (lane >= d) incl += o;
    }
    const int64_t run = sh->running;
    const int64_t ahead = run + warp_prefix(sh, __shfl_sync(kFull, incl, 31));
    // a sum that leaves 32 bits stays at the top: there are fewer pages than that
    const int64_t mine = ahead + incl - c;
    if (i < n) sum[i] = (int32_t)(mine < INT_MAX ? mine : INT_MAX);
    __syncthreads();
    if (threadIdx.x == kPlanThreads - 1) sh->running = ahead + incl;
    __syncthreads();
  }
  const int64_t all = sh->running;
  if (threadIdx.x == 0) sum[n] = (int32_t)(all < INT_MAX ? all : INT_MAX);
  __syncthreads();
  return all;
}

// The request that the page with number g is for: the last whose running sum is at most g.
__device__ __forceinline__ int owner_of(const int32_t* sum, int n, int64_t g) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sum[mid] <= g) lo = mid;
    else hi = mid;
  }
  return lo;
}

struct IsFree {
  __device__ bool operator()(int64_t, int v) const { return v == 0; }
};

// ------------------------------------------------------------------ fork
// A claim on an empty sequence is kept where its length stands until the plan is done: INT_MIN + i,
// so that the smallest i wins. Lengths that callers hold are not that small.
constexpr int kClaim = INT_MIN;

struct ForkArgs {
  PageState s;
  PageStore c;
  const int32_t* src;
  const int32_t* dst;
  int n;
  int32_t* new_pages;
};

__device__ __forceinline__ bool is_claim(int len) { return len < kClaim + NVFP4MLA_MAX_REQUESTS; }

// The length that pair i would copy, or -1 when the pair is bad in itself.
__device__ int fork_length(const ForkArgs& a, int i, bool& missing) {
  const int src = a.src[i], dst = a.dst[i];
  missing = false;
  if (src < 0 || src >= a.s.num_seqs || dst < 0 || dst >= a.s.num_seqs || src == dst) return -1;
  int len = __ldcg(a.s.lens + src);
  if (is_claim(len)) len = 0;      // an empty source that is some pair's target
  if (len < 0 || (len + (int64_t)kPageTokens - 1) / kPageTokens > a.s.max_pages) return -1;
  if (len % kPageTokens != 0) {
    const int page = a.s.table[(int64_t)src * a.s.max_pages + len / kPageTokens];
    if (page < 0 || page >= a.s.num_pages) {
      missing = true;
      return -1;
    }
  }
  return len;
}

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads) fork_plan_kernel(const ForkArgs a) {
  extern __shared__ int32_t sum[];   // [n + 1], then per pair the length that it copies, -1: none
  __shared__ PlanShared sh;
  int32_t* copies = sum + a.n + 1;   // (each is only its own thread's, pair i's thread i mod kPlanThreads)
  let_dependents_start();
  const int rank = (int)cluster_ctarank();
  const auto owns = [=](int i) { return i / kPlanThreads % kPlanCtas == rank; };
  // claims: every CTA makes all of them, as it needs the lengths, and once is as good as eight times
  for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
    bool missing;
    const int len = fork_length(a, i, missing);
    copies[i] = len;
    if (len < 0) {
      if (owns(i)) count_bad(a.s.status, missing ? NVFP4MLA_STAT_BAD_PAGE : NVFP4MLA_STAT_BAD_SLOT);
      continue;
    }
    int32_t* at = a.s.lens + a.dst[i];
    const int there = __ldcg(at);
    if (there == 0 || is_claim(there)) atomicMin(at, kClaim + i);
  }
  cluster_sync_all();   // every claim is made
  // who won, and what that needs
  const int64_t total = sum_needs(&sh, sum, a.n, [&](int i) {
    const int len = copies[i];
    if (len < 0 || __ldcg(a.s.lens + a.dst[i]) != kClaim + i) {
      copies[i] = -1;
      return 0;
    }
    return len % kPageTokens != 0 ? 1 : 0;
  });
  int64_t lo, hi;
  piece_of(a.s.num_pages, lo, hi);
  Counts free_pages, unused;
  exchange(&sh, 0, make_int2(warp_count(a.s.refs, lo, hi, a.s.num_pages, 1, IsFree()), 0), free_pages, unused);
  const int64_t all = free_pages.all;
  // (every CTA has read the lengths: they may change)
  for (int i = rank * kPlanThreads + threadIdx.x; i < a.n; i += kPlanCtas * kPlanThreads) {
    const int len = copies[i];
    const bool needs = sum[i + 1] > sum[i], refused = needs && sum[i] >= all;
    if (len >= 0) a.s.lens[a.dst[i]] = refused ? 0 : len;
    if (len < 0 || refused) a.new_pages[i] = -2;
    else if (!needs) a.new_pages[i] = -1;
  }
  warp_number(a.s.refs, lo, hi, a.s.num_pages, 1, free_pages.before, total, IsFree(), [&](int64_t page, int, int64_t g) {
    if (g >= total) return;
    a.s.refs[page] = 1;
    a.new_pages[owner_of(sum, a.n, g)] = (int32_t)page;
  });
  cluster_sync_all();   // no CTA leaves while another may read its count
}

// Blocks (pair, chunk of a layer's page) move the part-full pages; the last blocks of a pair write
// its row and count the shared pages.
constexpr int kRowEntries = 1024;      // of a row that a block takes

__global__ void __launch_bounds__(kCopyThreads) fork_apply_kernel(const ForkArgs a) {
  wait_for_planner();
  const int64_t chunks = chunks_of(a.c), copies = chunks * a.c.layers;
  const int64_t per = copies + (a.s.max_pages + kRowEntries - 1) / kRowEntries;
  const int64_t i = blockIdx.x / per, part = blockIdx.x % per;
  const int fresh = a.new_pages[i];
  if (fresh == -2) return;
  const int src = a.src[i], dst = a.dst[i];
  const int64_t full = a.s.lens[dst] / kPageTokens;
  const int32_t* from = a.s.table + (int64_t)src * a.s.max_pages;
  if (part < copies) {
    if (fresh >= 0) copy_chunk(a.c, part / chunks, from[full], fresh, part % chunks);
    return;
  }
  int32_t* to = a.s.table + (int64_t)dst * a.s.max_pages;
  const int64_t lo = (part - copies) * kRowEntries;
  for (int64_t k = lo + threadIdx.x; k < lo + kRowEntries && k < a.s.max_pages; k += kCopyThreads) {
    int32_t page = -1;
    if (k < full) {
      page = from[k];
      if (page < 0 || page >= a.s.num_pages) {
        page = -1;
        count_bad(a.s.status, NVFP4MLA_STAT_BAD_PAGE);
      } else {
        atomicAdd(a.s.refs + page, 1);
      }
    } else if (k == full && fresh >= 0) {
      page = fresh;
    }
    to[k] = page;
  }
}

// ------------------------------------------------------------------ extend
struct ExtendArgs {
  PageState s;
  const int32_t* add;
  int32_t* granted;
};

// Pages that sequence i lacks for its new length, or -1 when it cannot grow (bad: to be counted).
__device__ int64_t extend_need(const ExtendArgs& a, int i, int64_t& have, bool& bad) {
  const int64_t len = __ldcg(a.s.lens + i), add = a.add[i];
  have = (len + kPageTokens - 1) / kPageTokens;
  const int64_t want = (len + add + kPageTokens - 1) / kPageTokens;
  bad = len < 0 || add < 0 || (add > 0 && want > a.s.max_pages) || len + add > INT_MAX;
  return bad ? -1 : (want > have ? want - have : 0);
}

// When there are fewer pages than needs: the sequences in order, each granted if its need fits what those before
// it left, else passed over. sum[i] = the pages granted before sequence i; returns all that are granted. One warp,
// 32 sequences at a time: those whose need alone is too large are passed over at once, and the first whose
// running sum is too large where that happens; until no page is left. (Every CTA does the same; the others of its
// warps wait. 16,384 sequences that all ask, 3,581 of them granted before 16,384 pages run out: 76 us for the call,
// where all fit 36; 64 of them 15 and 11.)
__device__ int64_t settle(const ExtendArgs& a, PlanShared* sh, int32_t* sum, int n, int64_t free_pages) {
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    int64_t have;
    bool bad;
    const int64_t need = extend_need(a, i, have, bad);
    sum[i] = (int32_t)(need > 0 ? need : 0);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int64_t given = 0;
    int base = 0;
    for (; base < n && given < free_pages; base += 32) {
      const int need = base + lane < n ? sum[base + lane] : 0;
      int64_t left = free_pages - given;
      unsigned open = __ballot_sync(kFull, need > 0), granted = 0;
      while (open != 0) {
        open &= __ballot_sync(kFull, need <= left);
        const int mine = (open >> lane) & 1 ? need : 0;
        int incl = mine;                   // (32 needs of at most 2^25)
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(kFull, incl, d);
          if (lane >= d) incl += o;
        }
        const unsigned over = __ballot_sync(kFull, incl > left) & open;
        const int stop = over != 0 ? __ffs(over) - 1 : 32;             // passed over, those before it granted
        const unsigned now = over != 0 ? open & ((1u << stop) - 1) : open;
        left -= __reduce_add_sync(kFull, (now >> lane) & 1 ? need : 0);
        granted |= now;
        open = over != 0 ? open & ~((2u << stop) - 1) : 0u;
      }
      const int mine = (granted >> lane) & 1 ? need : 0;
      int incl = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kFull, incl, d);
        if (lane >= d) incl += o;
      }
      if (base + lane < n) sum[base + lane] = (int32_t)(given + incl - mine);
      given = free_pages - left;
    }
    if (lane == 0) {
      sh->running = given;
      sh->warp[0] = base;
    }
  }
  __syncthreads();
  const int64_t given = sh->running;
  for (int i = min(n, sh->warp[0]) + threadIdx.x; i <= n; i += kPlanThreads) sum[i] = (int32_t)given;   // nothing is left for these
  __syncthreads();
  return given;
}

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads) extend_kernel(const ExtendArgs a) {
  extern __shared__ int32_t sum[];   // [num_seqs + 1]
  __shared__ PlanShared sh;
  const int rank = (int)cluster_ctarank();
  const int n = a.s.num_seqs;
  int64_t total = sum_needs(&sh, sum, n, [&](int i) {
    int64_t have;
    bool bad;
    const int64_t need = extend_need(a, i, have, bad);
    return (int)(need > 0 ? need : 0);
  });
  int64_t lo, hi;
  piece_of(a.s.num_pages, lo, hi);
  Counts found, unused;
  exchange(&sh, 0, make_int2(warp_count(a.s.refs, lo, hi, a.s.num_pages, 1, IsFree()), 0), found, unused);
  if (total > found.all) total = settle(a, &sh, sum, n, found.all);
  warp_number(a.s.refs, lo, hi, a.s.num_pages, 1, found.before, total, IsFree(), [&](int64_t page, int, int64_t g) {
    if (g >= total) return;
    const int i = owner_of(sum, n, g);
    int64_t have;
    bool bad;
    extend_need(a, i, have, bad);
    a.s.refs[page] = 1;
    a.s.table[(int64_t)i * a.s.max_pages + have + (g - sum[i])] = (int32_t)page;
  });
  cluster_sync_all();   // the lengths change only when no CTA reads them any more, and no count is read after this
  for (int i = rank * kPlanThreads + threadIdx.x; i < n; i += kPlanCtas * kPlanThreads) {
    int64_t have;
    bool bad;
    const int64_t need = extend_need(a, i, have, bad);
    const bool ok = !bad && (need == 0 || sum[i + 1] > sum[i]);
    if (bad) count_bad(a.s.status, NVFP4MLA_STAT_BAD_SLOT);
    if (ok) a.s.lens[i] += a.add[i];
    if (a.granted != nullptr) a.granted[i] = ok ? 1 : 0;
  }
}

// ------------------------------------------------------------------ compact
// workspace: the free pages below the live ones' number, in order, then the live pages at or above
// it, in order (each at most half of the pages), then how many, and the next item of the copy.
struct CompactArgs {
  PageState s;
  PageStore c;
  int32_t* remap;
  int32_t* num_live;
  int32_t* holes;
  int32_t* movers;
  int32_t* num_moves;
  unsigned long long* next;
};

// remap of the g-th page that moves, until its new place is looked up in `holes`.
__device__ __forceinline__ int32_t moving(int64_t g) { return (int32_t)(-2 - g); }
__device__ __forceinline__ int32_t move_of(int32_t mark) { return -2 - mark; }

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads) compact_plan_kernel(const CompactArgs a) {
  __shared__ PlanShared sh;
  let_dependents_start();
  const int64_t n = a.s.num_pages;
  const auto live = [](int64_t, int v) { return v > 0; };
  int64_t lo, hi;
  piece_of(n, lo, hi);
  Counts live_pages, moved, holes;
  exchange(&sh, 0, make_int2(warp_count(a.s.refs, lo, hi, n, 0, live), 0), live_pages, holes);
  const int64_t num_live = live_pages.all;
  // live pages behind the live ones' number, and free ones before it: equally many
  const auto moves = [=](int64_t i, int v) { return v > 0 && i >= num_live; };
  const auto hole = [=](int64_t i, int v) { return v <= 0 && i < num_live; };
  const int lane = threadIdx.x & 31;
  int2 c = make_int2(0, 0);
#pragma unroll 4
  for (int64_t i = lo; i < hi; i += 128) {
    const int64_t at = i + lane * 4;
    const int4 v = four_at(a.s.refs, at, n, 0);
    c.x += moves(at, v.x) + moves(at + 1, v.y) + moves(at + 2, v.z) + moves(at + 3, v.w);
    c.y += hole(at, v.x) + hole(at + 1, v.y) + hole(at + 2, v.z) + hole(at + 3, v.w);
  }
  exchange(&sh, 1, make_int2(__reduce_add_sync(kFull, c.x), __reduce_add_sync(kFull, c.y)), moved, holes);
  // list both, and say where each page goes. (What a move does to the counts, and the places of the
  // pages that move, is left to the grid that follows: done here, it took 8 of this kernel's 18 us at 40,000 pages.)
#pragma unroll 2
  for (int64_t i = lo; i < hi; i += 128) {
    const int64_t at = i + lane * 4;
    const int4 v = four_at(a.s.refs, at, n, 0);
    const int vs[4] = {v.x, v.y, v.z, v.w};
    int mine = 0;                      // free pages below, live pages above in the upper half
#pragma unroll
    for (int k = 0; k < 4; ++k) mine += (hole(at + k, vs[k]) ? 1 : 0) + (moves(at + k, vs[k]) ? 1 << 16 : 0);
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(kFull, incl, d);
      if (lane >= d) incl += o;
    }
    const int all = __shfl_sync(kFull, incl, 31), before = incl - mine;
    int g = holes.before + (before & 0xFFFF), m = moved.before + (before >> 16);
    holes.before += all & 0xFFFF;
    moved.before += all >> 16;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t page = at + k;         // behind n it may leave 32 bits
      if (hole(page, vs[k])) a.holes[g++] = (int32_t)page;
      if (page < n) a.remap[page] = moves(page, vs[k]) ? moving(m) : (vs[k] > 0 ? (int32_t)page : -1);
      if (moves(page, vs[k])) a.movers[m++] = (int32_t)page;
    }
  }
  if (cluster_ctarank() == 0 && threadIdx.x == 0) {
    *a.num_live = (int32_t)num_live;
    *a.num_moves = moved.all;
    *a.next = 0;
  }
  cluster_sync_all();   // no CTA leaves while another may read its count
}

// The first blocks write the tables, the counts and the places of the pages that move; the others copy
// pages. A page's place is read by table blocks while another writes it over its mark: both say the same.
__global__ void __launch_bounds__(kCopyThreads) compact_apply_kernel(const CompactArgs a, int table_blocks) {
  wait_for_planner();
  const int64_t moves = *a.num_moves;
  if ((int)blockIdx.x < table_blocks) {
    const int64_t entries = (int64_t)a.s.num_seqs * a.s.max_pages, step = (int64_t)table_blocks * kCopyThreads;
    for (int64_t i = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; i < entries; i += step) {
      const int32_t page = a.s.table[i];
      if (page == -1) continue;
      int32_t to = -1;
      if (page >= 0 && page < a.s.num_pages) {
        to = *static_cast<volatile const int32_t*>(a.remap + page);
        if (to < -1) to = a.holes[move_of(to)];
      }
      if (to < 0) count_bad(a.s.status, NVFP4MLA_STAT_BAD_PAGE);
      if (to != page) a.s.table[i] = to;
    }
    for (int64_t i = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; i < moves; i += step) {
      const int32_t from = a.movers[i], to = a.holes[i];
      a.s.refs[to] = a.s.refs[from];
      a.s.refs[from] = 0;
      a.remap[from] = to;
    }
    return;
  }
  // Items (page, chunk of a layer's page) are taken from a counter, the next one while this one's bytes
  // move: with a fixed share each, blocks ended between 46 and 78 us after the start.
  __shared__ int64_t taken[2];
  const int64_t chunks = chunks_of(a.c), per = chunks * a.c.layers, items = moves * per;
  int64_t it = blockIdx.x - table_blocks;
  const int64_t others = gridDim.x - table_blocks;
  for (int round = 0; it < items; round ^= 1) {
    if (threadIdx.x == 0) taken[round] = others + (int64_t)atomicAdd(a.next, 1ull);
    const int64_t i = it / per, rest = it % per;
    copy_chunk(a.c, rest / chunks, a.movers[i], a.holes[i], rest % chunks);
    __syncthreads();
    it = taken[round];
  }
}

// A dependent launch: the grid may start while the planner runs and waits for it where it reads.
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), unsigned blocks, unsigned threads, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Shared memory of the running sums (up to MAX_REQUESTS + 1 of them) and lengths, allowed once per device.
cudaError_t allow_sums(const void* kernel, int which) {
  static std::mutex mu;
  static bool done[2][64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 64 && done[which][dev]) return cudaSuccess;
  err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (2 * NVFP4MLA_MAX_REQUESTS + 1) * 4);
  if (err == cudaSuccess && dev < 64) done[which][dev] = true;
  return err;
}

}  // namespace

int64_t pages_copy_blocks(const PageStore& c, int64_t n) { return n * c.layers * chunks_of(c); }

cudaError_t launch_pages_copy(const PageStore& c, int64_t num_pages, const int32_t* src, const int32_t* dst, int64_t n,
                              int32_t* status, cudaStream_t stream) {
  copy_kernel<<<(unsigned)pages_copy_blocks(c, n), kCopyThreads, 0, stream>>>(c, num_pages, src, dst, status);
  return cudaGetLastError();
}

cudaError_t launch_pages_free(const PageState& s, const int32_t* seqs, int n, cudaStream_t stream) {
  const int64_t parts = (s.max_pages + 1023) / 1024;
  free_kernel<<<dim3((unsigned)n, (unsigned)(parts < 64 ? parts : 64)), 256, 0, stream>>>(s, seqs);
  return cudaGetLastError();
}

cudaError_t launch_pages_trim(const PageState& s, const int32_t* new_lens, cudaStream_t stream) {
  trim_kernel<<<(unsigned)s.num_seqs, 32, 0, stream>>>(s, new_lens);
  return cudaGetLastError();
}

cudaError_t launch_pages_fork(const PageState& s, const PageStore& c, const int32_t* src, const int32_t* dst, int n,
                              int32_t* new_pages, cudaStream_t stream) {
  const ForkArgs a{s, c, src, dst, n, new_pages};
  cudaError_t err = allow_sums(reinterpret_cast<const void*>(fork_plan_kernel), 0);
  if (err != cudaSuccess) return err;
  fork_plan_kernel<<<kPlanCtas, kPlanThreads, (size_t)(2 * n + 1) * 4, stream>>>(a);
  if ((err = cudaGetLastError()) != cudaSuccess) return err;
  const int64_t per = pages_copy_blocks(c, 1) + (s.max_pages + kRowEntries - 1) / kRowEntries;
  return launch_after(fork_apply_kernel, (unsigned)(n * per), kCopyThreads, stream, a);
}

cudaError_t launch_pages_extend(const PageState& s, const int32_t* add, int32_t* granted, cudaStream_t stream) {
  const ExtendArgs a{s, add, granted};
  const cudaError_t err = allow_sums(reinterpret_cast<const void*>(extend_kernel), 1);
  if (err != cudaSuccess) return err;
  extend_kernel<<<kPlanCtas, kPlanThreads, (size_t)(s.num_seqs + 1) * 4, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_pages_compact(const PageState& s, const PageStore& c, int32_t* remap, int32_t* num_live,
                                 int32_t* workspace, cudaStream_t stream) {
  const int64_t half = (s.num_pages / 2 + 4) / 4 * 4;
  const CompactArgs a{s, c, remap, num_live, workspace, workspace + half, workspace + 2 * half,
                      reinterpret_cast<unsigned long long*>(workspace + 2 * half + 2)};
  compact_plan_kernel<<<kPlanCtas, kPlanThreads, 0, stream>>>(a);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  const int64_t entries = (int64_t)s.num_seqs * s.max_pages, words = entries > s.num_pages / 2 ? entries : s.num_pages / 2;
  int64_t table_blocks = (words + 4 * kCopyThreads - 1) / (4 * kCopyThreads);
  if (table_blocks > 1024) table_blocks = 1024;
  int64_t copy_blocks = pages_copy_blocks(c, s.num_pages / 2 + 1);
  if (table_blocks < 1) table_blocks = 1;
  const int64_t most = (int64_t)device_sm_count() * 8;     // every block resident: 2,048 threads an SM
  if (copy_blocks > most) copy_blocks = most;
  return launch_after(compact_apply_kernel, (unsigned)(table_blocks + copy_blocks), kCopyThreads, stream, a, (int)table_blocks);
}

}  // namespace nvfp4mla
