// How the attention kernels over the 8-bit per-head cache cut a step into CTAs' shares, and what else they
// have in common.
#pragma once
#include <cstdint>

#include "kv8.h"
#include "ptx.cuh"

namespace nvfp4mla {
namespace {

using namespace ptx;

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

// A walk over the segments of this CTA: per unit, the tiles of it that the CTA has. Units go by column
// tile, request and key/value head; so the column tiles of one head's tokens run on different CTAs at
// about the same time, and all but one of them read the codes from L2. (kUnitCost: what starting and ending
// a unit costs, in tiles: in the whole sequence, each unit's tiles come behind so many that are none.)
template <int kTile, int kUnitCost>
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

}  // namespace
}  // namespace nvfp4mla
