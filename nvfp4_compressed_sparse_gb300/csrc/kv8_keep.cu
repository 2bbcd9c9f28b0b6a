// kv8_keep: after a verify step, the accepted drafts' keys and values move up to the places behind the
// token that they follow.
//
// A warp takes one request, head, layer and kind (keys or values) and goes through the blocks of 16 places
// that the accepted drafts move to, in order: it reads the rows that the block will hold, 16 bytes a lane,
// with the scale bytes of their blocks, takes the largest byte for the block, and writes the rows again
// under that. A draft never moves to a higher place, and the i-th accepted one lies at i or above: what a
// block reads, the blocks before it have not written.
//
// What bounds it: latency. A block is four dependent reads (the path, the table, the scale bytes beside the rows) and a
// write; a step's bytes are few. Measured, back to back: 16 trees of 32 nodes, eight heads of 128 in eight layers (2 MB), with
// kv_pages_trim behind it: 6.9 us, 128 trees of 12 in four layers of four heads of 64 the same.
#include "../../include/nvfp4mla.h"
#include "kv8.h"
#include "kv8_codes.cuh"
#include "ptx.cuh"

namespace nvfp4mla {
namespace {

using namespace ptx;

constexpr int kKeepThreads = 128;
constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ uint32_t shrink4(uint32_t four, float less) {
  return shrink2(four & 0xFFFFu, less) | (shrink2(four >> 16, less) << 16);
}

template <int D>
__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const KeepParams p) {
  constexpr int kLanes = D / 16, kAtOnce = 32 / kLanes, kLoads = kBlockTokens / kAtOnce;
  const int lane = threadIdx.x & 31;
  int64_t item = (int64_t)blockIdx.x * (kKeepThreads / 32) + (threadIdx.x >> 5);
  const int64_t per = (int64_t)2 * p.kv_heads * p.layers;
  if (item >= p.B * per) return;
  const int b = (int)(item / per);
  item -= b * per;
  const int64_t layer = item / (2 * p.kv_heads);
  const int rest = (int)(item - layer * 2 * p.kv_heads), head = rest >> 1, which = rest & 1;
  const bool speaks = layer == 0 && rest == 0;
  const int len = p.seq_lens[b], base = len - p.Q, count = p.accepted[b];
  // lane i: the node that becomes the i-th accepted (and the 32 + i-th)
  const int32_t* path = p.path + (int64_t)b * p.Q;
  const int n0 = lane < count && lane < p.Q ? path[lane] : -1, n1 = 32 + lane < count && 32 + lane < p.Q ? path[32 + lane] : -1;
  const int u0 = __shfl_up_sync(kFull, n0, 1), last0 = __shfl_sync(kFull, n0, 31), u1 = __shfl_up_sync(kFull, n1, 1);
  const int b0 = lane == 0 ? 0 : u0, b1 = lane == 0 ? last0 : u1;
  const bool wrong = (lane < count && (n0 <= b0 || n0 >= p.Q)) || (32 + lane < count && (n1 <= b1 || n1 >= p.Q));
  const bool bad = __any_sync(kFull, wrong) || count >= p.Q || (base < 0 && count >= 0);
  if (speaks && lane == 0) {
    p.new_lens[b] = bad || count < 0 ? len : base + 1 + count;
    if (bad && p.status != nullptr) atomicAdd(p.status + NVFP4MLA_STAT_BAD_SLOT, 1);
  }
  if (bad || count <= 0) return;

  uint8_t* cache = p.cache + layer * p.layer_stride;
  const int32_t* table = p.page_table + (int64_t)b * p.max_pages;
  auto page_of = [&](int t) -> int64_t {
    const int col = t / kPageTokens;
    const int page = col < p.max_pages ? table[col] : -1;
    return page >= 0 && page < p.num_pages ? page : -1;
  };
  const int row0 = lane / kLanes, at16 = (lane % kLanes) * 16;
  for (int t0 = (base + 1) / kBlockTokens * kBlockTokens; t0 <= base + count; t0 += kBlockTokens) {
    const int64_t page = page_of(t0);
    uint4 w[kLoads];
    int byte[kLoads];                // -1: a row that stays what it is
    int src[kLoads];
    bool moves = false;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int t = t0 + i * kAtOnce + row0, nth = t - base - 1;
      const int a = __shfl_sync(kFull, n0, nth & 31), c = __shfl_sync(kFull, n1, nth & 31);
      src[i] = nth >= count ? -1 : (nth < 0 ? t : base + (nth < 32 ? a : c));
      moves = moves || (src[i] >= 0 && src[i] != t);
    }
    if (!__any_sync(kFull, moves)) continue;
    if (page < 0) {
      if (speaks && lane == 0 && p.status != nullptr) atomicAdd(p.status + NVFP4MLA_STAT_BAD_PAGE, 1);
      continue;
    }
    int top = -1;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      byte[i] = -1;
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (src[i] < 0) continue;
      const int64_t from = page_of(src[i]);
      if (from < 0) {
        if (speaks && at16 == 0 && p.status != nullptr) atomicAdd(p.status + NVFP4MLA_STAT_BAD_PAGE, 1);
        continue;
      }
      const int r = src[i] % kPageTokens;
      const uint8_t* at = cache + from * p.page_bytes;
      w[i] = *reinterpret_cast<const uint4*>(at + kv8_codes_off(p.kv_heads, D, which, head) + r * D + at16);
      byte[i] = min((int)at[kv8_scales_off(p.kv_heads, D, head) + which * kPageBlocks + r / kBlockTokens], 253);
      top = max(top, byte[i]);
    }
    top = __reduce_max_sync(kFull, top);
    if (top < 0) continue;           // none has a page
    __syncwarp();                    // every row and byte has been read
    uint8_t* to = cache + page * p.page_bytes;
    uint8_t* codes = to + kv8_codes_off(p.kv_heads, D, which, head) + (t0 % kPageTokens) * D + at16;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = i * kAtOnce + row0;
      if (byte[i] < 0 || (src[i] == t0 + row && byte[i] == top)) continue;
      if (byte[i] < top) {
        const float less = __uint_as_float((uint32_t)(127 - min(top - byte[i], 126)) << 23);
        w[i] = make_uint4(shrink4(w[i].x, less), shrink4(w[i].y, less), shrink4(w[i].z, less), shrink4(w[i].w, less));
      }
      *reinterpret_cast<uint4*>(codes + row * D) = w[i];
    }
    if (lane == 0) to[kv8_scales_off(p.kv_heads, D, head) + which * kPageBlocks + (t0 % kPageTokens) / kBlockTokens] = (uint8_t)top;
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_kv8_keep(const KeepParams& p, int head_dim, cudaStream_t stream) {
  const int64_t warps = (int64_t)p.B * 2 * p.kv_heads * p.layers;
  const unsigned blocks = (unsigned)((warps + kKeepThreads / 32 - 1) / (kKeepThreads / 32));
  if (head_dim == 128) keep_kernel<128><<<blocks, kKeepThreads, 0, stream>>>(p);
  else keep_kernel<64><<<blocks, kKeepThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace nvfp4mla
