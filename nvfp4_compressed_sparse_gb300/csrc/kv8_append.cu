// kv8_append: new keys and values into the 8-bit per-head cache.
//
// A warp takes one block of 16 tokens of one head, keys and values. It finds its request and block
// from its number, reads the block's new rows (all loads issued before any is used), takes the
// largest finite magnitude, and from it the block's exponent; the codes are x 2^(127 - e) rounded
// to E4M3, exact but for that one rounding, since a power of two moves no mantissa bit.
//
// The floor is the traffic, three bytes per value (two in, one out). Consecutive warps take
// consecutive heads of the same tokens, so that a token's row of all heads is read in one piece.
//
// Measured (device time): 12 prompts of 300-9,000 tokens, 8 heads of 128: 213 MB in 36.9 us, 5.8 TB/s,
// 85 % of the measured copy bandwidth, ALU pipe 55 % busy (it makes the codes); 64 requests of one token:
// 4.2 us, a launch and one chain of loads. Keys and values by one warp instead of two took 64 to 62 us,
// the path for finite blocks 62 to 40.
#include "../../include/nvfp4mla.h"
#include "kv8.h"
#include "kv8_codes.cuh"
#include "ptx.cuh"

namespace nvfp4mla {
namespace {

using namespace ptx;

constexpr int kAppendThreads = 128;    // five such blocks an SM: 37 us (a row above), three of 256 threads 40

template <int D, bool kHalf>
__global__ void __launch_bounds__(kAppendThreads, 5) append_kernel(const AppendParams p) {
  constexpr int kLanes = D / 8;              // lanes per row, 8 values (16 bytes) each
  constexpr int kRows = 32 / kLanes;         // rows per load
  constexpr int kLoads = kBlockTokens / kRows;
  const int lane = threadIdx.x & 31;
  const unsigned item = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int slot = (int)(item / (unsigned)p.kv_heads), head = (int)(item - (unsigned)slot * (unsigned)p.kv_heads);
  if (slot >= p.slots) return;

  const int b = request_of(p, slot);
  const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1), len = __ldg(p.seq_lens + b);
  const int nth = slot - first_slot(p, b);
  const int64_t n = (int64_t)c1 - c0, p0 = len - n;
  if (c0 < 0 || n < 0 || c1 > p.num_tokens || (p0 < 0 && n > 0)) {
    if (nth == 0 && head == 0 && lane == 0 && p.status != nullptr) atomicAdd(p.status + NVFP4MLA_STAT_BAD_SLOT, 1);
    return;
  }
  if (nth < 0 || n == 0) return;
  // the block's first position, its first new row, and the rows that are new: first .. behind - 1
  const int64_t t0 = (p0 / kBlockTokens + nth) * kBlockTokens;
  if (t0 >= len) return;
  const int first = p0 > t0 ? (int)(p0 - t0) : 0, behind = (int)min((int64_t)kBlockTokens, len - t0);
  const int64_t col = t0 / kPageTokens;
  const int64_t page = col < p.max_pages ? __ldg(p.page_table + (int64_t)b * p.max_pages + col) : -1;
  if (page < 0 || page >= p.num_pages) {
    if (head == 0 && lane == 0 && p.status != nullptr) atomicAdd(p.status + NVFP4MLA_STAT_BAD_PAGE, 1);
    return;
  }
  const int quarter = (int)(t0 % kPageTokens) / kBlockTokens;
  const int row0 = lane / kLanes, col8 = (lane % kLanes) * 8;
  const int64_t token = c0 + (t0 - p0);      // of the block's row 0 (behind the block's old rows: not read)
  uint8_t* base = p.cache + page * p.page_bytes;
  uint8_t* scales = base + kv8_scales_off(p.kv_heads, D, head) + quarter;

  uint4 w[2][kLoads];
  uint32_t before[2];
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const uint16_t* x = p.x[which] + head * p.head_stride[which] + col8;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = i * kRows + row0;
      w[which][i] = make_uint4(0u, 0u, 0u, 0u);
      if (row >= first && row < behind) w[which][i] = __ldcs(reinterpret_cast<const uint4*>(x + (token + row) * p.token_stride[which]));
    }
    before[which] = first > 0 ? min((uint32_t)scales[which * kPageBlocks], 253u) : 0u;
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    uint8_t* codes = base + kv8_codes_off(p.kv_heads, D, which, head) + quarter * kBlockTokens * D + col8;
    put_block<D, kHalf>(w[which], row0, first, behind, before[which], codes, scales + which * kPageBlocks);
  }
}

}  // namespace

cudaError_t launch_kv8_append(const AppendParams& p, int head_dim, bool fp16, cudaStream_t stream) {
  const int64_t warps = p.slots * p.kv_heads;
  const unsigned blocks = (unsigned)((warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32));
  if (head_dim == 128) {
    if (fp16) append_kernel<128, true><<<blocks, kAppendThreads, 0, stream>>>(p);
    else append_kernel<128, false><<<blocks, kAppendThreads, 0, stream>>>(p);
  } else {
    if (fp16) append_kernel<64, true><<<blocks, kAppendThreads, 0, stream>>>(p);
    else append_kernel<64, false><<<blocks, kAppendThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace nvfp4mla
