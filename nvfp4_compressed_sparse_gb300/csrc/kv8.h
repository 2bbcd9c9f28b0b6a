// Internal declarations of the 8-bit per-head cache, of the speculative step over it and of the page operators.
#pragma once
#include "internal.h"

namespace nvfp4mla {

constexpr int kBlockTokens = 16;                             // tokens per scale
constexpr int kPageBlocks = kPageTokens / kBlockTokens;      // scale bytes of a page, head and kind
constexpr int kMaxKvHeads = 256;
constexpr int kMaxGroup = 128;                               // query heads per key/value head

// Byte offsets inside a page (see kv8_page_bytes in the public header).
__host__ __device__ constexpr int64_t kv8_codes_off(int kv_heads, int head_dim, int which, int head) {
  return ((int64_t)which * kv_heads + head) * kPageTokens * head_dim;
}
__host__ __device__ constexpr int64_t kv8_scales_off(int kv_heads, int head_dim, int head) {
  return (int64_t)2 * kv_heads * kPageTokens * head_dim + 2 * kPageBlocks * head;
}
__host__ __device__ constexpr int64_t kv8_page_size(int kv_heads, int head_dim) {
  return (kv8_scales_off(kv_heads, head_dim, kv_heads) + 127) / 128 * 128;
}

struct AppendParams {
  const uint16_t* x[2];          // keys, values
  int64_t token_stride[2], head_stride[2];
  int64_t num_tokens;
  const int32_t* cu;             // [B + 1]
  const int32_t* seq_lens;       // [B]
  const int32_t* page_table;     // [B, max_pages]
  int64_t max_pages;
  int B, kv_heads;
  uint8_t* cache;
  int64_t num_pages, page_bytes;
  int64_t slots;                 // block slots: num_tokens / 16 + 2 B
  int32_t* status;
};
cudaError_t launch_kv8_append(const AppendParams& p, int head_dim, bool fp16, cudaStream_t stream);

constexpr int kMaxAxes = 4;
struct RopeParams : AppendParams {
  const uint16_t* q;
  int64_t q_token_stride, q_head_stride;
  uint16_t* q_out;
  int64_t out_token_stride, out_head_stride;
  int heads;                     // of q
  const uint16_t* weight[2];     // of queries' and keys' norms, [D], or null: none
  float eps;
  const float* cos_sin;          // [max_positions, rot]: the pairs' cosines, then their sines
  int64_t max_positions;
  int rot;                       // dims that are rotated
  const int32_t* positions;      // [axes, num_tokens], or null: a token's place in its sequence
  int64_t axis_stride;
  int axes, ends[kMaxAxes];      // pairs up to ends[a] go by axis a
};
cudaError_t launch_kv8_append_rope(const RopeParams& p, int head_dim, bool fp16, bool interleaved, cudaStream_t stream);

struct Kv8DecodeParams {
  CUtensorMap cache_map;         // see encode_pages_map
  const uint16_t* q;
  int64_t q_token_stride, q_head_stride;
  const uint8_t* cache;
  int64_t num_pages, page_bytes;
  const int32_t* page_table;     // [B, max_pages]
  int64_t max_pages;
  const int32_t* seq_lens;       // [B]
  int B, Q, H, kv_heads, group;  // group = H / kv_heads
  float scale_log2;              // softmax_scale * log2(e)
  int window;                    // 0: none
  uint16_t* out;                 // [B, Q, H, D]
  float* lse;                    // [B, Q, H]
  int32_t* status;
  int ctas;                      // grid size
  float* part_o;                 // [2 ctas, columns, D]: a CTA's first and last segment, where they are partial
  float* part_ml;                // [2 ctas, columns, 2]: maximum (log2 units) and sum
  uint64_t* arrived;             // [ctas]: this call's tag with the CTAs that have left their partials
  uint64_t tag;                  // unique per call; its low 16 bits are the count's
  uint32_t withhold;             // testing aid: 1 = no tile is ever loaded
};
int kv8_decode_columns(int Q, int group);                      // (query, head) columns of a CTA's tile
cudaError_t launch_kv8_decode(const Kv8DecodeParams& p, int head_dim, bool fp16, cudaStream_t stream);

struct Kv8TreeParams : Kv8DecodeParams {
  const uint64_t* masks;         // [B, Q]
  uint32_t group_inverse;        // 2^24 / group + 1: (c x that) >> 24 = c / group for c < 2^14, as group <= 128
};
int kv8_tree_columns();                                         // (node, head) columns of a CTA's tile
cudaError_t launch_kv8_decode_tree(const Kv8TreeParams& p, int head_dim, bool fp16, cudaStream_t stream);

struct KeepParams {
  uint8_t* cache;
  int64_t layers, layer_stride, num_pages, page_bytes;
  const int32_t* page_table;     // [B, max_pages]
  int64_t max_pages;
  const int32_t* seq_lens;       // [B]
  const int32_t* path;           // [B, Q]
  const int32_t* accepted;       // [B]
  int B, Q, kv_heads;
  int32_t* new_lens;             // [B]
  int32_t* status;
};
cudaError_t launch_kv8_keep(const KeepParams& p, int head_dim, cudaStream_t stream);

struct VerifyParams {
  const void* logits;            // [B, Q, V], rows row_stride elements apart
  int64_t row_stride;
  const float* probs;            // [B, Q, V], or null
  int64_t probs_stride;
  const int32_t* drafts;         // [B, Q]
  const int32_t* parents;        // [B, Q]
  const float* uniforms;         // [B, Q]
  const float* temperatures;     // [B], or null: 1
  int B, Q, V;
  int32_t *tokens, *path;        // [B, Q]
  int32_t* accepted;             // [B]
  int32_t* status;
  int chunks;                    // of a row, at most
  float2* chunk_ms;              // [B Q, chunks]: largest logit of a chunk, sum of exponentials against it
  int32_t* chunk_at;             // [B Q, chunks]: where the largest is
  double* entry_sum;             // [B, entries]: sums of what a walk has left, by chunks or finer
};
int verify_chunks(int64_t V);
int verify_entries(int64_t V);
int verify_requests();           // at most, of a call
cudaError_t launch_spec_verify(const VerifyParams& p, int type, cudaStream_t stream);   // type: NVFP4MLA_BF16, _FP16 or _FP32

// The three arrays of the page operators, and the caches whose pages they move.
struct PageState {
  int32_t* table;                // [num_seqs, max_pages]
  int64_t max_pages;
  int32_t* lens;                 // [num_seqs]
  int num_seqs;
  int32_t* refs;                 // [num_pages]
  int64_t num_pages;
  int32_t* status;
};
struct PageStore {
  uint8_t* base;
  int64_t layers, layer_stride, page_bytes;
};
cudaError_t launch_pages_copy(const PageStore& c, int64_t num_pages, const int32_t* src, const int32_t* dst, int64_t n,
                              int32_t* status, cudaStream_t stream);
cudaError_t launch_pages_free(const PageState& s, const int32_t* seqs, int n, cudaStream_t stream);
cudaError_t launch_pages_trim(const PageState& s, const int32_t* new_lens, cudaStream_t stream);
cudaError_t launch_pages_fork(const PageState& s, const PageStore& c, const int32_t* src, const int32_t* dst, int n,
                              int32_t* new_pages, cudaStream_t stream);
cudaError_t launch_pages_extend(const PageState& s, const int32_t* add, int32_t* granted, cudaStream_t stream);
cudaError_t launch_pages_compact(const PageState& s, const PageStore& c, int32_t* remap, int32_t* num_live,
                                 int32_t* workspace, cudaStream_t stream);
int64_t pages_copy_blocks(const PageStore& c, int64_t n);    // blocks of a copy grid over n pages

}  // namespace nvfp4mla
