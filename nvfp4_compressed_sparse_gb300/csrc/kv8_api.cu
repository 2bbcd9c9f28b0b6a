// Host side of the entry points of the 8-bit per-head cache, of the speculative step over it and of the
// page operators: argument checks and launches. As in api.cu: no allocation, no synchronisation, everything on the caller's stream.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "../../include/nvfp4mla.h"
#include "kv8.h"

using namespace nvfp4mla;

static bool kv8_sizes_ok(int kv_heads, int head_dim) {
  return kv_heads >= 1 && kv_heads <= kMaxKvHeads && (head_dim == 64 || head_dim == 128);
}

static bool all_device(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (pointer_kind(p) != kPtrDevice) return false;
  return true;
}
static bool any_null(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (p == nullptr) return true;
  return false;
}
static bool optional_ok(const void* p) { return p == nullptr || pointer_kind(p) == kPtrDevice; }
// Of [a, a + n) and [b, b + m); a null pointer overlaps nothing.
static bool overlap(const void* a, size_t n, const void* b, size_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && x < y + m && y < x + n;
}
static bool words_aligned(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return false;
  return true;
}
static int status_of(cudaError_t err) { return err == cudaSuccess ? NVFP4MLA_OK : NVFP4MLA_ERR_CUDA; }

extern "C" {

size_t kv8_page_bytes(int kv_heads, int head_dim) {
  return kv8_sizes_ok(kv_heads, head_dim) ? (size_t)kv8_page_size(kv_heads, head_dim) : 0;
}

// What kv8_append and kv8_append_rope have in common. NVFP4MLA_OK with p->num_tokens 0: nothing to enqueue.
static int check_append(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                        int64_t v_head_stride, int dtype, int64_t num_tokens, const int32_t* cu_tokens,
                        const int32_t* seq_lens, const int32_t* page_table, int64_t max_pages_per_seq, int B, int kv_heads,
                        int head_dim, void* cache, int64_t num_pages, int32_t* dev_status, AppendParams* to) {
  if (!kv8_sizes_ok(kv_heads, head_dim) || (dtype != NVFP4MLA_BF16 && dtype != NVFP4MLA_FP16)) return NVFP4MLA_ERR_INVALID_ARG;
  if (B < 0 || num_tokens < 0 || num_tokens > INT32_MAX || num_pages < 1 || num_pages > INT32_MAX || max_pages_per_seq < 1)
    return NVFP4MLA_ERR_INVALID_ARG;
  if (k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 || v_head_stride < 0) return NVFP4MLA_ERR_INVALID_ARG;
  to->num_tokens = 0;
  if (B == 0 || num_tokens == 0) return NVFP4MLA_OK;
  if (any_null({k, v, cu_tokens, seq_lens, page_table, cache})) return NVFP4MLA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cache, 128)) return NVFP4MLA_ERR_ALIGNMENT;
  if (((k_token_stride | k_head_stride | v_token_stride | v_head_stride) & 7) != 0) return NVFP4MLA_ERR_ALIGNMENT;
  if (!words_aligned({cu_tokens, seq_lens, page_table, dev_status})) return NVFP4MLA_ERR_ALIGNMENT;
  if (!all_device({k, v, cu_tokens, seq_lens, page_table, cache}) || !optional_ok(dev_status)) return NVFP4MLA_ERR_INVALID_ARG;
  AppendParams& p = *to;
  p.x[0] = static_cast<const uint16_t*>(k);
  p.x[1] = static_cast<const uint16_t*>(v);
  p.token_stride[0] = k_token_stride;
  p.token_stride[1] = v_token_stride;
  p.head_stride[0] = k_head_stride;
  p.head_stride[1] = v_head_stride;
  p.num_tokens = num_tokens;
  p.cu = cu_tokens;
  p.seq_lens = seq_lens;
  p.page_table = page_table;
  p.max_pages = max_pages_per_seq;
  p.B = B;
  p.kv_heads = kv_heads;
  p.cache = static_cast<uint8_t*>(cache);
  p.num_pages = num_pages;
  p.page_bytes = kv8_page_size(kv_heads, head_dim);
  p.slots = num_tokens / kBlockTokens + 2 * (int64_t)B;
  p.status = dev_status;
  return p.slots * kv_heads > (int64_t)INT32_MAX ? NVFP4MLA_ERR_UNSUPPORTED : NVFP4MLA_OK;
}

int kv8_append(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
               int64_t v_head_stride, int dtype, int64_t num_tokens, const int32_t* cu_tokens,
               const int32_t* seq_lens, const int32_t* page_table, int64_t max_pages_per_seq, int B, int kv_heads,
               int head_dim, void* cache, int64_t num_pages, int32_t* dev_status, void* stream) {
  AppendParams p{};
  const int rc = check_append(k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, dtype, num_tokens, cu_tokens,
                              seq_lens, page_table, max_pages_per_seq, B, kv_heads, head_dim, cache, num_pages, dev_status, &p);
  if (rc != NVFP4MLA_OK || p.num_tokens == 0) return rc;
  return status_of(launch_kv8_append(p, head_dim, dtype == NVFP4MLA_FP16, static_cast<cudaStream_t>(stream)));
}

int kv8_append_rope(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k, int64_t k_token_stride,
                    int64_t k_head_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride, int dtype,
                    int64_t num_tokens, const int32_t* cu_tokens, const int32_t* seq_lens, const int32_t* page_table,
                    int64_t max_pages_per_seq, int B, int heads, int kv_heads, int head_dim, const void* q_weight,
                    const void* k_weight, float eps, const float* cos_sin, int64_t max_positions, int rotary_dim,
                    int interleaved, const int32_t* positions, int64_t axis_stride, const int32_t* sections, int axes,
                    void* q_out, int64_t out_token_stride, int64_t out_head_stride, void* cache, int64_t num_pages,
                    int32_t* dev_status, void* stream) {
  if (heads < 1 || heads > kMaxKvHeads * kMaxGroup || rotary_dim < 16 || rotary_dim > head_dim || rotary_dim % 16 != 0)
    return NVFP4MLA_ERR_INVALID_ARG;
  if (max_positions < 1 || max_positions > INT32_MAX || axes < 1 || axes > kMaxAxes || !(eps >= 0.f) || std::isinf(eps)) return NVFP4MLA_ERR_INVALID_ARG;
  if (q_token_stride < 0 || q_head_stride < 0 || out_token_stride < 0 || out_head_stride < 0 || axis_stride < 0) return NVFP4MLA_ERR_INVALID_ARG;
  if (axes > 1 && (positions == nullptr || sections == nullptr)) return NVFP4MLA_ERR_INVALID_ARG;
  RopeParams p{};
  if (axes > 1) {
    int64_t end = 0;
    for (int a = 0; a < axes; ++a) {
      if (sections[a] < 0) return NVFP4MLA_ERR_INVALID_ARG;
      end += sections[a];
      p.ends[a] = (int)(end < rotary_dim ? end : rotary_dim);
    }
    if (end != rotary_dim / 2) return NVFP4MLA_ERR_INVALID_ARG;
  }
  if (B > 0 && num_tokens > 0) {
    if (any_null({q, q_out, cos_sin})) return NVFP4MLA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16)) return NVFP4MLA_ERR_ALIGNMENT;
    if (((q_token_stride | q_head_stride | out_token_stride | out_head_stride) & 7) != 0 || !words_aligned({cos_sin, positions}))
      return NVFP4MLA_ERR_ALIGNMENT;
    // rows of q_out that overlap one another, or q's under other strides: a row would be read or kept by chance
    const bool tokens = num_tokens > 1, more = heads > 1;
    if ((tokens && out_token_stride < head_dim) || (more && out_head_stride < head_dim)) return NVFP4MLA_ERR_INVALID_ARG;
    if (q == q_out && ((tokens && q_token_stride != out_token_stride) || (more && q_head_stride != out_head_stride))) return NVFP4MLA_ERR_INVALID_ARG;
  }
  const int rc = check_append(k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, dtype, num_tokens, cu_tokens,
                              seq_lens, page_table, max_pages_per_seq, B, kv_heads, head_dim, cache, num_pages, dev_status, &p);
  if (rc != NVFP4MLA_OK || p.num_tokens == 0) return rc;
  if (!all_device({q, q_out, cos_sin}) || !optional_ok(positions) || !optional_ok(q_weight) || !optional_ok(k_weight))
    return NVFP4MLA_ERR_INVALID_ARG;
  p.q = static_cast<const uint16_t*>(q);
  p.q_token_stride = q_token_stride;
  p.q_head_stride = q_head_stride;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.out_token_stride = out_token_stride;
  p.out_head_stride = out_head_stride;
  p.heads = heads;
  p.weight[0] = static_cast<const uint16_t*>(q_weight);
  p.weight[1] = static_cast<const uint16_t*>(k_weight);
  p.eps = eps;
  p.cos_sin = cos_sin;
  p.max_positions = max_positions;
  p.rot = rotary_dim;
  p.positions = positions;
  p.axis_stride = axis_stride;
  p.axes = axes;
  return status_of(launch_kv8_append_rope(p, head_dim, dtype == NVFP4MLA_FP16, interleaved != 0, static_cast<cudaStream_t>(stream)));
}

// Workspace: partial O [2 ctas, columns, D] f32 | partial (maximum, sum) [2 ctas, columns, 2] f32 |
// arrival counts [ctas] u64, or three words a CTA that say what is to be joined; each part 256-byte aligned.
struct Kv8Workspace {
  size_t ml, arrived, total;
};
static size_t align256(size_t x) { return (x + 255) / 256 * 256; }
static Kv8Workspace decode_workspace(int columns, int head_dim, int ctas, int words = 1) {
  Kv8Workspace w;
  w.ml = align256((size_t)2 * ctas * columns * head_dim * sizeof(float));
  w.arrived = w.ml + align256((size_t)2 * ctas * columns * 2 * sizeof(float));
  w.total = w.arrived + align256((size_t)ctas * words * sizeof(uint64_t));
  return w;
}

// The cache as a 5-D tensor of bytes: [pages][1 KB groups of a kind's heads][kinds][8 rows][128], a row
// being a token, or two of 64 dims. One box is a head's keys and values of one page, eight rows of the
// one beside eight of the other, so that the groups of either lie at one stride in shared memory, page
// after page; swizzled as the tensor cores read them. A page number behind the cache reads as zeros,
// from nowhere.
static bool encode_pages_map(CUtensorMap* map, const void* cache, int64_t num_pages, int64_t page_bytes, int kv_heads,
                             int head_dim) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (fn == nullptr) return false;
  const cuuint64_t block = (cuuint64_t)kPageTokens * head_dim, groups = block / 1024;
  const cuuint64_t dims[5] = {128, 8, 2, groups * (cuuint64_t)kv_heads, (cuuint64_t)num_pages};
  const cuuint64_t strides[4] = {128, block * (cuuint64_t)kv_heads, 1024, (cuuint64_t)page_bytes};
  const cuuint32_t box[5] = {128, 8, 2, (cuuint32_t)groups, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void*>(cache), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The cache as rows of head_dim bytes: [pages][heads of keys, then of values][64 tokens]. One box is a head's keys of one
// page, swizzled as the tensor cores read rows of that size.
static bool encode_rows_map(CUtensorMap* map, const void* cache, int64_t num_pages, int64_t page_bytes, int kv_heads,
                            int head_dim) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)2 * kv_heads * kPageTokens, (cuuint64_t)num_pages};
  const cuuint64_t strides[2] = {(cuuint64_t)head_dim, (cuuint64_t)page_bytes};
  const cuuint32_t box[3] = {(cuuint32_t)head_dim, (cuuint32_t)kPageTokens, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(cache), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static bool decode_sizes_ok(int B, int Q, int H, int kv_heads, int head_dim) {
  if (!kv8_sizes_ok(kv_heads, head_dim) || B < 1 || Q < 1 || Q > 16 || H < 1 || H % kv_heads != 0) return false;
  return H / kv_heads <= kMaxGroup;
}

size_t kv8_decode_workspace_size(int B, int Q, int H, int kv_heads, int head_dim, int num_sms) {
  if (!decode_sizes_ok(B, Q, H, kv_heads, head_dim)) return 0;
  if (num_sms <= 0) num_sms = device_sm_count();
  if (num_sms <= 0) return 0;
  return decode_workspace(kv8_decode_columns(Q, H / kv_heads), head_dim, num_sms).total;
}

// What kv8_decode and kv8_decode_tree have in common, their sizes checked before: columns and pages of a tile, words of the
// workspace for each CTA.
static int check_decode(const void* q, int64_t q_token_stride, int64_t q_head_stride, int dtype, const void* cache,
                        int64_t num_pages, const int32_t* page_table, int64_t max_pages_per_seq, const int32_t* seq_lens, int B,
                        int Q, int H, int kv_heads, int head_dim, float softmax_scale, int window, void* out, float* lse,
                        void* workspace, size_t workspace_bytes, int32_t* dev_status, uint32_t flags, int columns,
                        int tile_pages, int words, Kv8DecodeParams* to) {
  if (dtype != NVFP4MLA_BF16 && dtype != NVFP4MLA_FP16) return NVFP4MLA_ERR_INVALID_ARG;
  if (num_pages < 1 || num_pages >= INT32_MAX || max_pages_per_seq < 1 || window < 0) return NVFP4MLA_ERR_INVALID_ARG;
  if (q_token_stride < 0 || q_head_stride < 0) return NVFP4MLA_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || std::isinf(softmax_scale)) return NVFP4MLA_ERR_INVALID_ARG;
  if (any_null({q, cache, page_table, seq_lens, out, lse})) return NVFP4MLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cache, 128)) return NVFP4MLA_ERR_ALIGNMENT;
  if (((q_token_stride | q_head_stride) & 7) != 0 || !words_aligned({page_table, seq_lens, lse, dev_status}))
    return NVFP4MLA_ERR_ALIGNMENT;
  const int sms = device_sm_count();
  if (sms <= 0) return NVFP4MLA_ERR_CUDA;
  const Kv8Workspace w = decode_workspace(columns, head_dim, sms, words);
  if (workspace == nullptr || workspace_bytes < w.total) return NVFP4MLA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return NVFP4MLA_ERR_ALIGNMENT;
  if (!all_device({q, cache, page_table, seq_lens, out, lse, workspace}) || !optional_ok(dev_status))
    return NVFP4MLA_ERR_INVALID_ARG;
  // 32-bit row numbers, and tile numbers of the whole step
  const int64_t units = (int64_t)kv_heads * ((Q * (H / kv_heads) + columns - 1) / columns);
  if ((int64_t)B * Q * H > INT32_MAX || max_pages_per_seq > INT32_MAX) return NVFP4MLA_ERR_UNSUPPORTED;
  if (max_pages_per_seq / tile_pages + 16 > INT32_MAX / (B * units)) return NVFP4MLA_ERR_UNSUPPORTED;
  Kv8DecodeParams& p = *to;
  p.q = static_cast<const uint16_t*>(q);
  p.q_token_stride = q_token_stride;
  p.q_head_stride = q_head_stride;
  p.cache = static_cast<const uint8_t*>(cache);
  p.num_pages = num_pages;
  p.page_bytes = kv8_page_size(kv_heads, head_dim);
  p.page_table = page_table;
  p.max_pages = max_pages_per_seq;
  p.seq_lens = seq_lens;
  p.B = B;
  p.Q = Q;
  p.H = H;
  p.kv_heads = kv_heads;
  p.group = H / kv_heads;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.window = window;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.status = dev_status;
  const int cap = (int)(flags & 0xFFFFu);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.ctas = cap > 0 && cap < sms ? cap : sms;
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + w.ml);
  p.arrived = reinterpret_cast<uint64_t*>(ws + w.arrived);
  p.tag = (next_call_tag() & ~(uint64_t)0xFFFF) | 0x10000u;
  p.withhold = (flags & NVFP4MLA_FLAG_TEST_TIMEOUT) ? 1u : 0u;
  return NVFP4MLA_OK;
}

int kv8_decode(const void* q, int64_t q_token_stride, int64_t q_head_stride, int dtype, const void* cache,
               int64_t num_pages, const int32_t* page_table, int64_t max_pages_per_seq, const int32_t* seq_lens, int B,
               int Q, int H, int kv_heads, int head_dim, float softmax_scale, int window, void* out, float* lse,
               void* workspace, size_t workspace_bytes, int32_t* dev_status, uint32_t flags, void* stream) {
  if (!decode_sizes_ok(B, Q, H, kv_heads, head_dim)) return NVFP4MLA_ERR_INVALID_ARG;
  Kv8DecodeParams p{};
  const int rc = check_decode(q, q_token_stride, q_head_stride, dtype, cache, num_pages, page_table, max_pages_per_seq, seq_lens, B, Q, H,
                              kv_heads, head_dim, softmax_scale, window, out, lse, workspace, workspace_bytes, dev_status, flags,
                              kv8_decode_columns(Q, H / kv_heads), 2, 1, &p);
  if (rc != NVFP4MLA_OK) return rc;
  if (!encode_pages_map(&p.cache_map, cache, num_pages, p.page_bytes, kv_heads, head_dim)) return NVFP4MLA_ERR_CUDA;
  return status_of(launch_kv8_decode(p, head_dim, dtype == NVFP4MLA_FP16, static_cast<cudaStream_t>(stream)));
}

constexpr int kTreeWords = 3;
static bool tree_sizes_ok(int B, int Q, int H, int kv_heads, int head_dim) {
  if (!kv8_sizes_ok(kv_heads, head_dim) || B < 1 || Q < 1 || Q > NVFP4MLA_MAX_NODES || H < 1 || H % kv_heads != 0) return false;
  return H / kv_heads <= kMaxGroup;
}

size_t kv8_decode_tree_workspace_size(int B, int Q, int H, int kv_heads, int head_dim, int num_sms) {
  if (!tree_sizes_ok(B, Q, H, kv_heads, head_dim)) return 0;
  if (num_sms <= 0) num_sms = device_sm_count();
  if (num_sms <= 0) return 0;
  return decode_workspace(kv8_tree_columns(), head_dim, num_sms, kTreeWords).total;
}

int kv8_decode_tree(const void* q, int64_t q_token_stride, int64_t q_head_stride, int dtype, const void* cache,
                    int64_t num_pages, const int32_t* page_table, int64_t max_pages_per_seq, const int32_t* seq_lens,
                    const uint64_t* masks, int B, int Q, int H, int kv_heads, int head_dim, float softmax_scale, int window,
                    void* out, float* lse, void* workspace, size_t workspace_bytes, int32_t* dev_status, uint32_t flags,
                    void* stream) {
  if (!tree_sizes_ok(B, Q, H, kv_heads, head_dim) || masks == nullptr) return NVFP4MLA_ERR_INVALID_ARG;
  if (window > 0 && window < Q) return NVFP4MLA_ERR_UNSUPPORTED;
  if (!aligned(masks, 8)) return NVFP4MLA_ERR_ALIGNMENT;
  Kv8TreeParams p{};
  const int rc = check_decode(q, q_token_stride, q_head_stride, dtype, cache, num_pages, page_table, max_pages_per_seq, seq_lens, B, Q, H,
                              kv_heads, head_dim, softmax_scale, window, out, lse, workspace, workspace_bytes, dev_status, flags,
                              kv8_tree_columns(), 2, kTreeWords, &p);
  if (rc != NVFP4MLA_OK) return rc;
  if (!all_device({masks})) return NVFP4MLA_ERR_INVALID_ARG;
  if (!encode_rows_map(&p.cache_map, cache, num_pages, p.page_bytes, kv_heads, head_dim)) return NVFP4MLA_ERR_CUDA;
  p.masks = masks;
  p.group_inverse = (1u << 24) / (uint32_t)p.group + 1;
  return status_of(launch_kv8_decode_tree(p, head_dim, dtype == NVFP4MLA_FP16, static_cast<cudaStream_t>(stream)));
}

int kv8_keep(void* cache, int64_t layers, int64_t layer_stride, int64_t num_pages, const int32_t* page_table,
             int64_t max_pages_per_seq, const int32_t* seq_lens, const int32_t* path, const int32_t* accepted, int B, int Q,
             int kv_heads, int head_dim, int32_t* new_lens, int32_t* dev_status, void* stream) {
  if (!kv8_sizes_ok(kv_heads, head_dim) || B < 0 || Q < 1 || Q > NVFP4MLA_MAX_NODES || layers < 1) return NVFP4MLA_ERR_INVALID_ARG;
  if (num_pages < 1 || num_pages > INT32_MAX || max_pages_per_seq < 1) return NVFP4MLA_ERR_INVALID_ARG;
  const int64_t page_bytes = kv8_page_size(kv_heads, head_dim);
  if (layers > 1 && layer_stride < num_pages * page_bytes) return NVFP4MLA_ERR_INVALID_ARG;
  if (B == 0) return NVFP4MLA_OK;
  if (any_null({cache, page_table, seq_lens, path, accepted, new_lens})) return NVFP4MLA_ERR_INVALID_ARG;
  if (!aligned(cache, 128) || (layers > 1 && layer_stride % 16 != 0)) return NVFP4MLA_ERR_ALIGNMENT;
  if (!words_aligned({page_table, seq_lens, path, accepted, new_lens, dev_status})) return NVFP4MLA_ERR_ALIGNMENT;
  if (!all_device({cache, page_table, seq_lens, path, accepted, new_lens}) || !optional_ok(dev_status)) return NVFP4MLA_ERR_INVALID_ARG;
  const size_t n = (size_t)B * sizeof(int32_t);
  // (a request is read by many warps, one of which writes its new length)
  if (overlap(new_lens, n, seq_lens, n) || overlap(new_lens, n, accepted, n) || overlap(new_lens, n, path, n * Q)) return NVFP4MLA_ERR_INVALID_ARG;
  if (layers > INT32_MAX / (2 * kv_heads) / B) return NVFP4MLA_ERR_UNSUPPORTED;
  const KeepParams p{static_cast<uint8_t*>(cache), layers, layers > 1 ? layer_stride : 0, num_pages, page_bytes, page_table,
                     max_pages_per_seq, seq_lens, path, accepted, B, Q, kv_heads, new_lens, dev_status};
  return status_of(launch_kv8_keep(p, head_dim, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ verification
// Workspace: (largest, sum) of every chunk f32 x 2 | sums of what is left f64 | where the largest is i32.
struct VerifyWorkspace {
  size_t sums, at, total;
};
static VerifyWorkspace verify_workspace(int B, int Q, int64_t V) {
  const size_t chunks = (size_t)verify_chunks(V);
  VerifyWorkspace w;
  w.sums = align256((size_t)B * Q * chunks * sizeof(float2));
  w.at = w.sums + align256((size_t)B * verify_entries(V) * sizeof(double));
  w.total = w.at + align256((size_t)B * Q * chunks * sizeof(int32_t));
  return w;
}
static bool verify_sizes_ok(int B, int Q, int64_t V) {
  return B >= 1 && Q >= 1 && Q <= NVFP4MLA_MAX_NODES && V >= 1 && V <= NVFP4MLA_MAX_VOCABULARY;
}

size_t spec_verify_workspace_size(int B, int Q, int64_t V) { return verify_sizes_ok(B, Q, V) ? verify_workspace(B, Q, V).total : 0; }

int spec_verify(const void* logits, int64_t logits_row_stride, int dtype, const float* draft_probs, int64_t probs_row_stride,
                const int32_t* drafts, const int32_t* parents, const float* uniforms, const float* temperatures, int B,
                int Q, int64_t V, int32_t* tokens, int32_t* path, int32_t* accepted, void* workspace, size_t workspace_bytes,
                int32_t* dev_status, void* stream) {
  if (!verify_sizes_ok(B, Q, V) || dtype < NVFP4MLA_BF16 || dtype > NVFP4MLA_FP32) return NVFP4MLA_ERR_INVALID_ARG;
  if (logits_row_stride < 0 || probs_row_stride < 0) return NVFP4MLA_ERR_INVALID_ARG;
  if (B > verify_requests()) return NVFP4MLA_ERR_UNSUPPORTED;
  if (any_null({logits, drafts, parents, uniforms, tokens, path, accepted})) return NVFP4MLA_ERR_INVALID_ARG;
  const VerifyWorkspace w = verify_workspace(B, Q, V);
  if (workspace == nullptr || workspace_bytes < w.total) return NVFP4MLA_ERR_WORKSPACE;
  if (!aligned(logits, dtype == NVFP4MLA_FP32 ? 4 : 2) || !aligned(workspace, 256)) return NVFP4MLA_ERR_ALIGNMENT;
  if (!words_aligned({draft_probs, drafts, parents, uniforms, temperatures, tokens, path, accepted, dev_status})) return NVFP4MLA_ERR_ALIGNMENT;
  if (!all_device({logits, drafts, parents, uniforms, tokens, path, accepted, workspace})) return NVFP4MLA_ERR_INVALID_ARG;
  if (!optional_ok(draft_probs) || !optional_ok(temperatures) || !optional_ok(dev_status)) return NVFP4MLA_ERR_INVALID_ARG;
  // (a request's inputs are read by several CTAs, one of which writes its results)
  const size_t n = (size_t)B * Q * sizeof(int32_t), n1 = (size_t)B * sizeof(int32_t);
  const struct { const void* at; size_t bytes; } out[3] = {{tokens, n}, {path, n}, {accepted, n1}};
  for (int i = 0; i < 3; ++i) {
    if (overlap(out[i].at, out[i].bytes, drafts, n) || overlap(out[i].at, out[i].bytes, parents, n) || overlap(out[i].at, out[i].bytes, uniforms, n) ||
        overlap(out[i].at, out[i].bytes, temperatures, n1) || overlap(out[i].at, out[i].bytes, out[(i + 1) % 3].at, out[(i + 1) % 3].bytes))
      return NVFP4MLA_ERR_INVALID_ARG;
  }
  VerifyParams p{};
  p.chunks = verify_chunks(V);
  if ((int64_t)B * Q > INT32_MAX / p.chunks) return NVFP4MLA_ERR_UNSUPPORTED;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.logits = logits;
  p.row_stride = logits_row_stride;
  p.probs = draft_probs;
  p.probs_stride = probs_row_stride;
  p.drafts = drafts;
  p.parents = parents;
  p.uniforms = uniforms;
  p.temperatures = temperatures;
  p.B = B;
  p.Q = Q;
  p.V = (int)V;
  p.tokens = tokens;
  p.path = path;
  p.accepted = accepted;
  p.status = dev_status;
  p.chunk_ms = reinterpret_cast<float2*>(ws);
  p.entry_sum = reinterpret_cast<double*>(ws + w.sums);
  p.chunk_at = reinterpret_cast<int32_t*>(ws + w.at);
  return status_of(launch_spec_verify(p, dtype, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ pages
static int check_store(const void* cache, int64_t layers, int64_t layer_stride, int64_t num_pages, int64_t page_bytes,
                       PageStore* c) {
  if (num_pages < 1 || num_pages > INT32_MAX || page_bytes < 16 || layers < 1) return NVFP4MLA_ERR_INVALID_ARG;
  if (page_bytes > INT64_MAX / num_pages / layers) return NVFP4MLA_ERR_INVALID_ARG;
  if (cache == nullptr || (layers > 1 && layer_stride < num_pages * page_bytes)) return NVFP4MLA_ERR_INVALID_ARG;
  if (!aligned(cache, 16) || page_bytes % 16 != 0 || (layers > 1 && layer_stride % 16 != 0)) return NVFP4MLA_ERR_ALIGNMENT;
  if (pointer_kind(cache) != kPtrDevice) return NVFP4MLA_ERR_INVALID_ARG;
  *c = PageStore{static_cast<uint8_t*>(const_cast<void*>(cache)), layers, layers > 1 ? layer_stride : 0, page_bytes};
  return NVFP4MLA_OK;
}

static int check_state(int32_t* table, int64_t max_pages, int32_t* lens, bool has_lens, int num_seqs, int32_t* refs,
                       int64_t num_pages, int32_t* status, PageState* s) {
  if (num_seqs < 1 || max_pages < 1 || max_pages > INT32_MAX || num_pages < 1 || num_pages > INT32_MAX) return NVFP4MLA_ERR_INVALID_ARG;
  if (any_null({table, refs}) || (has_lens && lens == nullptr)) return NVFP4MLA_ERR_INVALID_ARG;
  if (!words_aligned({table, lens, status}) || !aligned(refs, 16)) return NVFP4MLA_ERR_ALIGNMENT;
  if (!all_device({table, refs}) || (has_lens && !all_device({lens})) || !optional_ok(status)) return NVFP4MLA_ERR_INVALID_ARG;
  *s = PageState{table, max_pages, lens, num_seqs, refs, num_pages, status};
  return NVFP4MLA_OK;
}

int kv_pages_copy(void* cache, int64_t layers, int64_t layer_stride, int64_t num_pages, int64_t page_bytes,
                  const int32_t* src, const int32_t* dst, int64_t n, int32_t* dev_status, void* stream) {
  if (n < 0) return NVFP4MLA_ERR_INVALID_ARG;
  PageStore c;
  const int rc = check_store(cache, layers, layer_stride, num_pages, page_bytes, &c);
  if (rc != NVFP4MLA_OK || n == 0) return rc;
  if (any_null({src, dst})) return NVFP4MLA_ERR_INVALID_ARG;
  if (!words_aligned({src, dst, dev_status})) return NVFP4MLA_ERR_ALIGNMENT;
  if (!all_device({src, dst}) || !optional_ok(dev_status)) return NVFP4MLA_ERR_INVALID_ARG;
  if (n > INT32_MAX || pages_copy_blocks(c, 1) > INT32_MAX / n) return NVFP4MLA_ERR_UNSUPPORTED;
  return status_of(launch_pages_copy(c, num_pages, src, dst, n, dev_status, static_cast<cudaStream_t>(stream)));
}

int kv_pages_free(int32_t* page_table, int64_t max_pages_per_seq, int32_t* seq_lens, int num_seqs, int32_t* refcounts,
                  int64_t num_pages, const int32_t* seqs, int n, int32_t* dev_status, void* stream) {
  if (n < 0) return NVFP4MLA_ERR_INVALID_ARG;
  PageState s;
  const int rc = check_state(page_table, max_pages_per_seq, seq_lens, true, num_seqs, refcounts, num_pages, dev_status, &s);
  if (rc != NVFP4MLA_OK || n == 0) return rc;
  if (seqs == nullptr) return NVFP4MLA_ERR_INVALID_ARG;
  if (!aligned(seqs, 4)) return NVFP4MLA_ERR_ALIGNMENT;
  if (!all_device({seqs})) return NVFP4MLA_ERR_INVALID_ARG;
  return status_of(launch_pages_free(s, seqs, n, static_cast<cudaStream_t>(stream)));
}

int kv_pages_trim(int32_t* page_table, int64_t max_pages_per_seq, int32_t* seq_lens, int num_seqs, int32_t* refcounts,
                  int64_t num_pages, const int32_t* new_lens, int32_t* dev_status, void* stream) {
  if (new_lens == nullptr) return NVFP4MLA_ERR_INVALID_ARG;
  if (!aligned(new_lens, 4)) return NVFP4MLA_ERR_ALIGNMENT;
  PageState s;
  const int rc = check_state(page_table, max_pages_per_seq, seq_lens, true, num_seqs, refcounts, num_pages, dev_status, &s);
  if (rc != NVFP4MLA_OK) return rc;
  if (!all_device({new_lens})) return NVFP4MLA_ERR_INVALID_ARG;
  // (a warp a sequence: what one reads, no other may write)
  const size_t n = (size_t)num_seqs * sizeof(int32_t);
  if ((new_lens != seq_lens && overlap(new_lens, n, seq_lens, n)) || overlap(new_lens, n, page_table, n * max_pages_per_seq) ||
      overlap(new_lens, n, refcounts, (size_t)num_pages * sizeof(int32_t)))
    return NVFP4MLA_ERR_INVALID_ARG;
  return status_of(launch_pages_trim(s, new_lens, static_cast<cudaStream_t>(stream)));
}

int kv_pages_fork(void* cache, int64_t layers, int64_t layer_stride, int64_t num_pages, int64_t page_bytes,
                  int32_t* page_table, int64_t max_pages_per_seq, int32_t* seq_lens, int num_seqs, int32_t* refcounts,
                  const int32_t* src, const int32_t* dst, int n, int32_t* new_pages, int32_t* dev_status, void* stream) {
  if (n < 0 || n > NVFP4MLA_MAX_REQUESTS) return NVFP4MLA_ERR_INVALID_ARG;
  PageStore c;
  PageState s;
  int rc = check_store(cache, layers, layer_stride, num_pages, page_bytes, &c);
  if (rc != NVFP4MLA_OK) return rc;
  rc = check_state(page_table, max_pages_per_seq, seq_lens, true, num_seqs, refcounts, num_pages, dev_status, &s);
  if (rc != NVFP4MLA_OK || n == 0) return rc;
  if (any_null({src, dst, new_pages})) return NVFP4MLA_ERR_INVALID_ARG;
  if (!words_aligned({src, dst, new_pages})) return NVFP4MLA_ERR_ALIGNMENT;
  if (!all_device({src, dst, new_pages})) return NVFP4MLA_ERR_INVALID_ARG;
  if (pages_copy_blocks(c, 1) + max_pages_per_seq > INT32_MAX / n) return NVFP4MLA_ERR_UNSUPPORTED;
  return status_of(launch_pages_fork(s, c, src, dst, n, new_pages, static_cast<cudaStream_t>(stream)));
}

int kv_pages_extend(int32_t* page_table, int64_t max_pages_per_seq, int32_t* seq_lens, int num_seqs,
                    int32_t* refcounts, int64_t num_pages, const int32_t* add, int32_t* granted, int32_t* dev_status,
                    void* stream) {
  if (num_seqs > NVFP4MLA_MAX_REQUESTS) return NVFP4MLA_ERR_INVALID_ARG;
  PageState s;
  const int rc = check_state(page_table, max_pages_per_seq, seq_lens, true, num_seqs, refcounts, num_pages, dev_status, &s);
  if (rc != NVFP4MLA_OK) return rc;
  if (add == nullptr) return NVFP4MLA_ERR_INVALID_ARG;
  if (!words_aligned({add, granted})) return NVFP4MLA_ERR_ALIGNMENT;
  if (!all_device({add}) || !optional_ok(granted)) return NVFP4MLA_ERR_INVALID_ARG;
  return status_of(launch_pages_extend(s, add, granted, static_cast<cudaStream_t>(stream)));
}

size_t kv_pages_compact_workspace_size(int64_t num_pages) {
  if (num_pages < 1 || num_pages > INT32_MAX) return 0;
  return ((size_t)(2 * ((num_pages / 2 + 4) / 4 * 4) + 4) * 4 + 255) / 256 * 256;
}

int kv_pages_compact(void* cache, int64_t layers, int64_t layer_stride, int64_t num_pages, int64_t page_bytes,
                     int32_t* page_table, int64_t max_pages_per_seq, int num_seqs, int32_t* refcounts, int32_t* remap,
                     int32_t* num_live, void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  PageStore c;
  PageState s;
  int rc = check_store(cache, layers, layer_stride, num_pages, page_bytes, &c);
  if (rc != NVFP4MLA_OK) return rc;
  rc = check_state(page_table, max_pages_per_seq, nullptr, false, num_seqs, refcounts, num_pages, dev_status, &s);
  if (rc != NVFP4MLA_OK) return rc;
  if (any_null({remap, num_live})) return NVFP4MLA_ERR_INVALID_ARG;
  if (workspace == nullptr || workspace_bytes < kv_pages_compact_workspace_size(num_pages)) return NVFP4MLA_ERR_WORKSPACE;
  if (!words_aligned({remap, num_live}) || !aligned(workspace, 256)) return NVFP4MLA_ERR_ALIGNMENT;
  if (!all_device({remap, num_live, workspace})) return NVFP4MLA_ERR_INVALID_ARG;
  return status_of(launch_pages_compact(s, c, remap, num_live, static_cast<int32_t*>(workspace), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
