// Internal launch interface between the C ABI (api.cu) and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

namespace mla {

// Launch `kern` as a programmatic dependent of the previous work in `stream`:
// its blocks may be scheduled while that work drains, and the kernel itself
// waits (griddepcontrol.wait) before reading anything.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                             Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// Return fn<bits_c, group_c, bits_r, group_r>(...) for the cache format of launch description L
// (falls through when the format is none of the sixteen).
#define MLA_FORMAT_CASE(L, fn, BC, GC, BR, GR, ...)                                            \
  if ((L).bits_c == BC && (L).group_c == GC && (L).bits_r == BR && (L).group_r == GR)        \
    return fn<BC, GC, BR, GR>(__VA_ARGS__);
#define MLA_FORMAT_CASES_R(L, fn, BC, GC, ...)                                                  \
  MLA_FORMAT_CASE(L, fn, BC, GC, 4, 64, __VA_ARGS__)                                            \
  MLA_FORMAT_CASE(L, fn, BC, GC, 4, 32, __VA_ARGS__)                                            \
  MLA_FORMAT_CASE(L, fn, BC, GC, 2, 64, __VA_ARGS__)                                            \
  MLA_FORMAT_CASE(L, fn, BC, GC, 2, 32, __VA_ARGS__)
#define MLA_FORMAT_DISPATCH(L, fn, ...)                                                         \
  MLA_FORMAT_CASES_R(L, fn, 4, 64, __VA_ARGS__)                                                 \
  MLA_FORMAT_CASES_R(L, fn, 4, 32, __VA_ARGS__)                                                 \
  MLA_FORMAT_CASES_R(L, fn, 2, 64, __VA_ARGS__)                                                 \
  MLA_FORMAT_CASES_R(L, fn, 2, 32, __VA_ARGS__)

struct AppendLaunch {
  void* pool;
  int num_pages;
  const int32_t* table;
  int max_pages;
  const int32_t* lens_before;
  const void* c_new;
  const void* kr_new;
  int B, n_new;
  int bits_c, group_c, bits_r, group_r;
  // optional token source for the quantized append: row j of BF16 page
  // src_pages[b] of src_pool ([pages][64][576]) instead of c_new / kr_new
  const void* src_pool;
  int src_num_pages;
  const int32_t* src_pages;
  int* status;
  cudaStream_t stream;
  // position of new token j of request b: lens_before[b] + lens_offset + j
  // (-n_new when the lengths passed already count the new tokens)
  int lens_offset;
};

cudaError_t launch_qcache_append(const AppendLaunch& L);
cudaError_t launch_bf16cache_append(const AppendLaunch& L);

// Norm + rotation + quantized append of new tokens, and the rotation of their queries.
struct NormRopeLaunch {
  void* pool;
  int num_pages;
  const int32_t* table;
  int max_pages;
  const int32_t* lens_before;
  const int32_t* new_lens;  // or null: every request has n_new tokens
  const void* kv;           // bf16 rows [B * n_new], kv_stride elements apart
  int64_t kv_stride;
  const void* norm_weight;  // bf16 [512] or null
  float eps;
  const void* q;            // bf16; (token, head) at token * q_token_stride + head * q_head_stride
  int64_t q_token_stride, q_head_stride;
  int H;                    // 0: no queries
  void* q_out;              // bf16 [B * n_new, H, 64]
  const float* cos_sin;     // [max_positions][64]
  int max_positions;
  const int32_t* positions;  // [B * n_new] or null
  int half_pairs;
  void* rows_out;  // bf16 [B * n_new, 576] or null
  int B, n_new;
  int bits_c, group_c, bits_r, group_r;
  int* status;
  cudaStream_t stream;
};
cudaError_t launch_norm_rope_append(const NormRopeLaunch& L);

// Dequantized rows of a token range of every request.
struct ReadLaunch {
  const void* pool;
  int num_pages;
  const int32_t* table;
  int max_pages;
  const int32_t* start;  // or null: 0
  const int32_t* cu_rows;
  int max_rows;
  int64_t total_rows;
  void* out_c;
  int64_t c_stride;
  void* out_kr;
  int64_t kr_stride;
  int B;
  int bits_c, group_c, bits_r, group_r;
  int sms;  // of the device
  int* status;
  cudaStream_t stream;
};
cudaError_t launch_qcache_read(const ReadLaunch& L);

// Mean keys of the pages that an append completed.
struct DigestLaunch {
  const void* pool;
  int num_pages;
  const int32_t* table;
  int max_pages;
  const int32_t* lens_before;
  const int32_t* new_lens;  // or null: n_new each
  int n_new;
  void* digests;
  int B;
  int bits_c, group_c, bits_r, group_r;
  int sms;  // of the device
  int* status;
  cudaStream_t stream;
};
cudaError_t launch_page_digest(const DigestLaunch& L);

// Scores of the candidate pages, and the selection by them.
struct PageScoresLaunch {
  const void* digests;
  int num_pages;
  const int32_t* table;
  int max_pages;
  const int32_t* seq_lens;
  int max_seq_len;
  const void* q_c;
  const void* q_r;
  int B, s_q, H;
  float scale;
  float* scores;  // [B, s_q, width]
  int width;
  int* status;
  cudaStream_t stream;
};
constexpr int kScoreHeads = 128;  // most heads a scores call takes
cudaError_t launch_page_scores(const PageScoresLaunch& L);

struct PageSelectLaunch {
  const int32_t* table;
  int max_pages;
  const int32_t* seq_lens;
  int max_seq_len;
  const float* scores;  // [B, s_q, width]; null when k_pages >= width
  int width;
  int B, s_q, k_pages, n_sink, n_recent;
  int32_t* sel_table;
  int32_t* sel_pages;  // or null
  int32_t* sel_lens;
  int* status;
  cudaStream_t stream;
};
cudaError_t launch_page_select(const PageSelectLaunch& L);

// One decode call, after validation and split planning.
struct DecodeLaunch {
  const void* pool;
  bool quantized;
  int bits_c, group_c, bits_r, group_r;
  int num_pages;
  const int32_t* table;
  int max_pages;
  const int32_t* seq_lens;
  int max_seq_len;
  const void* q_c;
  const void* q_r;
  int B, s_q, H;
  float scale;
  int n_split, chunk_pages;
  float* o_part;   // workspace (n_split > 1)
  float* lse_part;
  void* out;
  int out_f32;
  float* lse;
  unsigned flags;
  int* status;
  cudaStream_t stream;
  // fused append (tensor-core and small-row kernels): bf16 c_new [B, n_new, 512] and
  // kr_new [B, n_new, 64] are the last n_new of seq_lens[b] positions; each
  // unit quantizes those in its key range into the pool before reading it
  const void* c_new;
  const void* kr_new;
  int n_new;
  // tensor-core kernel with a split plan over a multi-wave grid: the order in
  // which clusters take their units (unit indices, longest first), built on
  // the device by launch_plan_units in the caller's workspace; null: index order
  int* worklist;
};

struct DecodeArgs;
DecodeArgs make_decode_args(const DecodeLaunch& L);

cudaError_t launch_decode_simt(const DecodeLaunch& L);
// out = log-sum-exp merge of two normalised partial results (fp32 [rows][512]
// each, natural-log lse; -inf carries weight 0), as bf16 (out_f32 = 0) or fp32.
cudaError_t launch_merge2(const float* o_a, const float* l_a, const float* o_b, const float* l_b, int rows,
                          void* out, int out_f32, float* lse, cudaStream_t stream);
cudaError_t launch_combine(const DecodeLaunch& L);
// Largest chunk (in pages) a work list handles: the split planner's cap.
constexpr int kMaxWorklistChunkPages = 128;
// Fill L.worklist (when set) with the tensor-core kernel's unit indices,
// longest unit first (one block; launched as a programmatic dependent).
cudaError_t launch_plan_units(const DecodeLaunch& L, int row_tiles);
// Returns cudaErrorNotSupported when the tensor-core kernel has no variant for
// the shape; the caller then uses the SIMT kernel.
cudaError_t launch_decode_tc(const DecodeLaunch& L);
// Warp-level MMA kernels for s_q * H <= 16 rows (quantized: INT4 g64 content
// and RoPE; or the BF16 cache); cudaErrorNotSupported for other shapes and formats.
cudaError_t launch_decode_small(const DecodeLaunch& L);
bool decode_small_supported(const DecodeLaunch& L);
// Warp-level MMA kernel for s_q * H <= 16 rows over the BF16 comparison cache.
cudaError_t launch_decode_small_bf16(const DecodeLaunch& L);
bool decode_small_bf16_supported(const DecodeLaunch& L);
// Query rows up to which a decode unit is one CTA of the small-row kernel.
constexpr int kSmallRows = 16;

}  // namespace mla
