// C ABI of a decoding step's calls: host-side validation and launches.  Every check runs before
// any HIP call.
#include "checks.h"
#include "decode.h"

namespace {

using namespace wf;

constexpr int32_t kMaxHeads = 4096;  // of rows that are turned
constexpr int32_t kMaxGiven = 65536;

int32_t check_rotary_rows(const wf_rotary_rows* r, int32_t dtype, int64_t rows, int32_t head_dim) {
  if (r->heads < 1 || r->heads > kMaxHeads) return WF_ERR_SHAPE;
  const int64_t width = static_cast<int64_t>(r->heads) * head_dim;
  const int32_t s = check_vectors(r->x, dtype, rows, width, r->stride);
  if (s != WF_OK) return s;
  if (r->x == r->out && r->out && r->stride != r->out_stride) return WF_ERR_SHAPE;
  return check_vectors(r->out, dtype, rows, width, r->out_stride);
}

int32_t check_cache8(const wf_page_cache8* c) {
  if (!c) return WF_ERR_NULL;
  if (c->pages.dtype != WF_E4M3) return WF_ERR_DTYPE;
  const int32_t s = check_pages(&c->pages, 1);
  if (s != WF_OK) return s;
  if (c->block < 1 || c->block > c->pages.page_size || (c->block & (c->block - 1)) != 0)
    return WF_ERR_SHAPE;
  const int64_t page = static_cast<int64_t>(c->pages.heads) * (c->pages.page_size / c->block);
  if (c->scale_page_stride < page || c->scale_page_stride > INT64_MAX / 16 / c->pages.pages ||
      (c->pages.layers > 1 && (c->scale_layer_stride < page ||
                               c->scale_layer_stride > INT64_MAX / 16 / c->pages.layers)))
    return WF_ERR_SHAPE;
  if (!c->k_scale || !c->v_scale) return WF_ERR_NULL;
  return WF_OK;
}

int32_t check_cache8_rows(const wf_page_cache8* cache, const wf_round_rows* rows, int64_t* total,
                          RowsArgs* out) {
  int32_t s = check_cache8(cache);
  if (s != WF_OK) return s;
  if ((s = check_sizes(rows, total)) != WF_OK) return s;
  if (rows->B == 0) return WF_OK;
  if ((s = check_pointers(rows, false)) != WF_OK) return s;
  *out = rows_args(rows, *total);
  if (static_cast<int64_t>(rows->B) * out->rmax > kMaxBlocks) return WF_ERR_SHAPE;
  return WF_OK;
}

}  // namespace

extern "C" {

int32_t whiflash_rotate(const wf_rotary* rotary, int32_t dtype, int32_t head_dim,
                        const wf_round_rows* rows, const int32_t* seq, const int32_t* context,
                        int32_t seqs, const wf_rotary_rows* q, const wf_rotary_rows* k,
                        hipStream_t stream) {
  if (!rotary || !q) return WF_ERR_NULL;
  if (!valid_dtype(dtype)) return WF_ERR_DTYPE;
  if (head_dim < 2 || head_dim > WHIFLASH_MAX_ROTARY_DIM || head_dim * elem_bytes(dtype) % 16 != 0 ||
      rotary->pairs < 1 || rotary->pairs > head_dim / 2 ||
      (rotary->layout != WF_ROTARY_HALF && rotary->layout != WF_ROTARY_INTERLEAVED) ||
      !isfinite(rotary->magnitude) || seqs < 0)
    return WF_ERR_SHAPE;
  int64_t total = 0;
  int32_t s = check_sizes(rows, &total);
  if (s != WF_OK) return s;
  if ((s = check_rotary_rows(q, dtype, total, head_dim)) != WF_OK) return s;
  if (k && (s = check_rotary_rows(k, dtype, total, head_dim)) != WF_OK) return s;
  if (rows->B == 0 || total == 0) return WF_OK;
  if ((s = check_pointers(rows, false)) != WF_OK) return s;
  if (!rotary->frequency || !context) return WF_ERR_NULL;
  const RowsArgs a = rows_args(rows, total);
  if (static_cast<int64_t>(rows->B) * a.rmax > kMaxBlocks) return WF_ERR_SHAPE;
  return launch_status(launch_rotate(*rotary, dtype, head_dim, a, seq, context, seqs, *q, k, stream));
}

int32_t whiflash_cache8_append(const wf_page_cache8* cache, int32_t layer,
                               const wf_round_rows* rows, const int32_t* seq, int32_t dtype,
                               const void* k_rows, int64_t k_row_stride, const void* v_rows,
                               int64_t v_row_stride, hipStream_t stream) {
  int64_t total = 0;
  RowsArgs a{};
  int32_t s = check_cache8_rows(cache, rows, &total, &a);
  if (s != WF_OK) return s;
  if (!valid_dtype(dtype)) return WF_ERR_DTYPE;
  if (layer < 0 || layer >= cache->pages.layers) return WF_ERR_SHAPE;
  const int64_t width = static_cast<int64_t>(cache->pages.heads) * cache->pages.head_dim;
  if ((s = check_vectors(k_rows, dtype, total, width, k_row_stride)) != WF_OK) return s;
  if ((s = check_vectors(v_rows, dtype, total, width, v_row_stride)) != WF_OK) return s;
  if (rows->B == 0 || total == 0) return WF_OK;
  if (cache8_append_blocks(*cache, a) > kMaxBlocks) return WF_ERR_SHAPE;
  return launch_status(launch_cache8_append(*cache, layer, a, seq, dtype, k_rows, k_row_stride,
                                            v_rows, v_row_stride, stream));
}

int32_t whiflash_cache8_read(const wf_page_cache8* cache, int32_t layer, int32_t B,
                             const int32_t* seq, const int32_t* first, int32_t count,
                             int32_t pending, int32_t dtype, void* k_out, void* v_out,
                             hipStream_t stream) {
  const int32_t s = check_cache8(cache);
  if (s != WF_OK) return s;
  if (!valid_dtype(dtype)) return WF_ERR_DTYPE;
  if (layer < 0 || layer >= cache->pages.layers || B < 0 || count < 0 || count > kMaxPositions ||
      pending < 0 || pending > kMaxPositions)
    return WF_ERR_SHAPE;
  if (B == 0 || count == 0 || (!k_out && !v_out)) return WF_OK;
  if (!aligned16(k_out) || !aligned16(v_out)) return WF_ERR_ALIGN;
  if (cache8_read_blocks(B, count) > kMaxBlocks) return WF_ERR_SHAPE;
  return launch_status(launch_cache8_read(*cache, layer, B, seq, first, count, pending, dtype, k_out,
                                          v_out, stream));
}

int32_t whiflash_cache8_compact(const wf_page_cache8* cache, const wf_round_rows* rows,
                                const int32_t* seq, const int32_t* accept_len,
                                const int32_t* best_node, int32_t* next_context,
                                hipStream_t stream) {
  int64_t total = 0;
  RowsArgs a{};
  const int32_t s = check_cache8_rows(cache, rows, &total, &a);
  if (s != WF_OK) return s;
  if (rows->B == 0) return WF_OK;
  if (!accept_len || (rows->kind != WF_ROWS_CHAIN && !best_node)) return WF_ERR_NULL;
  return launch_status(launch_cache8_compact(*cache, a, seq, accept_len, best_node, next_context,
                                             stream));
}

int32_t whiflash_cache8_fork(const wf_page_cache8* cache, int32_t n, const int32_t* src,
                             const int32_t* dst, int32_t* status, void* workspace,
                             size_t workspace_bytes, hipStream_t stream) {
  int32_t s = check_cache8(cache);
  if (s != WF_OK) return s;
  if (n < 0 || n > kMaxBlocks) return WF_ERR_SHAPE;
  if (n == 0) return WF_OK;
  if (!src || !dst || !status) return WF_ERR_NULL;
  if ((s = check_workspace(workspace, workspace_bytes,
                           whiflash_cache_pages_workspace_bytes(&cache->pages, n))) != WF_OK)
    return s;
  return launch_status(launch_cache8_fork(*cache, n, src, dst, status,
                                          static_cast<int32_t*>(workspace), stream));
}

size_t whiflash_attend8_workspace_bytes(const wf_page_cache8* cache, const wf_round_rows* rows,
                                        int32_t dtype, int32_t q_heads, int32_t max_context) {
  int64_t total = 0;
  RowsArgs a{};
  if (check_cache8_rows(cache, rows, &total, &a) != WF_OK || rows->B == 0 || !valid_dtype(dtype) ||
      !attend_sizes_ok(&cache->pages, q_heads, max_context))
    return 0;
  return round_up(attend8_workspace(*cache, a, dtype, q_heads, max_context, total), kWorkspaceAlign);
}

int32_t whiflash_attend8(const void* q, int64_t q_row_stride, int32_t q_heads, int32_t dtype,
                         const wf_page_cache8* cache, int32_t layer, const wf_round_rows* rows,
                         const int32_t* seq, int32_t max_context, float scale, void* out,
                         void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int64_t total = 0;
  RowsArgs a{};
  int32_t s = check_cache8_rows(cache, rows, &total, &a);
  if (s != WF_OK) return s;
  if (!valid_dtype(dtype)) return WF_ERR_DTYPE;
  if (layer < 0 || layer >= cache->pages.layers ||
      !attend_sizes_ok(&cache->pages, q_heads, max_context) || !isfinite(scale))
    return WF_ERR_SHAPE;
  const int64_t width = static_cast<int64_t>(q_heads) * cache->pages.head_dim;
  if ((s = check_vectors(q, dtype, total, width, q_row_stride)) != WF_OK) return s;
  if (rows->B == 0 || total == 0) return WF_OK;
  if (!out) return WF_ERR_NULL;
  if (!aligned16(out)) return WF_ERR_ALIGN;
  if (attend8_blocks(*cache, a, dtype, q_heads, max_context) > kMaxBlocks ||
      static_cast<int64_t>(a.B) * a.rmax * q_heads > kMaxBlocks * 4)
    return WF_ERR_SHAPE;
  if ((s = check_workspace(workspace, workspace_bytes,
                           whiflash_attend8_workspace_bytes(cache, rows, dtype, q_heads, max_context))) != WF_OK)
    return s;
  return launch_status(launch_attend8(q, q_row_stride, q_heads, dtype, *cache, layer, a, seq,
                                      max_context, scale, out, workspace, total, stream));
}

size_t whiflash_token_logprobs_workspace_bytes(int32_t n, int32_t V, int32_t top) {
  if (n <= 0 || n > kMaxBlocks || V <= 0 || V > kMaxVocab || top < 0 || top > WHIFLASH_MAX_TOP) return 0;
  return round_up(logprobs_workspace(n, V, top), kWorkspaceAlign);
}

int32_t whiflash_token_logprobs(const void* logits, int32_t dtype, int32_t total_rows, int32_t V,
                                int64_t row_stride, int32_t n, const int32_t* rows, int32_t given,
                                const int32_t* tokens, int32_t top, float* logprob, float* entropy,
                                int32_t* top_tokens, float* top_logprobs, void* workspace,
                                size_t workspace_bytes, hipStream_t stream) {
  if (total_rows < 0) return WF_ERR_SHAPE;
  int32_t s = check_matrix(logits, dtype, total_rows, V, row_stride);
  if (s != WF_OK) return s;
  if (n < 0 || n > kMaxBlocks || (!rows && n > total_rows) || given < 0 || given > kMaxGiven ||
      top < 0 || top > WHIFLASH_MAX_TOP)
    return WF_ERR_SHAPE;
  if (n == 0) return WF_OK;
  if (given > 0 && (!tokens || !logprob)) return WF_ERR_NULL;
  if (top > 0 && (!top_tokens || !top_logprobs)) return WF_ERR_NULL;
  if (static_cast<int64_t>(n) * logprobs_plan(dtype, n, V).chunks > kMaxBlocks) return WF_ERR_SHAPE;
  if ((s = check_workspace(workspace, workspace_bytes,
                           whiflash_token_logprobs_workspace_bytes(n, V, top))) != WF_OK)
    return s;
  return launch_status(launch_logprobs(logits, dtype, total_rows, V, row_stride, n, rows, given,
                                       tokens, top, logprob, entropy, top_tokens, top_logprobs,
                                       workspace, stream));
}

}  // extern "C"
