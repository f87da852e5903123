// C ABI of the calls around a round: host-side validation and launches.  As in
// api.hip, every check runs before any HIP call.
#include "checks.h"

namespace {

using namespace wf;

int32_t check_history(const uint16_t* h, int32_t slots, int32_t V, int64_t stride) {
  if (slots < 0 || V <= 0 || V > kMaxVocab || stride < V || stride > INT64_MAX / 4 / (slots > 0 ? slots : 1))
    return WF_ERR_SHAPE;
  if (slots > 0 && !h) return WF_ERR_NULL;
  if (!aligned16(h) || stride % 8 != 0) return WF_ERR_ALIGN;
  return WF_OK;
}

int32_t check_rules(const wf_logit_rules* r, int64_t rows, int32_t V) {
  if (!r) return WF_ERR_NULL;
  if (r->history) {
    const int32_t s = check_history(r->history, r->slots, V, r->history_stride);
    if (s != WF_OK) return s;
  }
  if (r->bias_offsets) {
    if (r->bias_count < 0) return WF_ERR_SHAPE;
    if (r->bias_count > 0 && (!r->bias_ids || !r->bias_values)) return WF_ERR_NULL;
  }
  if (r->allow && (r->allow_stride < (static_cast<int64_t>(V) + 31) / 32 ||
                   r->allow_stride > INT64_MAX / 16 / (rows > 0 ? rows : 1)))
    return WF_ERR_SHAPE;
  if (r->allow && reinterpret_cast<uintptr_t>(r->allow) % 4 != 0) return WF_ERR_ALIGN;
  return WF_OK;
}

// Checks shared by the two calls that apply rules.
int32_t check_ruled(const void* logits, int32_t dtype, int32_t V, int64_t row_stride,
                    const wf_round_rows* rows, const wf_logit_rules* rules, wf::RowsArgs* out) {
  int64_t total = 0;
  int32_t s = check_sizes(rows, &total);
  if (s != WF_OK) return s;
  if ((s = check_matrix(logits, dtype, total, V, row_stride)) != WF_OK) return s;
  if (rows->B == 0) return WF_OK;
  if ((s = check_pointers(rows, true)) != WF_OK) return s;
  if ((s = check_rules(rules, total, V)) != WF_OK) return s;
  *out = rows_args(rows, total);
  const wf::RulesPlan p = wf::rules_plan(dtype, rows->B, out->rmax, V);
  if (static_cast<int64_t>(rows->B) * p.groups * p.chunks > kMaxBlocks) return WF_ERR_SHAPE;
  return WF_OK;
}

}  // namespace

extern "C" {

int32_t whiflash_process_logits(const void* logits, int32_t dtype, int32_t V, int64_t row_stride,
                                const wf_round_rows* rows, const wf_logit_rules* rules, void* out,
                                int32_t out_dtype, int64_t out_stride, hipStream_t stream) {
  wf::RowsArgs a{};
  int32_t s = check_ruled(logits, dtype, V, row_stride, rows, rules, &a);
  if (s != WF_OK) return s;
  int64_t total = 0;
  check_sizes(rows, &total);
  if ((s = check_matrix(out, out_dtype, total, V, out_stride)) != WF_OK) return s;
  if (out == logits && out && (out_dtype != dtype || out_stride != row_stride)) return WF_ERR_SHAPE;
  if (rows->B == 0 || total == 0) return WF_OK;
  return launch_status(wf::launch_process(a, *rules, logits, dtype, V, row_stride, out, out_dtype,
                                          out_stride, stream));
}

size_t whiflash_verify_constrained_workspace_bytes(const wf_round_rows* rows, int32_t V) {
  int64_t total = 0;
  if (V <= 0 || V > kMaxVocab || check_sizes(rows, &total) != WF_OK || rows->B == 0) return 0;
  const wf::RowsArgs a = rows_args(rows, total);
  // The chunk count depends on the element type: the larger of the two.
  size_t most = 0;
  for (int32_t dtype : {WF_F32, WF_BF16}) {
    const wf::RulesPlan p = wf::rules_plan(dtype, rows->B, a.rmax, V);
    const size_t n = static_cast<size_t>(rows->B) * a.rmax * p.chunks * sizeof(wf::Partial);
    most = n > most ? n : most;
  }
  return round_up(most, kWorkspaceAlign);
}

int32_t whiflash_verify_constrained(const void* logits, int32_t dtype, int32_t V,
                                    int64_t row_stride, const wf_round_rows* rows,
                                    const wf_logit_rules* rules, int32_t* accept_len,
                                    int32_t* bonus, int32_t* best_node, int32_t* row_argmax,
                                    void* workspace, size_t workspace_bytes, hipStream_t stream) {
  wf::RowsArgs a{};
  int32_t s = check_ruled(logits, dtype, V, row_stride, rows, rules, &a);
  if (s != WF_OK) return s;
  if (rows->B == 0) return WF_OK;
  if (!accept_len || !bonus) return WF_ERR_NULL;
  if ((s = check_workspace(workspace, workspace_bytes,
                           whiflash_verify_constrained_workspace_bytes(rows, V))) != WF_OK)
    return s;
  return launch_status(wf::launch_constrained(a, *rules, logits, dtype, V, row_stride,
                                              static_cast<wf::Partial*>(workspace), accept_len,
                                              bonus, best_node, row_argmax, stream));
}

int32_t whiflash_history_prompt(uint16_t* history, int32_t slots, int32_t V, int64_t history_stride,
                                int32_t B, const int32_t* slot, const int32_t* tokens,
                                const int32_t* offsets, int32_t count, hipStream_t stream) {
  const int32_t s = check_history(history, slots, V, history_stride);
  if (s != WF_OK) return s;
  if (B < 0 || B > kMaxBlocks / 16 || count < 0) return WF_ERR_SHAPE;
  if (B == 0 || count == 0) return WF_OK;
  if (!tokens || !offsets) return WF_ERR_NULL;
  return launch_status(wf::launch_history_prompt(history, slots, V, history_stride, B, slot, tokens,
                                                 offsets, count, stream));
}

int32_t whiflash_history_update(uint16_t* history, int32_t slots, int32_t V, int64_t history_stride,
                                const wf_round_rows* rows, const int32_t* slot,
                                const int32_t* accept_len, const int32_t* best_node,
                                const int32_t* bonus, hipStream_t stream) {
  int32_t s = check_history(history, slots, V, history_stride);
  if (s != WF_OK) return s;
  int64_t total = 0;
  if ((s = check_sizes(rows, &total)) != WF_OK) return s;
  if (rows->B == 0) return WF_OK;
  if (rows->B > kMaxBlocks) return WF_ERR_SHAPE;
  if ((s = check_pointers(rows, true)) != WF_OK) return s;
  if (!accept_len || !bonus || (rows->kind != WF_ROWS_CHAIN && !best_node)) return WF_ERR_NULL;
  return launch_status(wf::launch_history_update(history, slots, V, history_stride,
                                                 rows_args(rows, total), slot, accept_len,
                                                 best_node, bonus, stream));
}

int32_t whiflash_cache_append(const wf_page_cache* cache, int32_t layer, const wf_round_rows* rows,
                              const int32_t* seq, const void* k_rows, int64_t k_row_stride,
                              const void* v_rows, int64_t v_row_stride, hipStream_t stream) {
  int64_t total = 0;
  wf::RowsArgs a{};
  int32_t s = check_cache_rows(cache, rows, &total, &a);
  if (s != WF_OK) return s;
  if (layer < 0 || layer >= cache->layers) return WF_ERR_SHAPE;
  const int64_t width = static_cast<int64_t>(cache->heads) * cache->head_dim;
  if ((s = check_vectors(k_rows, cache->dtype, total, width, k_row_stride)) != WF_OK) return s;
  if ((s = check_vectors(v_rows, cache->dtype, total, width, v_row_stride)) != WF_OK) return s;
  if (rows->B == 0 || total == 0) return WF_OK;
  return launch_status(wf::launch_cache_append(*cache, layer, a, seq, k_rows, k_row_stride, v_rows,
                                               v_row_stride, stream));
}

size_t whiflash_attend_workspace_bytes(const wf_page_cache* cache, const wf_round_rows* rows,
                                       int32_t q_heads, int32_t max_context) {
  int64_t total = 0;
  wf::RowsArgs a{};
  if (check_cache_rows(cache, rows, &total, &a) != WF_OK || rows->B == 0 ||
      !attend_sizes_ok(cache, q_heads, max_context))
    return 0;
  return round_up(wf::attend_workspace(*cache, a, q_heads, max_context, total), kWorkspaceAlign);
}

int32_t whiflash_attend(const void* q, int64_t q_row_stride, int32_t q_heads,
                        const wf_page_cache* cache, int32_t layer, const wf_round_rows* rows,
                        const int32_t* seq, int32_t max_context, float scale, void* out,
                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int64_t total = 0;
  wf::RowsArgs a{};
  int32_t s = check_cache_rows(cache, rows, &total, &a);
  if (s != WF_OK) return s;
  if (layer < 0 || layer >= cache->layers || !attend_sizes_ok(cache, q_heads, max_context) ||
      !isfinite(scale))
    return WF_ERR_SHAPE;
  const int64_t width = static_cast<int64_t>(q_heads) * cache->head_dim;
  if ((s = check_vectors(q, cache->dtype, total, width, q_row_stride)) != WF_OK) return s;
  if (rows->B == 0 || total == 0) return WF_OK;
  if (!out) return WF_ERR_NULL;
  if (!aligned16(out)) return WF_ERR_ALIGN;
  if (wf::attend_blocks(*cache, a, q_heads, max_context) > kMaxBlocks ||
      static_cast<int64_t>(a.B) * a.rmax * q_heads > kMaxBlocks * 4)
    return WF_ERR_SHAPE;
  if ((s = check_workspace(workspace, workspace_bytes,
                           whiflash_attend_workspace_bytes(cache, rows, q_heads, max_context))) !=
      WF_OK)
    return s;
  return launch_status(wf::launch_attend(q, q_row_stride, q_heads, *cache, layer, a, seq,
                                         max_context, scale, out, workspace, total, stream));
}

int32_t whiflash_cache_compact(const wf_page_cache* cache, const wf_round_rows* rows,
                               const int32_t* seq, const int32_t* accept_len,
                               const int32_t* best_node, int32_t* next_context,
                               hipStream_t stream) {
  int64_t total = 0;
  wf::RowsArgs a{};
  int32_t s = check_cache_rows(cache, rows, &total, &a);
  if (s != WF_OK) return s;
  if (rows->B == 0) return WF_OK;
  if (!accept_len || (rows->kind != WF_ROWS_CHAIN && !best_node)) return WF_ERR_NULL;
  return launch_status(wf::launch_cache_compact(*cache, a, seq, accept_len, best_node, next_context,
                                                stream));
}

size_t whiflash_cache_pages_workspace_bytes(const wf_page_cache* cache, int32_t n) {
  if (check_bookkeeping(cache) != WF_OK || n <= 0) return 0;
  return round_up(wf::pages_workspace_words(*cache, n) * sizeof(int32_t), kWorkspaceAlign);
}

int32_t whiflash_cache_fork(const wf_page_cache* cache, int32_t n, const int32_t* src,
                            const int32_t* dst, int32_t* status, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
  int32_t s = check_cache(cache);
  if (s != WF_OK) return s;
  if (n < 0 || n > kMaxBlocks) return WF_ERR_SHAPE;
  if (n == 0) return WF_OK;
  if (!src || !dst || !status) return WF_ERR_NULL;
  if ((s = check_workspace(workspace, workspace_bytes,
                           whiflash_cache_pages_workspace_bytes(cache, n))) != WF_OK)
    return s;
  return launch_status(wf::launch_cache_fork(*cache, n, src, dst, status,
                                             static_cast<int32_t*>(workspace), stream));
}

int32_t whiflash_cache_reserve(const wf_page_cache* cache, int32_t n, const int32_t* seq,
                               const int32_t* count, int32_t* status, void* workspace,
                               size_t workspace_bytes, hipStream_t stream) {
  int32_t s = check_bookkeeping(cache);
  if (s != WF_OK) return s;
  if (n < 0 || n > kMaxBlocks) return WF_ERR_SHAPE;
  if (n == 0) return WF_OK;
  if (!seq || !count || !status) return WF_ERR_NULL;
  if ((s = check_workspace(workspace, workspace_bytes,
                           whiflash_cache_pages_workspace_bytes(cache, n))) != WF_OK)
    return s;
  return launch_status(wf::launch_cache_reserve(*cache, n, seq, count, status,
                                                static_cast<int32_t*>(workspace), stream));
}

int32_t whiflash_cache_free(const wf_page_cache* cache, int32_t n, const int32_t* seq,
                            hipStream_t stream) {
  const int32_t s = check_bookkeeping(cache);
  if (s != WF_OK) return s;
  if (n < 0 || n > kMaxBlocks) return WF_ERR_SHAPE;
  if (n == 0) return WF_OK;
  if (!seq) return WF_ERR_NULL;
  return launch_status(wf::launch_cache_free(*cache, n, seq, stream));
}

}  // extern "C"
