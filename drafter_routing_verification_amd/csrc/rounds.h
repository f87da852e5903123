// Launches of the calls around a round (rules.hip, history.hip, attend.hip, pages.hip).
#pragma once

#include "common.h"
#include "rows.h"

namespace wf {

// How the rules' kernel cuts a round: chunks of a row's vocabulary, and groups of
// `group` rows of a sequence that one workgroup takes one after the other.
struct RulesPlan {
  int32_t chunks, groups, group;
};

RulesPlan rules_plan(int dtype, int32_t B, int32_t rmax, int32_t V);
hipError_t launch_process(const RowsArgs& rows, const wf_logit_rules& rules, const void* logits,
                          int dtype, int32_t V, int64_t row_stride, void* out, int out_dtype,
                          int64_t out_stride, hipStream_t stream);
// Partials [B * rmax][chunks], then the acceptance.
hipError_t launch_constrained(const RowsArgs& rows, const wf_logit_rules& rules,
                              const void* logits, int dtype, int32_t V, int64_t row_stride,
                              Partial* part, int32_t* accept_len, int32_t* bonus,
                              int32_t* best_node, int32_t* row_argmax, hipStream_t stream);

hipError_t launch_history_prompt(uint16_t* history, int32_t slots, int32_t V, int64_t stride,
                                 int32_t B, const int32_t* slot, const int32_t* tokens,
                                 const int32_t* offsets, int32_t count, hipStream_t stream);
hipError_t launch_history_update(uint16_t* history, int32_t slots, int32_t V, int64_t stride,
                                 const RowsArgs& rows, const int32_t* slot,
                                 const int32_t* accept_len, const int32_t* best_node,
                                 const int32_t* bonus, hipStream_t stream);

// How the attention cuts a sequence's positions: `splits` pieces of `span`
// positions (a multiple of a key tile).
struct AttendPlan {
  int32_t splits, span;
};

AttendPlan attend_plan(const wf_page_cache& cache, const RowsArgs& rows, int32_t q_heads,
                       int32_t max_context);
// Workgroups of the launch.
int64_t attend_blocks(const wf_page_cache& cache, const RowsArgs& rows, int32_t q_heads,
                      int32_t max_context);
size_t attend_workspace(const wf_page_cache& cache, const RowsArgs& rows, int32_t q_heads,
                        int32_t max_context, int64_t total_rows);
hipError_t launch_attend(const void* q, int64_t q_stride, int32_t q_heads,
                         const wf_page_cache& cache, int32_t layer, const RowsArgs& rows,
                         const int32_t* seq, int32_t max_context, float scale, void* out,
                         void* workspace, int64_t total_rows, hipStream_t stream);

hipError_t launch_cache_append(const wf_page_cache& cache, int32_t layer, const RowsArgs& rows,
                               const int32_t* seq, const void* k_rows, int64_t k_stride,
                               const void* v_rows, int64_t v_stride, hipStream_t stream);
hipError_t launch_cache_compact(const wf_page_cache& cache, const RowsArgs& rows,
                                const int32_t* seq, const int32_t* accept_len,
                                const int32_t* best_node, int32_t* next_context,
                                hipStream_t stream);
// The committed lengths alone, and a fork's pages alone (the copies come after them).
hipError_t launch_cache_commit(const wf_page_cache& cache, const RowsArgs& rows,
                               const int32_t* seq, const int32_t* accept_len,
                               const int32_t* best_node, int32_t* next_context,
                               hipStream_t stream);
hipError_t launch_pages_fork(const wf_page_cache& cache, int32_t n, const int32_t* src,
                             const int32_t* dst, int32_t* status, int32_t* ws, hipStream_t stream);
// int32 words of scratch of the page bookkeeping for n entries.
size_t pages_workspace_words(const wf_page_cache& cache, int32_t n);
hipError_t launch_cache_fork(const wf_page_cache& cache, int32_t n, const int32_t* src,
                             const int32_t* dst, int32_t* status, int32_t* ws,
                             hipStream_t stream);
hipError_t launch_cache_reserve(const wf_page_cache& cache, int32_t n, const int32_t* seq,
                                const int32_t* count, int32_t* status, int32_t* ws,
                                hipStream_t stream);
hipError_t launch_cache_free(const wf_page_cache& cache, int32_t n, const int32_t* seq,
                             hipStream_t stream);

}  // namespace wf
