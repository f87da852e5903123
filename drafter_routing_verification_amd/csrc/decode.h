// Launches of a decoding step's calls (rotary.hip, cache8.hip, attend8.hip, logprobs.hip).
#pragma once

#include "rounds.h"

namespace wf {

hipError_t launch_rotate(const wf_rotary& rotary, int dtype, int32_t head_dim, const RowsArgs& rows,
                         const int32_t* seq, const int32_t* context, int32_t seqs,
                         const wf_rotary_rows& q, const wf_rotary_rows* k, hipStream_t stream);

// Workgroups of the append's launch.
int64_t cache8_append_blocks(const wf_page_cache8& cache, const RowsArgs& rows);
hipError_t launch_cache8_append(const wf_page_cache8& cache, int32_t layer, const RowsArgs& rows,
                                const int32_t* seq, int dtype, const void* k_rows, int64_t k_stride,
                                const void* v_rows, int64_t v_stride, hipStream_t stream);
int64_t cache8_read_blocks(int32_t B, int32_t count);
hipError_t launch_cache8_read(const wf_page_cache8& cache, int32_t layer, int32_t B,
                              const int32_t* seq, const int32_t* first, int32_t count,
                              int32_t pending, int dtype, void* k_out, void* v_out,
                              hipStream_t stream);
hipError_t launch_cache8_compact(const wf_page_cache8& cache, const RowsArgs& rows,
                                 const int32_t* seq, const int32_t* accept_len,
                                 const int32_t* best_node, int32_t* next_context,
                                 hipStream_t stream);
hipError_t launch_cache8_fork(const wf_page_cache8& cache, int32_t n, const int32_t* src,
                              const int32_t* dst, int32_t* status, int32_t* ws, hipStream_t stream);

int64_t attend8_blocks(const wf_page_cache8& cache, const RowsArgs& rows, int dtype, int32_t q_heads,
                       int32_t max_context);
size_t attend8_workspace(const wf_page_cache8& cache, const RowsArgs& rows, int dtype,
                         int32_t q_heads, int32_t max_context, int64_t total_rows);
hipError_t launch_attend8(const void* q, int64_t q_stride, int32_t q_heads, int dtype,
                          const wf_page_cache8& cache, int32_t layer, const RowsArgs& rows,
                          const int32_t* seq, int32_t max_context, float scale, void* out,
                          void* workspace, int64_t total_rows, hipStream_t stream);

// How the log probabilities cut their rows: `chunks` workgroups a row, `vecs` 16-byte vectors each.
struct LogprobsPlan {
  int32_t chunks, vecs;
};

LogprobsPlan logprobs_plan(int dtype, int32_t n, int32_t V);
size_t logprobs_workspace(int32_t n, int32_t V, int32_t top);
hipError_t launch_logprobs(const void* logits, int dtype, int32_t total_rows, int32_t V,
                           int64_t row_stride, int32_t n, const int32_t* rows, int32_t given,
                           const int32_t* tokens, int32_t top, float* logprob, float* entropy,
                           int32_t* top_tokens, float* top_logprobs, void* ws, hipStream_t stream);

}  // namespace wf
