// The rules of decoding applied to the logits of a round's rows: written out
// (whiflash_process_logits), or folded into the greedy argmax
// (whiflash_verify_constrained), whose chunk partials the acceptance then merges.
#include <math.h>

#include "accept.h"
#include "elem.h"
#include "rounds.h"
#include "rules_math.h"

namespace wf {
namespace {

constexpr int kChunk = 8192;  // entries of a row per workgroup

struct RulesArgs {
  RowsArgs rows;
  wf_logit_rules rules;
  const unsigned char* logits;
  int64_t row_bytes;
  int V, chunks;
  Partial* part;       // argmax: [B * rmax][chunks]
  unsigned char* out;  // written form
  int64_t out_bytes;
};

// One workgroup per (sequence, row, chunk); OUT < 0: argmax.
template <int DT, int OUT>
__global__ __launch_bounds__(kThreads) void rules_kernel(RulesArgs a) {
  __shared__ int path_s[kMaxSeqRows];
  __shared__ int np_s;
  __shared__ float sv[kWaves];
  __shared__ int si[kWaves];
  const int tid = threadIdx.x;
  const int c = blockIdx.x % a.chunks;
  const int bi = blockIdx.x / a.chunks;
  const int b = bi / a.rows.rmax, i = bi - b * a.rows.rmax;
  const SeqRows q = seq_rows(a.rows, b);
  if (i >= q.n) return;
  const int64_t r = static_cast<int64_t>(q.row0) + i;
  // The row's path tokens.
  if (tid == 0) {
    int n = 0;
    for (int u = i; u > 0; u = node_parent(a.rows, b, q.tree, u)) {
      const int v = node_token(a.rows, b, q.tree, u, a.V);
      if (v >= 0 && v / kChunk == c) path_s[n++] = v;
    }
    np_s = n;
  }
  __syncthreads();
  const int np = np_s;
  const wf_logit_rules& R = a.rules;
  Penalties pen{1.f, 0.f, 0.f};
  const bool penal = R.penalties != nullptr;
  if (penal) pen = Penalties{R.penalties[3 * b], R.penalties[3 * b + 1], R.penalties[3 * b + 2]};
  const int slot = R.history ? slot_of(R.slot, b, R.slots) : -1;
  const uint16_t* hist = slot >= 0 ? R.history + slot * R.history_stride : nullptr;
  int blo = 0, bhi = 0;
  if (R.bias_offsets) {
    blo = min(max(R.bias_offsets[b], 0), R.bias_count);
    bhi = min(max(R.bias_offsets[b + 1], blo), R.bias_count);
  }
  const unsigned char* rowp = a.logits + r * a.row_bytes;
  const int32_t* allow = R.allow ? R.allow + r * R.allow_stride : nullptr;
  float best = -INFINITY;
  int idx = -1;
  const int end = min((c + 1) * kChunk, a.V);
  for (int v = c * kChunk + tid; v < end; v += kThreads) {
    float x = Elem<DT>::scalar(rowp, v);
    if (penal) {
      int extra = 0;
      for (int k = 0; k < np; ++k) extra += path_s[k] == v;
      x = apply_penalties(x, hist ? hist[v] : 0u, extra, pen);
    }
    if (blo < bhi) {
      const int k = lower_bound(R.bias_ids, blo, bhi, v);
      if (k < bhi && R.bias_ids[k] == v) x += R.bias_values[k];
    }
    if (allow && !((static_cast<unsigned>(allow[v >> 5]) >> (v & 31)) & 1u)) x = -INFINITY;
    if constexpr (OUT < 0) {
      if (x > best) {
        best = x;
        idx = v;
      }
    } else if constexpr (OUT == WF_F32) {
      reinterpret_cast<float*>(a.out + r * a.out_bytes)[v] = x;
    } else {
      reinterpret_cast<uint16_t*>(a.out + r * a.out_bytes)[v] = static_cast<uint16_t>(bf16_bits(x));
    }
  }
  if constexpr (OUT < 0) {
    wave_argmax_to_lane63(best, idx);
    if ((tid & 63) == 63) {
      sv[tid >> 6] = best;
      si[tid >> 6] = idx;
    }
    __syncthreads();
    if (tid == 0) {
      best = sv[0];
      idx = si[0];
      for (int w = 1; w < kWaves; ++w) better_partial(best, idx, sv[w], si[w]);
      a.part[static_cast<int64_t>(bi) * a.chunks + c] = Partial{best, idx};
    }
  }
}

// The acceptance over partials [B * rmax][chunks], one workgroup per sequence.
struct ConstrainedAccept {
  RowsArgs rows;
  const Partial* part;
  int splits, V;
  int32_t* accept_len;
  int32_t* bonus;
  int32_t* best_node;
  int32_t* row_argmax;
};

__global__ __launch_bounds__(kThreads) void constrained_accept_kernel(ConstrainedAccept a) {
  __shared__ AcceptLds L;
  const int b = blockIdx.x;
  const RowsArgs& rows = a.rows;
  const SeqRows q = seq_rows(rows, b);
  int32_t* best = a.best_node ? a.best_node + b : nullptr;
  if (q.n == 0) {
    if (threadIdx.x == 0) {
      a.accept_len[b] = 0;
      a.bonus[b] = -1;
      if (best) *best = -1;
    }
    return;
  }
  const Partial* part = a.part + static_cast<int64_t>(b) * rows.rmax * a.splits;
  int32_t* argmax = a.row_argmax ? a.row_argmax + q.row0 : nullptr;
  MergeIn mi;
  merge_load(mi, part, a.splits, 0, q.n);
  if (q.tree) {
    const int64_t o = static_cast<int64_t>(b) * rows.N;
    TreeIn ti;
    tree_load_ids(ti, rows.N, rows.parent + o, rows.draft_ids + o);
    tree_load_tokens(ti, rows.d2t, rows.Vd, a.V);
    merge_finish(mi, part, a.splits, 0, q.n, L.t_s, argmax);
    __syncthreads();
    tree_accept(ti, L.t_s, rows.N, L.anc, L.dep, L.ok, L.red, a.accept_len + b, a.bonus + b, best);
  } else {
    const int32_t* draft = rows.chain_draft + static_cast<int64_t>(b) * rows.K;
    const int draft0 = rows.K > 0 ? chain_load(draft, rows.K) : -1;
    merge_finish(mi, part, a.splits, 0, q.n, L.t_s, argmax);
    __syncthreads();
    chain_accept(draft0, L.t_s, rows.K, draft, a.accept_len + b, a.bonus + b, best);
  }
}

RulesArgs rules_args(const RowsArgs& rows, const wf_logit_rules& rules, const void* logits,
                     int dtype, int32_t V, int64_t row_stride) {
  RulesArgs a{};
  a.rows = rows;
  a.rules = rules;
  a.logits = static_cast<const unsigned char*>(logits);
  a.row_bytes = row_stride * (dtype == WF_BF16 ? 2 : 4);
  a.V = V;
  a.chunks = rules_plan(dtype, rows.B, rows.rmax, V).chunks;
  return a;
}

template <int DT>
void launch_written(const RulesArgs& a, int out_dtype, dim3 grid, hipStream_t stream) {
  if (out_dtype == WF_BF16) {
    hipLaunchKernelGGL((rules_kernel<DT, WF_BF16>), grid, dim3(kThreads), 0, stream, a);
  } else {
    hipLaunchKernelGGL((rules_kernel<DT, WF_F32>), grid, dim3(kThreads), 0, stream, a);
  }
}

}  // namespace

RulesPlan rules_plan(int, int32_t, int32_t rmax, int32_t V) {
  return RulesPlan{(V + kChunk - 1) / kChunk, rmax, 1};
}

hipError_t launch_process(const RowsArgs& rows, const wf_logit_rules& rules, const void* logits,
                          int dtype, int32_t V, int64_t row_stride, void* out, int out_dtype,
                          int64_t out_stride, hipStream_t stream) {
  RulesArgs a = rules_args(rows, rules, logits, dtype, V, row_stride);
  a.out = static_cast<unsigned char*>(out);
  a.out_bytes = out_stride * (out_dtype == WF_BF16 ? 2 : 4);
  const dim3 grid(static_cast<unsigned>(rows.B) * rows.rmax * a.chunks);
  if (dtype == WF_BF16) {
    launch_written<WF_BF16>(a, out_dtype, grid, stream);
  } else {
    launch_written<WF_F32>(a, out_dtype, grid, stream);
  }
  return hipGetLastError();
}

hipError_t launch_constrained(const RowsArgs& rows, const wf_logit_rules& rules,
                              const void* logits, int dtype, int32_t V, int64_t row_stride,
                              Partial* part, int32_t* accept_len, int32_t* bonus,
                              int32_t* best_node, int32_t* row_argmax, hipStream_t stream) {
  RulesArgs a = rules_args(rows, rules, logits, dtype, V, row_stride);
  a.part = part;
  const dim3 grid(static_cast<unsigned>(rows.B) * rows.rmax * a.chunks);
  if (dtype == WF_BF16) {
    hipLaunchKernelGGL((rules_kernel<WF_BF16, -1>), grid, dim3(kThreads), 0, stream, a);
  } else {
    hipLaunchKernelGGL((rules_kernel<WF_F32, -1>), grid, dim3(kThreads), 0, stream, a);
  }
  if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
  const ConstrainedAccept f{rows,       part,  a.chunks,  V,
                            accept_len, bonus, best_node, row_argmax};
  hipLaunchKernelGGL(constrained_accept_kernel, dim3(rows.B), dim3(kThreads), 0, stream, f);
  return hipGetLastError();
}

}  // namespace wf
