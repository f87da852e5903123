// The token history of the rules: one uint16 word per (slot, token), bit 15 for a
// prompt token, the low 15 bits how often the token was put out.
//
// A few words per sequence: both calls are bound by their launch and one chain of
// dependent reads (slot, drafts, word).  A word is half of an aligned 32-bit word,
// changed by compare-and-swap, so equal tokens, and sequences that share a slot,
// add up; sums and ORs do not depend on the order.
#include "rounds.h"

namespace wf {
namespace {

constexpr unsigned kCountMask = 0x7fffu;

// One change of the history word of token v: f(word) -> word, atomically.
template <typename F>
__device__ inline void change_word(uint16_t* row, int v, F f) {
  unsigned* w = reinterpret_cast<unsigned*>(row) + (v >> 1);
  const int shift = (v & 1) * 16;
  unsigned old = __hip_atomic_load(w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (;;) {
    const unsigned h = (old >> shift) & 0xffffu;
    const unsigned n = f(h);
    if (n == h) return;
    const unsigned want = (old & ~(0xffffu << shift)) | (n << shift);
    const unsigned was = atomicCAS(w, old, want);
    if (was == old) return;
    old = was;
  }
}

__device__ inline void count_once(uint16_t* row, int v) {
  change_word(row, v, [](unsigned h) { return (h & kCountMask) == kCountMask ? h : h + 1u; });
}

__global__ __launch_bounds__(kThreads) void history_prompt_kernel(
    uint16_t* __restrict__ history, int slots, int V, int64_t stride,
    const int32_t* __restrict__ slot, const int32_t* __restrict__ tokens,
    const int32_t* __restrict__ offsets, int count) {
  const int b = blockIdx.x;
  const int s = slot_of(slot, b, slots);
  if (s < 0) return;
  uint16_t* row = history + s * stride;
  const int lo = min(max(offsets[b], 0), count), hi = min(max(offsets[b + 1], lo), count);
  for (int64_t i = lo + static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x; i < hi;
       i += gridDim.y * kThreads) {
    const int v = tokens[i];
    if (v >= 0 && v < V) change_word(row, v, [](unsigned h) { return h | 0x8000u; });
  }
}

// One wave per sequence.
__global__ __launch_bounds__(64) void history_update_kernel(
    uint16_t* __restrict__ history, int slots, int V, int64_t stride, RowsArgs rows,
    const int32_t* __restrict__ slot, const int32_t* __restrict__ accept_len,
    const int32_t* __restrict__ best_node, const int32_t* __restrict__ bonus) {
  __shared__ int par_s[kMaxSeqRows];
  __shared__ int path_s[kMaxSeqRows];
  __shared__ int len_s;
  const int b = blockIdx.x, lane = threadIdx.x;
  const int s = slot_of(slot, b, slots);
  const SeqRows q = seq_rows(rows, b);
  if (s < 0 || q.n == 0) return;
  uint16_t* row = history + s * stride;
  if (!q.tree) {
    const int al = accept_len[b];
    if (al < 1 || al > q.n) return;
    for (int u = 1 + lane; u < al; u += 64) {
      const int v = node_token(rows, b, false, u, V);
      if (v >= 0) count_once(row, v);
    }
  } else {
    const int best = best_node[b];
    if (best < 0 || best >= q.n) return;
    for (int u = 1 + lane; u <= best; u += 64) par_s[u] = node_parent(rows, b, true, u);
    __syncthreads();
    if (lane == 0) {
      int u = best, n = 0;
      for (; u > 0; u = par_s[u]) path_s[n++] = u;
      len_s = u == 0 ? n : -1;
    }
    __syncthreads();
    if (len_s < 0) return;
    for (int i = lane; i < len_s; i += 64) {
      const int v = node_token(rows, b, true, path_s[i], V);
      if (v >= 0) count_once(row, v);
    }
  }
  if (lane == 0) {
    const int v = bonus[b];
    if (v >= 0 && v < V) count_once(row, v);
  }
}

}  // namespace

hipError_t launch_history_prompt(uint16_t* history, int32_t slots, int32_t V, int64_t stride,
                                 int32_t B, const int32_t* slot, const int32_t* tokens,
                                 const int32_t* offsets, int32_t count, hipStream_t stream) {
  // Up to 16 workgroups a sequence, each with eight tokens a thread.
  const int per = kThreads * 8;
  const int y = count / B / per + 1 < 16 ? count / B / per + 1 : 16;
  hipLaunchKernelGGL(history_prompt_kernel, dim3(B, y), dim3(kThreads), 0, stream, history, slots,
                     V, stride, slot, tokens, offsets, count);
  return hipGetLastError();
}

hipError_t launch_history_update(uint16_t* history, int32_t slots, int32_t V, int64_t stride,
                                 const RowsArgs& rows, const int32_t* slot,
                                 const int32_t* accept_len, const int32_t* best_node,
                                 const int32_t* bonus, hipStream_t stream) {
  hipLaunchKernelGGL(history_update_kernel, dim3(rows.B), dim3(64), 0, stream, history, slots, V,
                     stride, rows, slot, accept_len, best_node, bonus);
  return hipGetLastError();
}

}  // namespace wf
