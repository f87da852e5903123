// The token history of the rules: one uint16 word per (slot, token), bit 15 for a
// prompt token, the low 15 bits how often the token was put out.
//
// A few words per sequence: both calls are bound by their launch and one chain of
// dependent reads (slot, drafts, word).  A word is half of an aligned 32-bit word,
// changed by compare-and-swap, so equal tokens, and sequences that share a slot,
// add up; sums and ORs do not depend on the order.  An update takes 1.8 us (one chain) to
// 4.6 us (128 sequences, trees among them), a prompt of 8 sequences x 4,000 tokens 13 us.
//
// The last token of an odd vocabulary has its 32 bits together with the element past the
// row, which the last slot's storage need not hold: it is read and written as the 16 bits
// that it has.  Every workgroup of history_prompt writes the same value there; of
// history_update one workgroup a slot writes it, for all sequences that share the slot.
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

// Whether token v has no other token of its row in its 32-bit word.
__device__ inline bool alone(int v, int V) { return v == V - 1 && (V & 1); }

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
    if (v < 0 || v >= V) continue;
    if (alone(v, V)) {
      row[v] |= 0x8000u;
    } else {
      change_word(row, v, [](unsigned h) { return h | 0x8000u; });
    }
  }
}

// How often a verified sequence enters token v: by one lane, along its path.
__device__ inline int times_entered(const RowsArgs& rows, int b, int V, int v,
                                    const int32_t* __restrict__ accept_len,
                                    const int32_t* __restrict__ best_node,
                                    const int32_t* __restrict__ bonus) {
  const SeqRows q = seq_rows(rows, b);
  int u = q.n == 0 ? -1 : q.tree ? best_node[b] : accept_len[b] - 1;
  if (u < 0 || u >= q.n) return 0;
  int times = bonus[b] == v;
  for (; u > 0; u = node_parent(rows, b, q.tree, u)) times += node_token(rows, b, q.tree, u, V) == v;
  return u == 0 ? times : 0;
}

// One wave per sequence.  The last token of an odd vocabulary, where the wave's own sequence
// enters it, is counted by the first such sequence of its slot: that wave looks through the
// slots for the others.  Waves that do not come upon that token do nothing of this.
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
  int last = 0;  // how often this lane came upon the last token of an odd vocabulary
  auto enter = [&](int v) {
    if (v < 0 || v >= V) return;
    if (alone(v, V)) {
      ++last;
    } else {
      count_once(row, v);
    }
  };
  if (!q.tree) {
    const int al = accept_len[b];
    if (al < 1 || al > q.n) return;
    for (int u = 1 + lane; u < al; u += 64) enter(node_token(rows, b, false, u, V));
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
    for (int i = lane; i < len_s; i += 64) enter(node_token(rows, b, true, path_s[i], V));
  }
  if (lane == 0) enter(bonus[b]);
  if (!__any(last > 0)) return;
  bool earlier = false;
  for (int o = lane; slot && o < rows.B; o += 64) {
    if (o == b || slot[o] != s) continue;
    const int times = times_entered(rows, o, V, V - 1, accept_len, best_node, bonus);
    if (o > b) last += times;
    earlier = earlier || (o < b && times > 0);
  }
  if (__any(earlier)) return;
  for (int off = 32; off > 0; off >>= 1) last += __shfl_xor(last, off);
  if (lane == 0) {
    const unsigned h = row[V - 1], count = h & kCountMask;
    const unsigned room = kCountMask - count;
    row[V - 1] = static_cast<uint16_t>(h + min(static_cast<unsigned>(last), room));
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
