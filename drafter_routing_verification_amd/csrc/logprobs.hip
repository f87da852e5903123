// Log probabilities of given tokens, entropy and most likely tokens of logits rows
// (whiflash_token_logprobs), in one pass over the logits.
//
// Every thread keeps, for the vectors it takes, S = sum of e^(x - r), U = sum of (x - r) e^(x - r)
// and the true maximum; r is a maximum it has seen, raised only when a vector's exceeds it by
// more than kSlack, so that hardly any vector rescales.  Sums over another reference follow from
//   S' = f S,  U' = f (U + (r - r') S),  f = e^(r - r'),
// and with the row's maximum M: log p(x) = (x - M) - ln S, H = ln S - U / S.
//
// The most likely tokens: a wave keeps the 64 best it has seen as a sorted list, one a lane.  What
// exceeds the list's place `top` is put aside in LDS, 64 at a time are sorted and merged.  The
// first vectors set the bar: the top-th largest of the lanes' maxima is held by as many elements.
// A wave's vectors come in the order of their indices, so that a later element equal to the bar
// never displaces an earlier one.
#include <limits.h>
#include <math.h>

#include "decode.h"
#include "elem.h"

namespace wf {
namespace {

constexpr float kLog2E = 1.44269504088896340736f;
constexpr float kFloor = -3.402823466e38f;  // a reference below every finite logit
constexpr float kSlack = 8.f;
constexpr float kFar = -1000.f;  // e^kFar is 0: what stands for -inf where it meets that 0
constexpr int kAhead = 4;        // vectors in flight per thread
constexpr int kList = 64;

struct LogprobsArgs {
  const unsigned char* logits;
  int64_t row_bytes;
  int total_rows, V, n, given, top, chunks, vecs, nvec;
  const int32_t* rows;
  const int32_t* tokens;
  float* logprob;
  float* entropy;
  int32_t* top_tokens;
  float* top_logprobs;
  float4* stats;   // [n][chunks] maximum, S, U
  float2* lists;   // [n][chunks][top] value, index bits
};

// Sums relative to a reference m.
struct Sums {
  float m, s, u;
  __device__ inline void move(float to) {
    const float f = __builtin_amdgcn_exp2f((m - to) * kLog2E);
    u = f > 0.f ? f * (u + (m - to) * s) : 0.f;
    s = f > 0.f ? f * s : (s != s ? s : 0.f);
    m = to;
  }
};

__device__ inline bool better(float av, int ai, float bv, int bi) {
  return (av > bv) | ((av == bv) & (ai < bi));
}

// Orders a wave's LDS accesses: what a lane wrote before, every lane reads after.
__device__ inline void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// One value and index a lane.
struct Entry {
  float v;
  int i;
};

__device__ inline void exchange(Entry& e, int j, bool keep_better) {
  const Entry o{__shfl_xor(e.v, j), __shfl_xor(e.i, j)};
  if (better(o.v, o.i, e.v, e.i) == keep_better) e = o;
}

// Sorts a wave's entries, the best in lane 0.
__device__ inline void sort_wave(Entry& e) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int k = 2; k <= 64; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) exchange(e, j, ((lane & j) == 0) == ((lane & k) == 0));
}

// The 64 best of two sorted lists, sorted.
__device__ inline void merge_wave(Entry& e, const Entry& other) {
  const int lane = threadIdx.x & 63;
  const Entry o{__shfl(other.v, 63 - lane), __shfl(other.i, 63 - lane)};
  if (better(o.v, o.i, e.v, e.i)) e = o;
#pragma unroll
  for (int j = 32; j > 0; j >>= 1) exchange(e, j, (lane & j) == 0);
}

// The most likely entries that a wave has seen.
struct Best {
  Entry list;
  float bar;
  int waiting;      // uniform
  float2* aside;    // the wave's 128 places

  __device__ inline void start(float2* lds) {
    list = Entry{-INFINITY, INT_MAX};
    bar = -INFINITY;
    waiting = 0;
    aside = lds;
  }
  __device__ inline void take_in() {
    const int lane = threadIdx.x & 63;
    wave_sync();
    const float2 x = aside[lane], rest = aside[lane + kList];
    wave_sync();
    aside[lane] = rest;
    Entry e{x.x, __float_as_int(x.y)};
    if (lane >= waiting) e = Entry{-INFINITY, INT_MAX};
    waiting = max(waiting - kList, 0);
    sort_wave(e);
    merge_wave(list, e);
  }
  // Puts this lane's entry aside if `on`.
  __device__ inline void offer(bool on, float v, int i) {
    const unsigned long long mask = __ballot(on);
    if (mask == 0) return;
    const int before = __builtin_amdgcn_mbcnt_hi(static_cast<unsigned>(mask >> 32),
                                                 __builtin_amdgcn_mbcnt_lo(static_cast<unsigned>(mask), 0));
    if (on) aside[waiting + before] = make_float2(v, __int_as_float(i));
    waiting += __popcll(mask);
    if (waiting >= kList) take_in();
  }
  __device__ inline void raise(int top) {
    bar = fmaxf(bar, __shfl(list.v, top - 1));
  }
  // The bar that the lanes' largest values set.
  __device__ inline void first_bar(float lane_max, int top) {
    Entry e{lane_max, static_cast<int>(threadIdx.x & 63)};
    sort_wave(e);
    bar = __shfl(e.v, top - 1);
  }
};

__device__ inline int64_t row_of(const LogprobsArgs& a, int i) {
  const int r = a.rows ? a.rows[i] : i;
  return r >= 0 && r < a.total_rows ? r : -1;
}

// Writes row i's results from its sums and (a lane each) its best entries.
template <int DT>
__device__ inline void emit(const LogprobsArgs& a, int i, int64_t row, const Sums& x, const Entry& e) {
  const int lane = threadIdx.x & 63;
  const bool any = row >= 0 && x.s > 0.f && x.s < INFINITY;  // (false for NaN)
  const float ln = any ? logf(x.s) : NAN;
  for (int j = lane; j < a.given; j += 64) {
    const int64_t at = static_cast<int64_t>(i) * a.given + j;
    const int t = a.tokens[at];
    float p = NAN;
    if (any && t >= 0 && t < a.V) p = (Elem<DT>::scalar(a.logits + row * a.row_bytes, t) - x.m) - ln;
    a.logprob[at] = p;
  }
  if (a.entropy && lane == 0) a.entropy[i] = any ? ln - x.u / x.s : NAN;
  if (lane < a.top) {
    const int64_t at = static_cast<int64_t>(i) * a.top + lane;
    const bool is = any && e.v > -INFINITY;
    a.top_tokens[at] = is ? e.i : -1;
    a.top_logprobs[at] = is ? (e.v - x.m) - ln : any ? -INFINITY : NAN;
  }
}

// Sums over the lanes of a wave, relative to the largest maximum, in every lane.
__device__ inline Sums wave_sums(Sums x, float largest) {
  for (int off = 32; off > 0; off >>= 1) largest = fmaxf(largest, __shfl_xor(largest, off));
  x.move(largest);
  for (int off = 32; off > 0; off >>= 1) {
    x.s += __shfl_xor(x.s, off);
    x.u += __shfl_xor(x.u, off);
  }
  return x;
}

// One workgroup per (row, chunk).
template <int DT, bool TOP>
__global__ __launch_bounds__(kThreads) void logprobs_kernel(LogprobsArgs a) {
  using E = Elem<DT>;
  constexpr int kPer = E::kPerVec;
  __shared__ float2 aside_s[kWaves][2 * kList];
  __shared__ float4 stats_s[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int i = blockIdx.x / a.chunks, c = blockIdx.x - i * a.chunks;
  const int64_t row = row_of(a, i);
  Sums x{kFloor, 0.f, 0.f};
  float largest = kFloor;
  Best best;
  best.start(aside_s[wave]);
  if (row >= 0) {
    const unsigned char* rowp = a.logits + row * a.row_bytes;
    const u32x4* vp = reinterpret_cast<const u32x4*>(rowp);
    const int v0 = c * a.vecs, v1 = min(v0 + a.vecs, a.nvec);
    auto absorb = [&](const float* y, float top) {
      largest = fmaxf(largest, top);
      if (top > x.m + kSlack) x.move(top);
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const float d = y[k] - x.m;
        const float e = __builtin_amdgcn_exp2f(d * kLog2E);
        x.s += e;
        x.u += fmaxf(d, kFar) * e;
      }
    };
    auto choose = [&](const float* y, float top, int at, bool first) {
      if (__ballot(first ? top >= best.bar : top > best.bar) == 0) return;
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        best.offer(first ? y[k] >= best.bar : y[k] > best.bar, y[k], at + k);
      if (!first) best.raise(a.top);
    };
    bool first = true;
    for (int v = v0 + tid - lane; v < v1; v += kAhead * kThreads) {  // (uniform over the wave)
      u32x4 d[kAhead];
      float top[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (v + lane + u * kThreads < v1) d[u] = load16(vp + v + lane + u * kThreads);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) top[u] = v + lane + u * kThreads < v1 ? E::vmax(d[u]) : -INFINITY;
      if (TOP && first) {
        float most = top[0];
#pragma unroll
        for (int u = 1; u < kAhead; ++u) most = fmaxf(most, top[u]);
        best.first_bar(most, a.top);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const bool have = v + lane + u * kThreads < v1;
        float y[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) y[k] = have ? E::at(d[u], k) : -INFINITY;
        if (have) absorb(y, top[u]);
        if (TOP) choose(y, top[u], (v + lane + u * kThreads) * kPer, first);
      }
      if (TOP && first) best.raise(a.top);
      first = false;
    }
    // What does not fill a vector, by the last wave of the last chunk (its indices are the largest).
    const int rest = a.V - a.nvec * kPer;
    if (rest > 0 && c == a.chunks - 1 && wave == kWaves - 1) {
      float y[kPer];
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        y[k] = lane == 0 && k < rest ? E::scalar(rowp, a.nvec * kPer + k) : -INFINITY;
        top = fmaxf(top, y[k]);
      }
      absorb(y, top);
      if (TOP) choose(y, top, a.nvec * kPer, first);
    }
    if (TOP && best.waiting > 0) best.take_in();
  }
  x = wave_sums(x, largest);
  if (lane == 0) stats_s[wave] = make_float4(x.m, x.s, x.u, 0.f);
  if (TOP) {
    wave_sync();
    aside_s[wave][lane] = make_float2(best.list.v, __int_as_float(best.list.i));
  }
  __syncthreads();
  if (wave > 0) return;
  const float4 mine = stats_s[lane & (kWaves - 1)];
  x = wave_sums(lane < kWaves ? Sums{mine.x, mine.y, mine.z} : Sums{kFloor, 0.f, 0.f},
                lane < kWaves ? mine.x : kFloor);
  Entry e = best.list;
  if (TOP)
    for (int w = 1; w < kWaves; ++w) {
      const float2 o = aside_s[w][lane];
      merge_wave(e, Entry{o.x, __float_as_int(o.y)});
    }
  if (a.chunks == 1) {
    emit<DT>(a, i, row, x, e);
    return;
  }
  const int64_t at = static_cast<int64_t>(i) * a.chunks + c;
  if (lane == 0) a.stats[at] = make_float4(x.m, x.s, x.u, 0.f);
  if (TOP && lane < a.top) a.lists[at * a.top + lane] = make_float2(e.v, __int_as_float(e.i));
}

// Joins a row's chunks: one wave each.
template <int DT>
__global__ __launch_bounds__(64) void logprobs_join_kernel(LogprobsArgs a) {
  __shared__ float2 aside_s[2 * kList];
  const int i = blockIdx.x, lane = threadIdx.x;
  const int64_t row = row_of(a, i), base = static_cast<int64_t>(i) * a.chunks;
  Sums x{kFloor, 0.f, 0.f};
  for (int c = lane; c < a.chunks; c += 64) {
    const float4 y = a.stats[base + c];
    const float m = fmaxf(x.m, y.x);
    Sums o{y.x, y.y, y.z};
    x.move(m);
    o.move(m);
    x.s += o.s;
    x.u += o.u;
  }
  x = wave_sums(x, x.m);
  Best best;
  best.start(aside_s);
  if (a.top > 0) {
    const float2* all = a.lists + base * a.top;
    const int many = a.chunks * a.top;
    float most = -INFINITY;
    for (int t = lane; t < many; t += 64) most = fmaxf(most, all[t].x);
    best.first_bar(most, a.top);
    for (int t0 = 0; t0 < many; t0 += 64) {
      const float2 y = t0 + lane < many ? all[t0 + lane] : make_float2(-INFINITY, 0.f);
      best.offer(t0 + lane < many && y.x >= best.bar, y.x, __float_as_int(y.y));
    }
    if (best.waiting > 0) best.take_in();
  }
  emit<DT>(a, i, row, x, best.list);
}

template <int DT>
void launch_typed(const LogprobsArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.n) * a.chunks), block(kThreads);
  if (a.top > 0) {
    hipLaunchKernelGGL((logprobs_kernel<DT, true>), grid, block, 0, stream, a);
  } else {
    hipLaunchKernelGGL((logprobs_kernel<DT, false>), grid, block, 0, stream, a);
  }
  if (a.chunks > 1)
    hipLaunchKernelGGL((logprobs_join_kernel<DT>), dim3(a.n), dim3(64), 0, stream, a);
}

}  // namespace

// Workgroups enough for every CU, of no fewer than a batch of vectors a thread.
LogprobsPlan logprobs_plan(int dtype, int32_t n, int32_t V) {
  const int nvec = V / (dtype == WF_BF16 ? 8 : 4);
  const int most = (nvec + kAhead * kThreads - 1) / (kAhead * kThreads);
  int chunks = (2048 + n - 1) / n;
  chunks = chunks > most ? most : chunks;
  chunks = chunks < 1 ? 1 : chunks;
  int vecs = (nvec + chunks - 1) / chunks;
  vecs = (vecs + kThreads - 1) / kThreads * kThreads;
  vecs = vecs < kThreads ? kThreads : vecs;
  chunks = (nvec + vecs - 1) / vecs;
  return LogprobsPlan{chunks < 1 ? 1 : chunks, vecs};
}

size_t logprobs_workspace(int32_t n, int32_t V, int32_t top) {
  size_t most = 0;
  for (int dtype : {WF_F32, WF_BF16}) {
    const LogprobsPlan p = logprobs_plan(dtype, n, V);
    const size_t parts = p.chunks > 1 ? static_cast<size_t>(n) * p.chunks : 0;
    const size_t bytes = parts * (sizeof(float4) + top * sizeof(float2));
    most = bytes > most ? bytes : most;
  }
  return most;
}

hipError_t launch_logprobs(const void* logits, int dtype, int32_t total_rows, int32_t V,
                           int64_t row_stride, int32_t n, const int32_t* rows, int32_t given,
                           const int32_t* tokens, int32_t top, float* logprob, float* entropy,
                           int32_t* top_tokens, float* top_logprobs, void* ws, hipStream_t stream) {
  const LogprobsPlan plan = logprobs_plan(dtype, n, V);
  LogprobsArgs a{};
  a.logits = static_cast<const unsigned char*>(logits);
  a.row_bytes = row_stride * (dtype == WF_BF16 ? 2 : 4);
  a.total_rows = total_rows;
  a.V = V;
  a.n = n;
  a.given = given;
  a.top = top;
  a.chunks = plan.chunks;
  a.vecs = plan.vecs;
  a.nvec = V / (dtype == WF_BF16 ? 8 : 4);
  a.rows = rows;
  a.tokens = tokens;
  a.logprob = logprob;
  a.entropy = entropy;
  a.top_tokens = top_tokens;
  a.top_logprobs = top_logprobs;
  a.stats = static_cast<float4*>(ws);
  if (plan.chunks > 1)
    a.lists = reinterpret_cast<float2*>(a.stats + static_cast<size_t>(n) * plan.chunks);
  if (dtype == WF_BF16) {
    launch_typed<WF_BF16>(a, stream);
  } else {
    launch_typed<WF_F32>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace wf
