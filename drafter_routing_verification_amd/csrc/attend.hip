// Attention of a round's rows over the paged cache.
#include <math.h>

#include "elem.h"
#include "rounds.h"

namespace wf {
namespace {

constexpr int kKeys = 64;      // positions a wave takes at once, one per lane
constexpr int kMaxDim = 128;
constexpr float kLog2E = 1.44269504088896340736f;

struct AttendArgs {
  RowsArgs rows;
  const unsigned char* q;
  int64_t q_bytes;
  int q_heads, group;
  const unsigned char* k;  // the layer
  const unsigned char* v;
  int64_t page_elems;
  int pages, heads, page_log, seqs, max_pages;
  const int32_t* table;
  const int32_t* context;
  const int32_t* seq;
  int max_context;
  float scale_log2;
  unsigned char* out;
};

// One workgroup per (sequence, row, query head); each wave takes every fourth tile of
// 64 positions, one per lane, and the waves' running maxima, sums and outputs join at
// the end.
template <int DT, int D>
__global__ __launch_bounds__(kThreads) void attend_kernel(AttendArgs a) {
  using E = Elem<DT>;
  constexpr int kVecs = D / E::kPerVec;
  constexpr int kPer = D / 64;
  __shared__ float q_s[D];
  __shared__ float p_s[kWaves][kKeys];
  __shared__ int64_t at_s[kWaves][kKeys];
  __shared__ unsigned char see_s[kMaxSeqRows];
  __shared__ float m_s[kWaves], l_s[kWaves], o_s[kWaves][D];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int h = blockIdx.y;
  const int b = blockIdx.x / a.rows.rmax, i = blockIdx.x - b * a.rows.rmax;
  const SeqRows q = seq_rows(a.rows, b);
  if (i >= q.n) return;
  const int64_t r = static_cast<int64_t>(q.row0) + i;
  const int s = slot_of(a.seq, b, a.seqs);
  int c = s < 0 ? -1 : a.context[s];
  if (c > a.max_context || static_cast<int64_t>(c) + q.n > static_cast<int64_t>(a.max_pages) << a.page_log)
    c = -1;
  for (int u = tid; u < q.n; u += kThreads) see_s[u] = 0;
  if (tid < D) q_s[tid] = E::scalar(a.q + r * a.q_bytes, h * D + tid) * a.scale_log2;
  __syncthreads();
  if (tid == 0)
    for (int u = i; u >= 0; u = u > 0 ? node_parent(a.rows, b, q.tree, u) : -1) see_s[u] = 1;
  __syncthreads();
  const int64_t head = static_cast<int64_t>(h / a.group) * D << a.page_log;
  const int end = c < 0 ? 0 : c + q.n;
  float m = -INFINITY, l = 0.f, o[kPer] = {};
  for (int j0 = wave * kKeys; j0 < end; j0 += kWaves * kKeys) {
    const int j = j0 + lane;
    float x = -INFINITY;
    int64_t at = -1;
    if (j < end && (j < c || see_s[j - c])) {
      const int p = a.table[static_cast<int64_t>(s) * a.max_pages + (j >> a.page_log)];
      if (p >= 0 && p < a.pages) {
        at = p * a.page_elems + head + static_cast<int64_t>(j & ((1 << a.page_log) - 1)) * D;
        const u32x4* kp = reinterpret_cast<const u32x4*>(a.k + at * E::kBytes);
        x = 0.f;
        for (int e = 0; e < kVecs; ++e) {
          const u32x4 d = kp[e];
#pragma unroll
          for (int t = 0; t < E::kPerVec; ++t) x += q_s[e * E::kPerVec + t] * E::at(d, t);
        }
      }
    }
    float top = x;
    for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    const float mn = fmaxf(m, top);
    if (mn == -INFINITY) continue;
    const float f = exp2f(m - mn);
    const float p = at >= 0 ? exp2f(x - mn) : 0.f;
    m = mn;
    float sum = p;
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
    l = l * f + sum;
    p_s[wave][lane] = p;
    at_s[wave][lane] = at;
    for (int t = 0; t < kPer; ++t) o[t] *= f;
    for (int k = 0; k < kKeys; ++k) {
      const int64_t w = at_s[wave][k];
      if (w < 0) continue;
      for (int t = 0; t < kPer; ++t)
        o[t] += p_s[wave][k] * E::scalar(a.v + w * E::kBytes, lane + 64 * t);
    }
  }
  if (lane == 0) {
    m_s[wave] = m;
    l_s[wave] = l;
  }
  for (int t = 0; t < kPer; ++t) o_s[wave][lane + 64 * t] = o[t];
  __syncthreads();
  if (tid >= D) return;
  float top = m_s[0];
  for (int w = 1; w < kWaves; ++w) top = fmaxf(top, m_s[w]);
  float x = 0.f, sum = 0.f;
  for (int w = 0; w < kWaves; ++w) {
    const float f = m_s[w] == -INFINITY ? 0.f : exp2f(m_s[w] - top);
    x += f * o_s[w][tid];
    sum += f * l_s[w];
  }
  x = sum > 0.f ? x / sum : 0.f;
  const int64_t to = (r * a.q_heads + h) * D + tid;
  if constexpr (DT == WF_F32) {
    reinterpret_cast<float*>(a.out)[to] = x;
  } else {
    const unsigned u = __float_as_uint(x);
    reinterpret_cast<uint16_t*>(a.out)[to] =
        static_cast<uint16_t>((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
  }
}

}  // namespace

AttendPlan attend_plan(const wf_page_cache&, const RowsArgs&, int32_t, int32_t) {
  return AttendPlan{1, 0};
}

size_t attend_workspace(const wf_page_cache&, const RowsArgs&, int32_t, int32_t, int64_t) {
  return 0;
}

hipError_t launch_attend(const void* q, int64_t q_stride, int32_t q_heads,
                         const wf_page_cache& cache, int32_t layer, const RowsArgs& rows,
                         const int32_t* seq, int32_t max_context, float scale, void* out, void*,
                         int64_t, hipStream_t stream) {
  const int bytes = cache.dtype == WF_BF16 ? 2 : 4;
  AttendArgs a{};
  a.rows = rows;
  a.q = static_cast<const unsigned char*>(q);
  a.q_bytes = q_stride * bytes;
  a.q_heads = q_heads;
  a.group = q_heads / cache.heads;
  a.k = static_cast<const unsigned char*>(cache.k) + layer * cache.layer_stride * bytes;
  a.v = static_cast<const unsigned char*>(cache.v) + layer * cache.layer_stride * bytes;
  a.page_elems = cache.page_stride;
  a.pages = cache.pages;
  a.heads = cache.heads;
  a.page_log = __builtin_ctz(static_cast<unsigned>(cache.page_size));
  a.seqs = cache.seqs;
  a.max_pages = cache.max_pages;
  a.table = cache.table;
  a.context = cache.context;
  a.seq = seq;
  a.max_context = max_context;
  a.scale_log2 = scale * kLog2E;
  a.out = static_cast<unsigned char*>(out);
  const dim3 grid(static_cast<unsigned>(rows.B) * rows.rmax, q_heads);
  if (cache.dtype == WF_BF16) {
    if (cache.head_dim == 64) {
      hipLaunchKernelGGL((attend_kernel<WF_BF16, 64>), grid, dim3(kThreads), 0, stream, a);
    } else {
      hipLaunchKernelGGL((attend_kernel<WF_BF16, 128>), grid, dim3(kThreads), 0, stream, a);
    }
  } else if (cache.head_dim == 64) {
    hipLaunchKernelGGL((attend_kernel<WF_F32, 64>), grid, dim3(kThreads), 0, stream, a);
  } else {
    hipLaunchKernelGGL((attend_kernel<WF_F32, 128>), grid, dim3(kThreads), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace wf
