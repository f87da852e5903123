// Attention of a round's rows over the paged cache of 8 bits (whiflash_attend8).
//
// One wave per (row, query head) walks the positions 64 at a time, a lane each, with the running
// maximum and sum of the softmax; then every lane adds up its dimensions of the values.
#include <math.h>

#include "decode.h"
#include "e4m3.h"

namespace wf {
namespace {

constexpr float kLog2E = 1.44269504088896340736f;
constexpr float kLowest = -3.0e38f;

struct Attend8Args {
  RowsArgs rows;
  const unsigned char* q;
  int64_t q_bytes;
  int q_heads, group;
  const unsigned char *k, *v, *k_scale, *v_scale;  // the layer
  int64_t page_bytes, scale_page;
  int pages, heads, page_log, block_log, seqs, max_pages;
  const int32_t* table;
  const int32_t* context;
  const int32_t* seq;
  int max_context;
  float scale_log2;
  unsigned char* out;
};

template <int DT, int D>
__global__ __launch_bounds__(kThreads) void attend8_kernel(Attend8Args a) {
  using E = Elem<DT>;
  __shared__ float q_s[kWaves][D];
  __shared__ int16_t par_s[kMaxSeqRows];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int groups = (a.q_heads + kWaves - 1) / kWaves;
  const int bi = blockIdx.x / groups, h = (blockIdx.x - bi * groups) * kWaves + wave;
  const int b = bi / a.rows.rmax, i = bi - b * a.rows.rmax;
  const SeqRows sq = seq_rows(a.rows, b);
  if (i >= sq.n) return;
  if (sq.tree)
    for (int u = 1 + threadIdx.x; u < sq.n; u += kThreads)
      par_s[u] = static_cast<int16_t>(node_parent(a.rows, b, true, u));
  const int s = slot_of(a.seq, b, a.seqs);
  int c = s < 0 ? -1 : a.context[s];
  if (c > a.max_context || static_cast<int64_t>(c) + sq.n > static_cast<int64_t>(a.max_pages) << a.page_log) c = -1;
  if (c < 0) c = -1;
  const int64_t r = static_cast<int64_t>(sq.row0) + i;
  if (h < a.q_heads)
    for (int d = lane; d < D; d += 64)
      q_s[wave][d] = E::scalar(a.q + r * a.q_bytes, h * D + d) * a.scale_log2;
  __syncthreads();
  if (h >= a.q_heads) return;
  constexpr int kPer = D / 64;
  float m = kLowest, l = 0.f, o[kPer] = {};
  const int kvh = h / a.group, end = c < 0 ? 0 : c + i + 1;
  for (int j0 = 0; j0 < end; j0 += 64) {
    const int j = j0 + lane;
    bool see = j < end;
    if (see && sq.tree && j >= c) {
      int u = i;
      while (u > j - c) u = par_s[u];
      see = u == j - c;
    }
    int p = see ? a.table[static_cast<int64_t>(s) * a.max_pages + (j >> a.page_log)] : -1;
    if (p >= a.pages) p = -1;
    see = p >= 0;
    const int off = j & ((1 << a.page_log) - 1);
    const int64_t at = max(p, 0) * a.page_bytes + ((static_cast<int64_t>(kvh) << a.page_log) + off) * D;
    const int64_t sat = max(p, 0) * a.scale_page + (static_cast<int64_t>(kvh) << (a.page_log - a.block_log)) + (off >> a.block_log);
    float w = -INFINITY;
    if (see) {
      w = 0.f;
      for (int d = 0; d < D; d += 16) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(a.k + at + d);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y[4];
          unpack_e4m3(x[e], y);
#pragma unroll
          for (int f = 0; f < 4; ++f) w = fmaf(q_s[wave][d + 4 * e + f], y[f], w);
        }
      }
      w *= scale_of(a.k_scale[sat]);
    }
    float top = w;
    for (int x = 32; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
    const float now = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - now);
    const float e = see ? __builtin_amdgcn_exp2f(w - now) : 0.f;
    float sum = e;
    for (int x = 32; x > 0; x >>= 1) sum += __shfl_xor(sum, x);
    l = l * f + sum;
    m = now;
#pragma unroll
    for (int k = 0; k < kPer; ++k) o[k] *= f;
    for (int x = 0; x < 64; ++x) {
      if (!__shfl(static_cast<int>(see), x)) continue;
      const float wx = __shfl(e, x), sx = scale_of(a.v_scale[__shfl(sat, x)]);
      const unsigned char* v = a.v + __shfl(at, x);
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        float y[4];
        unpack_e4m3(v[lane + 64 * k], y);
        o[k] = fmaf(wx, y[0] * sx, o[k]);
      }
    }
  }
  const float f = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t to = (r * a.q_heads + h) * D + lane + 64 * k;
    if constexpr (DT == WF_F32) {
      reinterpret_cast<float*>(a.out)[to] = o[k] * f;
    } else {
      reinterpret_cast<uint16_t*>(a.out)[to] = static_cast<uint16_t>(two_bf16(o[k] * f, 0.f));
    }
  }
}

}  // namespace

int64_t attend8_blocks(const wf_page_cache8&, const RowsArgs& rows, int, int32_t q_heads, int32_t) {
  return static_cast<int64_t>(rows.B) * rows.rmax * ((q_heads + kWaves - 1) / kWaves);
}

size_t attend8_workspace(const wf_page_cache8&, const RowsArgs&, int, int32_t, int32_t, int64_t) { return 0; }

hipError_t launch_attend8(const void* q, int64_t q_stride, int32_t q_heads, int dtype,
                          const wf_page_cache8& cache, int32_t layer, const RowsArgs& rows,
                          const int32_t* seq, int32_t max_context, float scale, void* out,
                          void*, int64_t, hipStream_t stream) {
  Attend8Args a{};
  a.rows = rows;
  a.q = static_cast<const unsigned char*>(q);
  a.q_bytes = q_stride * (dtype == WF_BF16 ? 2 : 4);
  a.q_heads = q_heads;
  a.group = q_heads / cache.pages.heads;
  a.k = static_cast<const unsigned char*>(cache.pages.k) + layer * cache.pages.layer_stride;
  a.v = static_cast<const unsigned char*>(cache.pages.v) + layer * cache.pages.layer_stride;
  a.k_scale = cache.k_scale + layer * cache.scale_layer_stride;
  a.v_scale = cache.v_scale + layer * cache.scale_layer_stride;
  a.page_bytes = cache.pages.page_stride;
  a.scale_page = cache.scale_page_stride;
  a.pages = cache.pages.pages;
  a.heads = cache.pages.heads;
  a.page_log = __builtin_ctz(static_cast<unsigned>(cache.pages.page_size));
  a.block_log = __builtin_ctz(static_cast<unsigned>(cache.block));
  a.seqs = cache.pages.seqs;
  a.max_pages = cache.pages.max_pages;
  a.table = cache.pages.table;
  a.context = cache.pages.context;
  a.seq = seq;
  a.max_context = max_context;
  a.scale_log2 = scale * kLog2E;
  a.out = static_cast<unsigned char*>(out);
  const dim3 grid(static_cast<unsigned>(attend8_blocks(cache, rows, dtype, q_heads, max_context))), block(kThreads);
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
  const bool wide = cache.pages.head_dim == 128;
  if (dtype == WF_BF16) {
    wide ? go(attend8_kernel<WF_BF16, 128>) : go(attend8_kernel<WF_BF16, 64>);
  } else {
    wide ? go(attend8_kernel<WF_F32, 128>) : go(attend8_kernel<WF_F32, 64>);
  }
  return hipGetLastError();
}

}  // namespace wf
