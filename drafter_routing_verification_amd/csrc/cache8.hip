// The paged cache of 8 bits: rows quantised as they are written, positions read back, accepted
// tree paths moved to the front, sequences forked.
//
// A block is `block` positions of one head under one scale 2^e (e4m3.h).  A power of two, because
// the relative step of e4m3 does not depend on the scale: nothing is lost against any other scale
// of the block, products with it are exact, and what a block holds can be brought under another
// scale by shifting exponents.
//
// Everywhere a team of D / 8 lanes owns a block of one head of the keys or of the values, eight
// dimensions a lane: a row is eight bytes a lane, its maximum a reduction over the team, and no
// two teams touch one byte.
#include <limits.h>

#include "decode.h"
#include "e4m3.h"

namespace wf {
namespace {

struct Cache8Args {
  unsigned char* data[2];   // keys, values
  unsigned char* scale[2];
  int64_t layer_bytes, page_bytes, scale_layer, scale_page;
  int pages, heads, page_log, block_log, seqs, max_pages;
  int32_t* table;
  int32_t* context;
  int32_t* refs;
};

Cache8Args cache8_args(const wf_page_cache8& c) {
  Cache8Args a{};
  a.data[0] = static_cast<unsigned char*>(c.pages.k);
  a.data[1] = static_cast<unsigned char*>(c.pages.v);
  a.scale[0] = c.k_scale;
  a.scale[1] = c.v_scale;
  a.layer_bytes = c.pages.layer_stride;
  a.page_bytes = c.pages.page_stride;
  a.scale_layer = c.scale_layer_stride;
  a.scale_page = c.scale_page_stride;
  a.pages = c.pages.pages;
  a.heads = c.pages.heads;
  a.page_log = __builtin_ctz(static_cast<unsigned>(c.pages.page_size));
  a.block_log = __builtin_ctz(static_cast<unsigned>(c.block));
  a.seqs = c.pages.seqs;
  a.max_pages = c.pages.max_pages;
  a.table = c.pages.table;
  a.context = c.pages.context;
  a.refs = c.pages.refs;
  return a;
}

// The page of position pos >= 0 of sequence s, or -1.
__device__ inline int page_of(const Cache8Args& a, int s, int64_t pos) {
  const int64_t j = pos >> a.page_log;
  if (j >= a.max_pages) return -1;
  const int p = a.table[static_cast<int64_t>(s) * a.max_pages + j];
  return p >= 0 && p < a.pages ? p : -1;
}

// Where head h's position `pos` lies in page p, and the scale of its block.
template <int D>
__device__ inline int64_t byte_of(const Cache8Args& a, int p, int h, int64_t pos) {
  const int o = static_cast<int>(pos) & ((1 << a.page_log) - 1);
  return p * a.page_bytes + ((static_cast<int64_t>(h) << a.page_log) + o) * D;
}
__device__ inline int64_t scale_at(const Cache8Args& a, int p, int h, int64_t pos) {
  const int o = static_cast<int>(pos) & ((1 << a.page_log) - 1);
  return p * a.scale_page + (static_cast<int64_t>(h) << (a.page_log - a.block_log)) + (o >> a.block_log);
}

// The largest over a team's lanes.
template <int TEAM>
__device__ inline float team_max(float x) {
#pragma unroll
  for (int off = 1; off < TEAM; off <<= 1) x = fmaxf(x, __shfl_xor(x, off));
  return x;
}

// The largest finite magnitude of eight values.
__device__ inline float largest(const float* x) {
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = fmaxf(m, finite_bits(x[k]) ? fabsf(x[k]) : 0.f);
  return m;
}

__device__ inline uint2 quantise(const float* x, float inv) {
  float y[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) y[k] = scaled_down(x[k], inv);
  return make_uint2(pack_e4m3(y[0], y[1], y[2], y[3]), pack_e4m3(y[4], y[5], y[6], y[7]));
}

// 2^-e of a scale byte.
__device__ inline float inverse_scale(int byte) { return __uint_as_float(static_cast<unsigned>(254 - byte) << 23); }

// What eight stored values stand for, from the byte of their scale.
__device__ inline void stand_for(uint2 w, int byte, float* x) {
  unpack_e4m3(w.x, x);
  unpack_e4m3(w.y, x + 4);
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = ldexpf(x[k], byte - 127);
}

// ---------------------------------------------------------------- append

template <int DT, int D>
__global__ __launch_bounds__(kThreads) void cache8_append_kernel(
    Cache8Args a, int layer, RowsArgs rows, const int32_t* __restrict__ seq,
    const unsigned char* __restrict__ k_rows, int64_t k_bytes,
    const unsigned char* __restrict__ v_rows, int64_t v_bytes, int wgs) {
  constexpr int kTeam = D / 8, kTeams = kThreads / kTeam;
  const int b = blockIdx.x / wgs;
  const SeqRows q = seq_rows(rows, b);
  const int s = slot_of(seq, b, a.seqs);
  if (q.n == 0 || s < 0) return;
  const int64_t c = a.context[s];
  if (c < 0) return;
  // Unit: (block of the span, keys or values, head).
  const int64_t unit = static_cast<int64_t>(blockIdx.x - b * wgs) * kTeams + threadIdx.x / kTeam;
  const int lane8 = (threadIdx.x % kTeam) * 8;
  const int64_t nth = unit / (2 * a.heads);
  const int rest = static_cast<int>(unit - nth * 2 * a.heads);
  const int which = rest >= a.heads ? 1 : 0, h = rest - which * a.heads;
  const int64_t lo = ((c >> a.block_log) + nth) << a.block_log;
  const int64_t hi = min(lo + (int64_t{1} << a.block_log), c + q.n);
  if (lo >= c + q.n) return;
  const int p = page_of(a, s, lo);
  if (p < 0) return;
  unsigned char* data = a.data[which] + layer * a.layer_bytes + byte_of<D>(a, p, h, lo) + lane8;
  unsigned char* scale = a.scale[which] + layer * a.scale_layer + scale_at(a, p, h, lo);
  const int64_t stride = which ? v_bytes : k_bytes;
  // Row i of the round is position c + i.
  const unsigned char* from = (which ? v_rows : k_rows) + (q.row0 + lo - c) * stride +
                              (static_cast<int64_t>(h) * D + lane8) * Elem<DT>::kBytes;
  const int kept = static_cast<int>(min(max(c - lo, int64_t{0}), hi - lo)), all = static_cast<int>(hi - lo);
  const int old = kept > 0 ? *scale : 0;
  float top = 0.f;
  for (int j = 0; j < kept; ++j) {
    float x[8];
    stand_for(*reinterpret_cast<const uint2*>(data + j * D), old, x);
    top = fmaxf(top, largest(x));
  }
  for (int j = kept; j < all; ++j) {
    float x[8];
    load_eight<DT>(from + j * stride, x);
    top = fmaxf(top, largest(x));
  }
  const int now = scale_for(team_max<kTeam>(top));
  const float inv = inverse_scale(now);
  if (now != old) {
    for (int j = 0; j < kept; ++j) {
      float x[8];
      stand_for(*reinterpret_cast<const uint2*>(data + j * D), old, x);
      *reinterpret_cast<uint2*>(data + j * D) = quantise(x, inv);
    }
  }
  for (int j = kept; j < all; ++j) {
    float x[8];
    load_eight<DT>(from + j * stride, x);
    *reinterpret_cast<uint2*>(data + j * D) = quantise(x, inv);
  }
  if (lane8 == 0) *scale = static_cast<unsigned char>(now);
}

// ---------------------------------------------------------------- read

constexpr int kReadRows = 16;  // positions of a workgroup

template <int DT, int D>
__global__ __launch_bounds__(kThreads) void cache8_read_kernel(
    Cache8Args a, int layer, const int32_t* __restrict__ seq, const int32_t* __restrict__ first,
    int count, int pending, unsigned char* __restrict__ k_out, unsigned char* __restrict__ v_out,
    int wgs) {
  constexpr int kTeam = D / 8, kTeams = kThreads / kTeam;
  const int b = blockIdx.x / wgs, i0 = (blockIdx.x - b * wgs) * kReadRows;
  const int s = slot_of(seq, b, a.seqs);
  const int64_t c = s < 0 ? -1 : a.context[s];
  const int64_t end = c < 0 ? 0 : c + pending;
  const int64_t from = first ? first[b] : 0;
  const int lane8 = (threadIdx.x % kTeam) * 8;
  const int units = min(count - i0, kReadRows) * a.heads;
  for (int which = 0; which < 2; ++which) {
    unsigned char* out = which ? v_out : k_out;
    if (!out) continue;
    for (int t = threadIdx.x / kTeam; t < units; t += kTeams) {
      const int i = t / a.heads, h = t - i * a.heads;
      const int64_t pos = from + i0 + i;
      const int p = pos >= 0 && pos < end ? page_of(a, s, pos) : -1;
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (p >= 0)
        stand_for(*reinterpret_cast<const uint2*>(a.data[which] + layer * a.layer_bytes + byte_of<D>(a, p, h, pos) + lane8),
                  a.scale[which][layer * a.scale_layer + scale_at(a, p, h, pos)], x);
      const int64_t row = static_cast<int64_t>(b) * count + i0 + i;
      store_eight<DT>(out + ((row * a.heads + h) * D + lane8) * Elem<DT>::kBytes, x);
    }
  }
}

// ---------------------------------------------------------------- compact

// One workgroup per (sequence, layer).  Row u_j of the path moves to row j <= u_j, block of
// destinations after block: a block's new scale is that of what it will hold, found from the
// sources, which lie in this block or behind it and so still have their own scales.
template <int D>
__global__ __launch_bounds__(kThreads) void cache8_compact_kernel(
    Cache8Args a, RowsArgs rows, const int32_t* __restrict__ seq,
    const int32_t* __restrict__ accept_len, const int32_t* __restrict__ best_node,
    int32_t* __restrict__ after) {
  constexpr int kTeam = D / 8, kTeams = kThreads / kTeam;
  __shared__ int par_s[kMaxSeqRows], row_s[kMaxSeqRows], page_s[kMaxSeqRows];
  __shared__ int len_s, stays_s;
  const int b = blockIdx.x, tid = threadIdx.x;
  for (int u = 1 + tid; u < rows.N; u += kThreads) par_s[u] = node_parent(rows, b, true, u);
  const SeqRows q = seq_rows(rows, b);
  const int s = slot_of(seq, b, a.seqs);
  if (s < 0) return;
  const int c = a.context[s], al = accept_len[b], best = best_node[b];
  const bool commits = after && blockIdx.y == 0 && tid == 0;
  if (q.n == 0 || !q.tree) {
    if (commits) after[s] = c >= 0 && q.n > 0 && al >= 0 && al <= q.n ? c + al : c;
    return;
  }
  if (c < 0 || al < 1 || al > q.n || best < 0 || best >= q.n) {
    if (commits) after[s] = c;
    return;
  }
  __syncthreads();
  if (tid == 0) {
    int u = best, j = al - 1, stays = al;
    for (; u > 0 && j > 0; u = par_s[u]) {
      row_s[j] = u;
      if (u != j) stays = j;
      --j;
    }
    row_s[0] = 0;
    len_s = u == 0 && j == 0 ? al : 0;
    stays_s = stays;
    if (commits) after[s] = c + len_s;
  }
  __syncthreads();
  const int len = len_s, moved = stays_s;  // the first row that moves
  if (moved >= len) return;
  for (int j = tid; j < len; j += kThreads) page_s[j] = page_of(a, s, static_cast<int64_t>(c) + row_s[j]);
  __syncthreads();
  const int lane8 = (tid % kTeam) * 8;
  for (int unit = tid / kTeam; unit < 2 * a.heads; unit += kTeams) {
    const int which = unit >= a.heads ? 1 : 0, h = unit - which * a.heads;
    unsigned char* data = a.data[which] + blockIdx.y * a.layer_bytes + lane8;
    unsigned char* scale = a.scale[which] + blockIdx.y * a.scale_layer;
    const int64_t end = static_cast<int64_t>(c) + len;
    for (int64_t lo = (static_cast<int64_t>(c) + moved) >> a.block_log << a.block_log; lo < end;
         lo += int64_t{1} << a.block_log) {
      const int p = page_of(a, s, lo);
      if (p < 0) continue;
      const int64_t hi = min(lo + (int64_t{1} << a.block_log), end);
      unsigned char* to = data + byte_of<D>(a, p, h, lo);
      unsigned char* to_scale = scale + scale_at(a, p, h, lo);
      const int old = *to_scale, all = static_cast<int>(hi - lo);
      // Position lo + j holds row u's values afterwards (its own, before the round's): where they
      // are now (-1: in no page), with their scale.
      auto source = [&](int j, int* byte) -> int64_t {
        const int64_t pos = lo + j;
        const int64_t from = pos < c ? pos : static_cast<int64_t>(c) + row_s[pos - c];
        const int page = pos < c ? p : page_s[pos - c];
        if (page < 0) return -1;
        *byte = (from >> a.block_log) == (lo >> a.block_log) ? old : scale[scale_at(a, page, h, from)];
        return byte_of<D>(a, page, h, from);
      };
      float top = 0.f;
      for (int j = 0; j < all; ++j) {
        int byte = 0;
        float x[8];
        const int64_t at = source(j, &byte);
        if (at < 0) continue;
        stand_for(*reinterpret_cast<const uint2*>(data + at), byte, x);
        top = fmaxf(top, largest(x));
      }
      const int now = scale_for(team_max<kTeam>(top));
      const float inv = inverse_scale(now);
      for (int j = 0; j < all; ++j) {
        int byte = 0;
        float x[8];
        const int64_t at = source(j, &byte);
        if (at < 0) continue;
        const uint2 w = *reinterpret_cast<const uint2*>(data + at);
        stand_for(w, byte, x);
        *reinterpret_cast<uint2*>(to + j * D) = byte == now ? w : quantise(x, inv);
      }
      if (lane8 == 0) *to_scale = static_cast<unsigned char>(now);
    }
  }
}

// ---------------------------------------------------------------- fork

// One workgroup per (entry, layer and k or v): the partly filled last page's rows and scales; the
// first also shares the full pages.
template <int D>
__global__ __launch_bounds__(kThreads) void cache8_fork_kernel(Cache8Args a,
                                                               const int32_t* __restrict__ src,
                                                               const int32_t* __restrict__ dst,
                                                               const int32_t* __restrict__ status) {
  const int i = blockIdx.x, tid = threadIdx.x;
  if (!status[i]) return;
  const int o = src[i], s = dst[i];
  const int c = a.context[o];
  const int full = c >> a.page_log, part = c & ((1 << a.page_log) - 1);
  const int32_t* from = a.table + static_cast<int64_t>(o) * a.max_pages;
  int32_t* to = a.table + static_cast<int64_t>(s) * a.max_pages;
  if (blockIdx.y == 0) {
    for (int j = tid; j < full; j += kThreads) {
      const int p = from[j];
      to[j] = p;
      if (p >= 0 && p < a.pages) atomicAdd(a.refs + p, 1);
    }
  }
  if (part == 0) return;
  const int p = from[full], d = to[full];
  if (p < 0 || p >= a.pages) return;
  const int which = blockIdx.y & 1, layer = blockIdx.y >> 1;
  const unsigned char* base = a.data[which] + layer * a.layer_bytes;
  const u32x4* ps = reinterpret_cast<const u32x4*>(base + p * a.page_bytes);
  u32x4* pd = reinterpret_cast<u32x4*>(a.data[which] + layer * a.layer_bytes + d * a.page_bytes);
  constexpr int kVecs = D / 16;
  const int each = part * kVecs, head = kVecs << a.page_log;
  for (int e = tid; e < each * a.heads; e += kThreads) {
    const int h = e / each;
    const int at = h * head + (e - h * each);
    pd[at] = ps[at];
  }
  unsigned char* scale = a.scale[which] + layer * a.scale_layer;
  const int blocks = 1 << (a.page_log - a.block_log), used = (part + (1 << a.block_log) - 1) >> a.block_log;
  for (int e = tid; e < used * a.heads; e += kThreads) {
    const int h = e / used;
    const int at = h * blocks + (e - h * used);
    scale[d * a.scale_page + at] = scale[p * a.scale_page + at];
  }
}

// Blocks of positions that n rows can reach into.
int64_t span_blocks(const wf_page_cache8& c, int n) {
  return (static_cast<int64_t>(n) + 2 * static_cast<int64_t>(c.block) - 2) / c.block;
}

// Workgroups a sequence of the append.
int64_t append_wgs(const wf_page_cache8& c, const RowsArgs& rows) {
  const int teams = kThreads / (c.pages.head_dim / 8);
  return (span_blocks(c, rows.rmax) * 2 * c.pages.heads + teams - 1) / teams;
}

}  // namespace

int64_t cache8_append_blocks(const wf_page_cache8& cache, const RowsArgs& rows) {
  return append_wgs(cache, rows) * rows.B;
}

hipError_t launch_cache8_append(const wf_page_cache8& cache, int32_t layer, const RowsArgs& rows,
                                const int32_t* seq, int dtype, const void* k_rows, int64_t k_stride,
                                const void* v_rows, int64_t v_stride, hipStream_t stream) {
  const int bytes = dtype == WF_BF16 ? 2 : 4, wgs = static_cast<int>(append_wgs(cache, rows));
  const dim3 grid(static_cast<unsigned>(rows.B) * wgs), block(kThreads);
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, cache8_args(cache), layer, rows, seq,
                       static_cast<const unsigned char*>(k_rows), k_stride * bytes,
                       static_cast<const unsigned char*>(v_rows), v_stride * bytes, wgs);
  };
  const bool wide = cache.pages.head_dim == 128;
  if (dtype == WF_BF16) {
    wide ? go(cache8_append_kernel<WF_BF16, 128>) : go(cache8_append_kernel<WF_BF16, 64>);
  } else {
    wide ? go(cache8_append_kernel<WF_F32, 128>) : go(cache8_append_kernel<WF_F32, 64>);
  }
  return hipGetLastError();
}

int64_t cache8_read_blocks(int32_t B, int32_t count) {
  return static_cast<int64_t>(B) * ((static_cast<int64_t>(count) + kReadRows - 1) / kReadRows);
}

hipError_t launch_cache8_read(const wf_page_cache8& cache, int32_t layer, int32_t B,
                              const int32_t* seq, const int32_t* first, int32_t count,
                              int32_t pending, int dtype, void* k_out, void* v_out,
                              hipStream_t stream) {
  const int wgs = static_cast<int>(cache8_read_blocks(1, count));
  const dim3 grid(static_cast<unsigned>(B) * wgs), block(kThreads);
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, cache8_args(cache), layer, seq, first, count,
                       pending, static_cast<unsigned char*>(k_out),
                       static_cast<unsigned char*>(v_out), wgs);
  };
  const bool wide = cache.pages.head_dim == 128;
  if (dtype == WF_BF16) {
    wide ? go(cache8_read_kernel<WF_BF16, 128>) : go(cache8_read_kernel<WF_BF16, 64>);
  } else {
    wide ? go(cache8_read_kernel<WF_F32, 128>) : go(cache8_read_kernel<WF_F32, 64>);
  }
  return hipGetLastError();
}

hipError_t launch_cache8_compact(const wf_page_cache8& cache, const RowsArgs& rows,
                                 const int32_t* seq, const int32_t* accept_len,
                                 const int32_t* best_node, int32_t* next_context,
                                 hipStream_t stream) {
  int32_t* after = next_context && next_context != cache.pages.context ? next_context : nullptr;
  if (rows.kind != WF_ROWS_CHAIN) {
    const dim3 grid(rows.B, cache.pages.layers), block(kThreads);
    const auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, block, 0, stream, cache8_args(cache), rows, seq, accept_len,
                         best_node, after);
    };
    cache.pages.head_dim == 128 ? go(cache8_compact_kernel<128>) : go(cache8_compact_kernel<64>);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || after) return e;
  }
  return launch_cache_commit(cache.pages, rows, seq, accept_len, best_node,
                             after ? after : cache.pages.context, stream);
}

hipError_t launch_cache8_fork(const wf_page_cache8& cache, int32_t n, const int32_t* src,
                              const int32_t* dst, int32_t* status, int32_t* ws,
                              hipStream_t stream) {
  const hipError_t e = launch_pages_fork(cache.pages, n, src, dst, status, ws, stream);
  if (e != hipSuccess) return e;
  const dim3 grid(n, 2 * cache.pages.layers), block(kThreads);
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, cache8_args(cache), src, dst, status);
  };
  cache.pages.head_dim == 128 ? go(cache8_fork_kernel<128>) : go(cache8_fork_kernel<64>);
  return hipGetLastError();
}

}  // namespace wf
