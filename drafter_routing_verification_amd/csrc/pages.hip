// The paged key-value cache: rows put in, accepted tree paths moved to the front,
// and the bookkeeping of pages (fork, reserve, free).
//
// Free pages are those with refs 0, handed out lowest first: there is no free list
// to keep in order, so freeing is one atomic decrement a page and the result never
// depends on the order of workgroups.
#include <limits.h>

#include "elem.h"
#include "rounds.h"

namespace wf {
namespace {

constexpr int kAllocThreads = 1024;
constexpr int kScan = 16;  // pages a thread looks at in one pass
constexpr int kAllocWaves = kAllocThreads / 64;

// The cache with every size a kernel needs in bytes of 16-byte vectors.
struct CacheArgs {
  u32x4* k;
  u32x4* v;
  int64_t layer_vecs, page_vecs;
  int pages, heads, page_log, row_vecs, seqs, max_pages;
  int32_t* table;
  int32_t* held;
  int32_t* context;
  int32_t* refs;
};

CacheArgs cache_args(const wf_page_cache& c) {
  const int per = c.dtype == WF_BF16 ? 8 : 4;
  CacheArgs a{};
  a.k = static_cast<u32x4*>(c.k);
  a.v = static_cast<u32x4*>(c.v);
  a.layer_vecs = c.layer_stride / per;
  a.page_vecs = c.page_stride / per;
  a.pages = c.pages;
  a.heads = c.heads;
  a.page_log = __builtin_ctz(static_cast<unsigned>(c.page_size));
  a.row_vecs = c.head_dim / per;
  a.seqs = c.seqs;
  a.max_pages = c.max_pages;
  a.table = c.table;
  a.held = c.held;
  a.context = c.context;
  a.refs = c.refs;
  return a;
}

// Vector offset of head 0 of position `pos` of sequence s inside a layer, or -1
// where it has no page.
__device__ inline int64_t position_vec(const CacheArgs& a, int s, int64_t pos) {
  const int64_t j = pos >> a.page_log;
  if (pos < 0 || j >= a.max_pages) return -1;
  const int p = a.table[static_cast<int64_t>(s) * a.max_pages + j];
  if (p < 0 || p >= a.pages) return -1;
  return p * a.page_vecs + (pos & ((1 << a.page_log) - 1)) * a.row_vecs;
}

// ---------------------------------------------------------------- append

// One workgroup per (sequence, row): every thread moves 16-byte vectors of k, then of v.
// Bound by the reads that find the place (context, table): 2 us for one row, 5 for 488.
__global__ __launch_bounds__(kThreads) void cache_append_kernel(
    CacheArgs a, int layer, RowsArgs rows, const int32_t* __restrict__ seq,
    const u32x4* __restrict__ k_rows, int64_t k_stride, const u32x4* __restrict__ v_rows,
    int64_t v_stride) {
  const int b = blockIdx.x / rows.rmax, i = blockIdx.x - b * rows.rmax;
  const SeqRows q = seq_rows(rows, b);
  const int s = slot_of(seq, b, a.seqs);
  if (i >= q.n || s < 0) return;
  const int c = a.context[s];
  const int64_t at = c < 0 ? -1 : position_vec(a, s, static_cast<int64_t>(c) + i);
  if (at < 0) return;
  const int64_t r = static_cast<int64_t>(q.row0) + i;
  const int cols = a.heads * a.row_vecs;
  for (int t = threadIdx.x; t < 2 * cols; t += kThreads) {
    const bool key = t < cols;
    const int col = key ? t : t - cols;
    const int h = col / a.row_vecs, e = col - h * a.row_vecs;
    const u32x4 x = key ? k_rows[r * k_stride + col] : v_rows[r * v_stride + col];
    (key ? a.k : a.v)[layer * a.layer_vecs + at + (static_cast<int64_t>(h) << a.page_log) * a.row_vecs + e] = x;
  }
}

// ---------------------------------------------------------------- compact

constexpr int kMoveBatch = 8;  // rows in flight per thread

// One workgroup per (sequence, layer).  Row u_j of the path moves to row j <= u_j.  Each
// thread owns 16-byte columns (of k, then of v) and takes the path's rows in order: the
// destination of step j is a source of steps before j only, so no step overwrites what a
// later one reads, and no two threads touch one column.
//
// Bound by chains of reads: those that find the path (the parents are fetched before it is
// known which are needed), its pages, then the rows.
// With `after` apart from the context the first layer's workgroups commit too.
__global__ __launch_bounds__(kThreads) void cache_compact_kernel(
    CacheArgs a, RowsArgs rows, const int32_t* __restrict__ seq,
    const int32_t* __restrict__ accept_len, const int32_t* __restrict__ best_node,
    int32_t* __restrict__ after) {
  __shared__ int par_s[kMaxSeqRows];
  __shared__ int64_t src_s[kMaxSeqRows], dst_s[kMaxSeqRows];
  __shared__ int len_s;
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
    // The path from its end: step al - 1 is the best node.
    int u = best, j = al - 1;
    for (; u > 0 && j > 0; u = par_s[u]) src_s[j--] = u;
    len_s = u == 0 && j == 0 ? al : 0;
    if (commits) after[s] = c + len_s;
  }
  __syncthreads();
  const int len = len_s;
  for (int j = 1 + tid; j < len; j += kThreads) {
    const int64_t u = src_s[j];
    const int64_t from = u == j ? -1 : position_vec(a, s, c + u);
    src_s[j] = from;
    dst_s[j] = from < 0 ? -1 : position_vec(a, s, static_cast<int64_t>(c) + j);
  }
  __syncthreads();
  const int cols = a.heads * a.row_vecs;
  for (int t = tid; t < 2 * cols; t += kThreads) {
    const int col = t < cols ? t : t - cols;
    const int h = col / a.row_vecs, e = col - h * a.row_vecs;
    u32x4* p = (t < cols ? a.k : a.v) + blockIdx.y * a.layer_vecs +
               (static_cast<int64_t>(h) << a.page_log) * a.row_vecs + e;
    for (int j0 = 1; j0 < len; j0 += kMoveBatch) {
      u32x4 d[kMoveBatch];
#pragma unroll
      for (int k = 0; k < kMoveBatch; ++k)
        if (j0 + k < len && dst_s[j0 + k] >= 0) d[k] = p[src_s[j0 + k]];
#pragma unroll
      for (int k = 0; k < kMoveBatch; ++k)
        if (j0 + k < len && dst_s[j0 + k] >= 0) p[dst_s[j0 + k]] = d[k];
    }
  }
}

// The committed lengths in a launch of their own, after the moves: for a round of chains,
// and where next_context is the context that the moves read.
__global__ __launch_bounds__(kThreads) void cache_commit_kernel(
    CacheArgs a, RowsArgs rows, const int32_t* __restrict__ seq,
    const int32_t* __restrict__ accept_len, const int32_t* __restrict__ best_node,
    int32_t* next_context) {
  const int b = blockIdx.x * kThreads + threadIdx.x;
  if (b >= rows.B) return;
  const int s = slot_of(seq, b, a.seqs);
  if (s < 0) return;
  const SeqRows q = seq_rows(rows, b);
  const int c = a.context[s], al = accept_len[b];
  bool ok = c >= 0 && q.n > 0 && al >= 0 && al <= q.n;
  if (ok && q.tree) {
    int u = best_node[b], j = al - 1;
    ok = al > 0 && u >= 0 && u < q.n;
    while (ok && u > 0 && j > 0) {
      u = node_parent(rows, b, true, u);
      --j;
    }
    ok = ok && u == 0 && j == 0;
  }
  next_context[s] = ok ? c + al : c;
}

// ---------------------------------------------------------------- pages

__device__ inline int64_t wave_inclusive(int64_t x, int lane) {
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t o = __shfl_up(x, off);
    if (lane >= off) x += o;
  }
  return x;
}

// Exclusive prefix sum over the workgroup; *total gets the sum.  sums: LDS scratch.
__device__ inline int64_t block_exclusive(int64_t x, int64_t* sums, int64_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t inc = wave_inclusive(x, lane);
  __syncthreads();
  if (lane == 63) sums[wave] = inc;
  __syncthreads();
  int64_t before = 0, all = 0;
  for (int w = 0; w < kAllocWaves; ++w) {
    if (w < wave) before += sums[w];
    all += sums[w];
  }
  *total = all;
  return before + inc - x;
}

// Scratch (int32 words): rank [n + 1], mark [seqs], source [seqs], fresh [pages].
struct PagesWs {
  int32_t* rank;
  int32_t* mark;
  int32_t* source;
  int32_t* fresh;
};

PagesWs pages_ws(const wf_page_cache& c, int32_t n, int32_t* ws) {
  PagesWs w;
  w.rank = ws;
  w.mark = w.rank + static_cast<size_t>(n) + 1;
  w.source = w.mark + c.seqs;
  w.fresh = w.source + c.seqs;
  return w;
}

// Hands out pages in one workgroup.  FORK: entry i makes seq[i] a fork of src[i] and
// needs a page if the context ends inside one; else entry i gives seq[i] room for
// context + count[i] positions.  Ranks are prefix sums of the needs; the free page of
// rank g (lowest first) goes to the entry whose range holds g, if all of that entry's
// range was found.  One workgroup, so that ranks need no second launch: 7 to 10 us, its
// barriers and dependent reads, for pools of some thousand pages; 16 past 20,000 taken pages and
// 101 past 200,000, which it looks through one pass after the other.
template <bool FORK>
__global__ __launch_bounds__(kAllocThreads) void pages_alloc_kernel(
    CacheArgs a, int n, const int32_t* __restrict__ src, const int32_t* __restrict__ seq,
    const int32_t* __restrict__ count, int32_t* __restrict__ status, PagesWs w) {
  __shared__ int64_t sums[kAllocWaves];
  const int tid = threadIdx.x;
  const int ps = 1 << a.page_log;
  for (int s = tid; s < a.seqs; s += kAllocThreads) {
    w.mark[s] = INT_MAX;
    if (FORK) w.source[s] = 0;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kAllocThreads) {
    const int s = seq[i];
    if (s >= 0 && s < a.seqs) atomicMin(w.mark + s, i);
    if (FORK) {
      const int o = src[i];
      if (o >= 0 && o < a.seqs) w.source[o] = 1;
    }
  }
  __syncthreads();
  // Needs and ranks (cut at pages + 1: nothing that high can be granted).
  int64_t want = 0;
  for (int i0 = 0; i0 < n; i0 += kAllocThreads) {
    const int i = i0 + tid;
    int need = 0;
    bool ok = false;
    if (i < n) {
      const int s = seq[i];
      ok = s >= 0 && s < a.seqs && w.mark[s] == i;
      if (ok && FORK) {
        const int o = src[i];
        ok = o >= 0 && o < a.seqs && o != s && !w.source[s] && a.held[s] == 0;
        if (ok) {
          const int c = a.context[o], h = a.held[o];
          ok = c >= 0 && h <= a.max_pages && c <= static_cast<int64_t>(h) << a.page_log;
          need = ok && (c & (ps - 1)) ? 1 : 0;
        }
      } else if (ok) {
        const int c = a.context[s], m = count[i], h = a.held[s];
        const int64_t pages = (static_cast<int64_t>(c) + m + ps - 1) >> a.page_log;
        ok = c >= 0 && m >= 0 && h >= 0 && h <= a.max_pages && pages <= a.max_pages;
        need = ok && pages > h ? static_cast<int>(pages - h) : 0;
      }
      status[i] = ok ? 1 + (need > 0) : 0;  // 2: if its pages are found
    }
    int64_t total;
    const int64_t before = block_exclusive(need, sums, &total);
    if (i < n) w.rank[i] = static_cast<int>(min(want + before, static_cast<int64_t>(a.pages) + 1));
    want += total;
  }
  if (tid == 0) w.rank[n] = static_cast<int>(min(want, static_cast<int64_t>(a.pages) + 1));
  // The lowest free pages, as many as are wanted.
  const int64_t most = min(want, static_cast<int64_t>(a.pages));
  int64_t found = 0;
  for (int64_t p0 = 0; p0 < a.pages && found < most; p0 += kAllocThreads * kScan) {
    // A thread's kScan pages in a row: a bit for each free one.
    const int64_t p = p0 + tid * kScan;
    int refs[kScan];
#pragma unroll
    for (int k = 0; k < kScan; ++k) refs[k] = p + k < a.pages ? a.refs[p + k] : 1;
    unsigned bits = 0;
#pragma unroll
    for (int k = 0; k < kScan; ++k) bits |= refs[k] == 0 ? 1u << k : 0u;
    int64_t total;
    int64_t g = found + block_exclusive(__popc(bits), sums, &total);
    for (; bits && g < most; bits &= bits - 1, ++g)
      w.fresh[g] = static_cast<int>(p) + __ffs(bits) - 1;
    found += total;
  }
  found = min(found, most);
  __syncthreads();
  for (int g = tid; g < found; g += kAllocThreads) {
    // The entry whose range [rank[i], rank[i + 1]) holds g.
    int lo = 0, hi = n;
    while (lo + 1 < hi) {
      const int mid = lo + (hi - lo) / 2;
      if (w.rank[mid] <= g) {
        lo = mid;
      } else {
        hi = mid;
      }
    }
    if (w.rank[lo + 1] > found) continue;
    const int s = seq[lo], p = w.fresh[g];
    const int at = FORK ? a.context[src[lo]] >> a.page_log : a.held[s] + (g - w.rank[lo]);
    a.table[static_cast<int64_t>(s) * a.max_pages + at] = p;
    a.refs[p] = 1;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kAllocThreads) {
    if (!status[i]) continue;
    // (The ranks of entries behind the pool's end are all the same.)
    const bool needs = status[i] == 2;
    const int s = seq[i];
    if (needs && w.rank[i + 1] > found) {
      status[i] = 0;
      continue;
    }
    status[i] = 1;
    if (FORK) {
      const int c = a.context[src[i]];
      a.held[s] = (c >> a.page_log) + (needs ? 1 : 0);
      a.context[s] = c;
    } else {
      a.held[s] += w.rank[i + 1] - w.rank[i];
    }
  }
}

// One workgroup per (entry, layer and k or v): the partly filled last page's rows; the
// first also shares the full pages.  A copy: 128 forks of 32 sequences, 36 layers, 278 MB read
// and written, 44 us (6.3 TB/s: four forks read one source).
__global__ __launch_bounds__(kThreads) void cache_fork_kernel(CacheArgs a,
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
  u32x4* base = ((blockIdx.y & 1) ? a.v : a.k) + (blockIdx.y >> 1) * a.layer_vecs;
  const u32x4* ps = base + p * a.page_vecs;
  u32x4* pd = base + d * a.page_vecs;
  const int each = part * a.row_vecs, head = a.row_vecs << a.page_log;
  for (int e = tid; e < each * a.heads; e += kThreads) {
    const int h = e / each;
    const int at = h * head + (e - h * each);
    pd[at] = ps[at];
  }
}

__global__ __launch_bounds__(kThreads) void cache_free_kernel(CacheArgs a,
                                                              const int32_t* __restrict__ seq) {
  __shared__ int held_s;
  const int s = seq[blockIdx.x];
  if (s < 0 || s >= a.seqs) return;
  // One of the workgroups that name a sequence gets its pages, the others none.
  if (threadIdx.x == 0) {
    held_s = min(atomicExch(a.held + s, 0), a.max_pages);
    if (held_s > 0) a.context[s] = 0;
  }
  __syncthreads();
  int32_t* row = a.table + static_cast<int64_t>(s) * a.max_pages;
  for (int j = threadIdx.x; j < held_s; j += kThreads) {
    const int p = row[j];
    row[j] = -1;
    if (p >= 0 && p < a.pages) atomicSub(a.refs + p, 1);
  }
}

}  // namespace

hipError_t launch_cache_append(const wf_page_cache& cache, int32_t layer, const RowsArgs& rows,
                               const int32_t* seq, const void* k_rows, int64_t k_stride,
                               const void* v_rows, int64_t v_stride, hipStream_t stream) {
  const int per = cache.dtype == WF_BF16 ? 8 : 4;
  hipLaunchKernelGGL(cache_append_kernel, dim3(static_cast<unsigned>(rows.B) * rows.rmax),
                     dim3(kThreads), 0, stream, cache_args(cache), layer, rows, seq,
                     static_cast<const u32x4*>(k_rows), k_stride / per,
                     static_cast<const u32x4*>(v_rows), v_stride / per);
  return hipGetLastError();
}

hipError_t launch_cache_compact(const wf_page_cache& cache, const RowsArgs& rows,
                                const int32_t* seq, const int32_t* accept_len,
                                const int32_t* best_node, int32_t* next_context,
                                hipStream_t stream) {
  const CacheArgs a = cache_args(cache);
  int32_t* after = next_context && next_context != cache.context ? next_context : nullptr;
  if (rows.kind != WF_ROWS_CHAIN) {
    hipLaunchKernelGGL(cache_compact_kernel, dim3(rows.B, cache.layers), dim3(kThreads), 0, stream,
                       a, rows, seq, accept_len, best_node, after);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || after) return e;
  }
  hipLaunchKernelGGL(cache_commit_kernel, dim3((rows.B + kThreads - 1) / kThreads), dim3(kThreads),
                     0, stream, a, rows, seq, accept_len, best_node,
                     after ? after : cache.context);
  return hipGetLastError();
}

size_t pages_workspace_words(const wf_page_cache& cache, int32_t n) {
  return static_cast<size_t>(n) + 1 + 2 * static_cast<size_t>(cache.seqs) + cache.pages;
}

hipError_t launch_cache_fork(const wf_page_cache& cache, int32_t n, const int32_t* src,
                             const int32_t* dst, int32_t* status, int32_t* ws,
                             hipStream_t stream) {
  const CacheArgs a = cache_args(cache);
  hipLaunchKernelGGL((pages_alloc_kernel<true>), dim3(1), dim3(kAllocThreads), 0, stream, a, n, src,
                     dst, nullptr, status, pages_ws(cache, n, ws));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(cache_fork_kernel, dim3(n, 2 * cache.layers), dim3(kThreads), 0, stream, a,
                     src, dst, status);
  return hipGetLastError();
}

hipError_t launch_cache_reserve(const wf_page_cache& cache, int32_t n, const int32_t* seq,
                                const int32_t* count, int32_t* status, int32_t* ws,
                                hipStream_t stream) {
  hipLaunchKernelGGL((pages_alloc_kernel<false>), dim3(1), dim3(kAllocThreads), 0, stream,
                     cache_args(cache), n, nullptr, seq, count, status, pages_ws(cache, n, ws));
  return hipGetLastError();
}

hipError_t launch_cache_free(const wf_page_cache& cache, int32_t n, const int32_t* seq,
                             hipStream_t stream) {
  hipLaunchKernelGGL(cache_free_kernel, dim3(n), dim3(kThreads), 0, stream, cache_args(cache), seq);
  return hipGetLastError();
}

}  // namespace wf
