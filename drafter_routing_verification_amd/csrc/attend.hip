// Attention of a round's rows over the paged cache (whiflash_attend).
//
// Per sequence and key-value head, the M = rows x (q_heads / heads) queries that share
// its keys form tiles of 16, and a wave walks its share of the positions in tiles of
// 16 or 32 with a one-pass softmax (attend_body.h).  K and V are loaded in rows: K takes its operand layout through LDS, V is transposed by
// byte permutes (bfloat16) or used as it lies (float32).
//
// Two forms, by the number of query tiles that share a key-value head (attend_shape):
// up to two (one in float32), every wave has positions of its own and all queries; with
// more, every wave has queries of its own and the four share the positions.
//
// Measured (MI355X, 32 query heads on 8, head_dim 128, pages of 16; whole passes with their
// append and join, inputs changing from pass to pass, and in brackets the kernel alone under
// the profiler):
//   64 sequences of 4,096-8,192 positions, one row each: 256 us [247-252], 6.3 TB/s of keys and
//     values (a pure streaming read of the same memory: 7.3); bound by HBM and, for a quarter of
//     it, by sequences of unequal length.  float32 542 us, 6.0 TB/s; head_dim 64 140 us, 5.8.
//   2 chains of 17 rows over 131,000 positions: 188 us [189-212], 5.0 TB/s and 341 TFLOP/s (of
//     1,205 that a large product reaches); 8 trees of 61 rows over 2,048-4,096: 77 us [69], 335
//     TFLOP/s.  Neither the vector units (35%) nor the matrix units (25%) are full: two waves a
//     SIMD do not cover the chain from scores through maxima and exponentials to the second
//     product.  A third is kept out by the registers of two query tiles (spilled: slower) and by
//     67,584 bytes of LDS, of which a CU holds two workgroups' worth.  3 to 5 query tiles a wave,
//     with its own positions, spill too (1,047 us for the long chains).
//   float32 there: 1,200 us (floor 415: its matrix rate) and 336 us (168).
//   Far from their floors: fewer than eight pieces leave XCDs idle (unit_of): 2 chains of 1,001
//     rows over 4,000 positions 763 us, 172 TFLOP/s, where 8 of 1,024 rows reach 532; and the plan
//     knows the bound alone: one sequence of 131,000 positions among 63 of up to 1,000 1,142 us
//     for 92 us of bytes.
#include <math.h>

#include "attend_body.h"

namespace wf {
namespace {

constexpr int kMinSpan = 128;
// The plan of pieces: workgroups that run at a time (two a CU; with head_dim 64 three or four
// would fit, which the plan does not use), and the time of a workgroup's start and end, in
// positions.  64 sequences of up to 8,192 positions: one piece
// 256 us, two rounds 270, four 269, sixteen 272.
constexpr int kSlots = 512;
constexpr int kStart = 256;
constexpr int kMaxSplits = 512;
constexpr int kMaxRounds = 8;

struct Unit {
  int split, b, kvh, mg;
  bool ok;
};

// Workgroup -> (sequence, piece, key-value head, query group), such that all heads and
// query groups of a piece go to the same XCD (every eighth workgroup does).  Eight pieces at
// least give every XCD work.
__device__ inline Unit unit_of(const AttendArgs& a) {
  Unit x;
  int64_t y = blockIdx.x / 8;
  x.mg = static_cast<int>(y % a.mgroups);
  y /= a.mgroups;
  x.kvh = static_cast<int>(y % a.heads);
  const int64_t piece = y / a.heads * 8 + blockIdx.x % 8;
  x.split = static_cast<int>(piece % a.splits);
  x.b = static_cast<int>(piece / a.splits);
  x.ok = x.b < a.rows.B;
  return x;
}

// Up to 16 MT queries: one workgroup per (sequence, key-value head, piece, query group),
// whose four waves share the piece's positions and join their m, l and O in LDS.  Every
// byte is read once, by loads that take whole lines and do not stay in the caches (the
// values of bfloat16 with head_dim 64 by plain loads of 8 bytes a lane); the next tile's keys are fetched as soon as this one's are in LDS, its values after the
// second product.
template <int DT, int D, int MT>
__global__ __launch_bounds__(kThreads, 2) void attend_kernel(AttendArgs a) {
  using X = Ops<DT, D>;
  constexpr int kTile = 16 * X::kSub;
  __shared__ int16_t par_s[kMaxSeqRows];
  // The keys of each wave's tile, and after the last one what the waves join.
  __shared__ union {
    u32x4 k[kWaves][kTile * D * X::kBytes / 16];
    struct {
      f32x4 o[kWaves / 2][MT * X::kOut][64];
      float2 ml[kWaves / 2][MT][64];
    } join;
  } share_s;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = lane & 15, g = lane >> 4;
  const Unit x = unit_of(a);
  if (!x.ok) return;
  const SeqCall call = seq_call(a, x.b);
  const int rows = call.q.n, first = x.mg * MT * 16;
  if (first >= rows * a.group) return;
  const Sight sight = sight_of(a, call, first, MT * 16);
  const int k0 = x.split * a.span;
  if (x.split > 0 && k0 >= sight.end) return;
  const int k1 = min(k0 + a.span, sight.end);
  // The wave's positions [w0, w1), in whole tiles of the piece.
  const int share = (a.span / kTile + kWaves - 1) / kWaves * kTile;
  const int w0 = min(k0 + wave * share, k1), w1 = min(w0 + share, k1);
  PageWalk walk(a, call, w0, w1);
  if (call.q.tree && k1 > call.c && call.c >= 0) {
    for (int u = 1 + tid; u < rows; u += kThreads)
      par_s[u] = static_cast<int16_t>(node_parent(a.rows, x.b, true, u));
    __syncthreads();
  }
  Queries<X, MT> Q;
  Q.load(a, call, x.kvh, first);

  const unsigned v_lane = X::v_lane(n, g);
  const int64_t head_bytes = static_cast<int64_t>(x.kvh) * D * X::kBytes << a.page_log;
  const int in_page = (1 << a.page_log) - 1;
  // A tile's keys as they lie in memory: piece i of a lane is piece i * 64 + lane.
  constexpr int kRow = D * X::kBytes / 16;         // 16-byte pieces of a row
  constexpr int kPieces = kTile * kRow / 64;       // ... of a tile's keys per lane
  constexpr int kSubPieces = kPieces / X::kSub;
  constexpr int kSwizzle = kRow < 16 ? kRow - 1 : 15;
  u32x4 k[kPieces];
  typename X::V v;
  int64_t at[X::kSub];
  // Places the tile from j on; its bits that have a page.
  auto place = [&](int j) {
    unsigned pages = 0;
    walk.reach(j, kTile);
#pragma unroll
    for (int t = 0; t < X::kSub; ++t) {
      const int id = walk.at(j + 16 * t);
      pages |= id >= 0 ? 0xffffu << (16 * t) : 0u;
      at[t] = max(id, 0) * a.page_bytes + head_bytes +
              static_cast<int64_t>((j + 16 * t) & in_page) * (D * X::kBytes);
    }
    return pages;
  };
  auto load_k = [&]() {
#pragma unroll
    for (int t = 0; t < X::kSub; ++t)
#pragma unroll
      for (int i = 0; i < kSubPieces; ++i)
        k[t * kSubPieces + i] = load16(reinterpret_cast<const u32x4*>(a.k + at[t]) + i * 64 + lane);
  };
  auto load_v = [&]() {
#pragma unroll
    for (int t = 0; t < X::kSub; ++t) X::template load_v<true>(v, t, a.v + at[t], v_lane);
  };
  unsigned pages = 0;
  if (w0 < w1) {
    pages = place(w0);
    load_k();
    load_v();
  }
  using Weights = typename Queries<X, MT>::Weights;
  constexpr unsigned kWhole = X::kSub == 2 ? ~0u : 0xffffu;
  // Rows to operand layout through the wave's own LDS.  A row's pieces are exchanged by
  // the row's number, so that 16 rows' pieces spread over the banks.
  auto share_k = [&]() {
    constexpr int kRows = 64 / kRow;  // rows of a piece of all lanes
    const int row = lane / kRow, piece = (lane % kRow) ^ (row & kSwizzle);
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      share_s.k[wave][(i * kRows + row) * kRow + (piece ^ (i * kRows & kSwizzle))] = k[i];
    wave_sync();
  };
  auto scores = [&](Weights& p) {
#pragma unroll
    for (int t = 0; t < X::kSub; ++t) {
      u32x4 kf[X::kFrags];
#pragma unroll
      for (int f = 0; f < X::kFrags; ++f)
        kf[f] = share_s.k[wave][(16 * t + n) * kRow + ((4 * f + g) ^ (n & kSwizzle))];
      Q.score(p, t, kf);
    }
    wave_sync();
  };
  // Tiles that every query sees, then (without fetching ahead) those that some do not.
  int j0 = w0;
  for (; j0 + kTile <= min(sight.all, w1); j0 += kTile) {
    Weights p;
    share_k();
    const unsigned here = pages;
    const bool more = j0 + kTile < w1;
    if (more) {
      pages = place(j0 + kTile);
      if (MT == 1) load_k();
    }
    scores(p);
    // (With two query tiles the registers are short until the scores are there.)
    if (more && MT > 1) load_k();
    if (here != kWhole) Q.hide(p, v, here);
    Q.soften(p, a.scale_log2);
    X::template outputs<MT>(Q.o, Q.sum, v, p);
    if (more) load_v();
  }
#pragma unroll 1
  for (; j0 < w1; j0 += kTile) {
    Weights p;
    share_k();
    scores(p);
    const unsigned any = Q.visible(j0, sight.end, pages);
    Q.hide(p, v, any);
    unsigned see[MT];
    Q.mask(p, see, j0, any, a, call, par_s);
    Q.soften(p, a.scale_log2);
    if (__any(X::odd(v))) X::template poison<MT>(Q.o, v, p, see);
    X::template outputs<MT>(Q.o, Q.sum, v, p);
    if (j0 + kTile < w1) {
      pages = place(j0 + kTile);
      load_k();
      load_v();
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
    if constexpr (!X::kSums) Q.sum[m][0] = rows_sum(Q.sum[m][0]);

  // The waves join, halves at a time.
#pragma unroll
  for (int half = kWaves / 2; half > 0; half /= 2) {
    __syncthreads();
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        share_s.join.ml[wave - half][m][lane] = make_float2(Q.mx[m], Q.sum[m][0]);
#pragma unroll
        for (int j = 0; j < X::kOut; ++j) share_s.join.o[wave - half][m * X::kOut + j][lane] = Q.o[m][j];
      }
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float2 y = share_s.join.ml[wave][m][lane];
        const float now = fmaxf(Q.mx[m], y.x);
        const float fa = __builtin_amdgcn_exp2f(Q.mx[m] - now);
        const float fb = __builtin_amdgcn_exp2f(y.x - now);
        Q.mx[m] = now;
        Q.sum[m][0] = Q.sum[m][0] * fa + y.y * fb;
#pragma unroll
        for (int j = 0; j < X::kOut; ++j)
          Q.o[m][j] = Q.o[m][j] * fa + share_s.join.o[wave][m * X::kOut + j][lane] * fb;
      }
    }
  }
  if (wave == 0) Q.store(a, call, x.kvh, x.split);
}

// Many queries: one workgroup per (sequence, key-value head, piece, query group) whose
// four waves take MT tiles of 16 queries each and share every tile of keys and values
// through LDS, where the next one is put while this one is used.
template <int DT, int D, int MT>
__global__ __launch_bounds__(kThreads, 2) void attend_wide_kernel(AttendArgs a) {
  using X = Ops<DT, D>;
  constexpr int kStep = 16 * X::kSub;                // positions per product
  constexpr int kTile = 2 * kStep;                   // positions in LDS at a time
  constexpr int kRow = D * X::kBytes / 16;           // 16-byte pieces of a row
  constexpr int kLoads = kTile * kRow / kThreads;    // ... of k (and of v) per thread
  constexpr int kSwizzle = kRow < 16 ? kRow - 1 : 15;
  __shared__ int16_t par_s[kMaxSeqRows];
  __shared__ u32x4 k_s[2][kTile * kRow], v_s[2][kTile * kRow];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = lane & 15, g = lane >> 4;
  const Unit x = unit_of(a);
  if (!x.ok) return;
  const SeqCall call = seq_call(a, x.b);
  const int rows = call.q.n, first = x.mg * kWaves * MT * 16;
  if (first >= rows * a.group) return;
  // Where the last waves have no query, two workgroups of a CU leave different SIMDs idle
  // (an XCD's 32 CUs get one workgroup each before any gets a second).
  const int set = (wave + (blockIdx.x >> 8 & 1) * 2) % kWaves;
  const int mine = first + set * MT * 16;
  const bool work = mine < rows * a.group;
  const Sight sight = sight_of(a, call, first, kWaves * MT * 16);
  const int k0 = x.split * a.span;
  if (x.split > 0 && k0 >= sight.end) return;
  const int k1 = min(k0 + a.span, sight.end);
  PageWalk walk(a, call, k0, k1);
  if (call.q.tree && k1 > call.c && call.c >= 0)
    for (int u = 1 + tid; u < rows; u += kThreads)
      par_s[u] = static_cast<int16_t>(node_parent(a.rows, x.b, true, u));
  Queries<X, MT> Q;
  Q.load(a, call, x.kvh, mine);

  const int64_t head_bytes = static_cast<int64_t>(x.kvh) * D * X::kBytes << a.page_log;
  const int in_page = (1 << a.page_log) - 1;
  u32x4 stage_k[kLoads], stage_v[kLoads];
  // Piece i of a thread: row (i * 256 + tid) / kRow of the tile.  The rows of a wave's
  // load lie in one sub-tile, so their page is uniform.
  auto fetch = [&](int j) {
    walk.reach(j, kTile);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = (i * kThreads + tid) / kRow, piece = (i * kThreads + tid) % kRow;
      const int sub = __builtin_amdgcn_readfirstlane(row >> 4);
      const int id = walk.at(j + 16 * sub);
      const int64_t at = max(id, 0) * a.page_bytes + head_bytes +
                         static_cast<int64_t>((j + 16 * sub) & in_page) * (D * X::kBytes);
      const unsigned off = ((row & 15) * kRow + piece) * 16;
      stage_k[i] = load16(reinterpret_cast<const u32x4*>(a.k + at + off));
      stage_v[i] = load16(reinterpret_cast<const u32x4*>(a.v + at + off));
    }
    unsigned long long pages = 0;
#pragma unroll
    for (int t = 0; t < kTile / 16; ++t)
      pages |= walk.at(j + 16 * t) >= 0 ? 0xffffull << (16 * t) : 0ull;
    return pages;
  };
  // Keys are read a row per lane: a row's pieces are rotated among each other by the row
  // so that 16 rows' pieces spread over the banks.  Values are read 16 lanes a row.
  auto put = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = (i * kThreads + tid) / kRow, piece = (i * kThreads + tid) % kRow;
      k_s[buf][row * kRow + (piece ^ (row & kSwizzle))] = stage_k[i];
      v_s[buf][row * kRow + piece] = stage_v[i];
    }
  };
  unsigned long long pages = 0;
  if (k0 < k1) {
    pages = fetch(k0);
    put(0);
  }
  __syncthreads();
  using Weights = typename Queries<X, MT>::Weights;
  constexpr unsigned kWhole = X::kSub == 2 ? ~0u : 0xffffu;
  int buf = 0;
  // The scores and values of half h of the tile in LDS.
  auto take = [&](Weights& p, typename X::V& v, int h) {
#pragma unroll
    for (int t = 0; t < X::kSub; ++t) {
      u32x4 k[X::kFrags];
      const int row = h * kStep + 16 * t + n;
#pragma unroll
      for (int f = 0; f < X::kFrags; ++f) k[f] = k_s[buf][row * kRow + ((4 * f + g) ^ (n & kSwizzle))];
      Q.score(p, t, k);
    }
    const unsigned char* vp = reinterpret_cast<const unsigned char*>(v_s[buf]);
#pragma unroll
    for (int t = 0; t < X::kSub; ++t)
      X::template load_v<false>(v, t, vp + (h * kStep + 16 * t) * kRow * 16, X::v_lane(n, g));
  };
  // Tiles that every query sees, then (without fetching ahead) those that some do not.
  int j0 = k0;
  for (; j0 + kTile <= min(sight.all, k1); j0 += kTile) {
    const unsigned long long here = pages;
    const bool more = j0 + kTile < k1;
    if (more) pages = fetch(j0 + kTile);
    if (work) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        Weights p;
        typename X::V v;
        take(p, v, h);
        const unsigned have = static_cast<unsigned>(here >> (h * kStep)) & kWhole;
        if (have != kWhole) Q.hide(p, v, have);
        Q.soften(p, a.scale_log2);
        X::template outputs<MT>(Q.o, Q.sum, v, p);
      }
    }
    if (more) put(buf ^ 1);
    __syncthreads();
    buf ^= 1;
  }
  for (; j0 < k1; j0 += kTile) {
#pragma unroll 1
    for (int h = 0; work && h < 2; ++h) {
      const int j = j0 + h * kStep;
      if (j >= k1) break;
      Weights p;
      typename X::V v;
      take(p, v, h);
      const unsigned any = Q.visible(j, sight.end, static_cast<unsigned>(pages >> (h * kStep)));
      Q.hide(p, v, any);
      unsigned see[MT];
      Q.mask(p, see, j, any, a, call, par_s);
      Q.soften(p, a.scale_log2);
      if (__any(X::odd(v))) X::template poison<MT>(Q.o, v, p, see);
      X::template outputs<MT>(Q.o, Q.sum, v, p);
    }
    if (j0 + kTile < k1) {
      pages = fetch(j0 + kTile);
      put(buf ^ 1);
    }
    __syncthreads();
    buf ^= 1;
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
    if constexpr (!X::kSums) Q.sum[m][0] = rows_sum(Q.sum[m][0]);
  Q.store(a, call, x.kvh, x.split);
}

// Query tiles per wave, and whether the waves take tiles of their own.
struct Shape {
  int mt;
  bool wide;
};

// (64 sequences x 8 rows, two tiles: positions apart 267 us, queries apart 286; head_dim 64:
// 143 and 161.)
Shape attend_shape(int tiles, int dtype) {
  if (tiles <= 1) return Shape{1, false};
  // (float32 operands of two tiles a wave do not fit the registers of two waves a SIMD.)
  if (dtype == WF_F32) return Shape{1, true};
  if (tiles <= 2) return Shape{2, false};
  if (tiles <= 4) return Shape{1, true};
  return Shape{2, true};
}

template <int DT, int D>
void launch_typed(const AttendArgs& a, Shape shape, int64_t blocks, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(blocks)), block(kThreads);
  if (!shape.wide && shape.mt == 1) {
    hipLaunchKernelGGL((attend_kernel<DT, D, 1>), grid, block, 0, stream, a);
  } else if (shape.mt == 1 && shape.wide) {
    hipLaunchKernelGGL((attend_wide_kernel<DT, D, 1>), grid, block, 0, stream, a);
  } else if constexpr (DT == WF_BF16) {
    if (shape.wide) {
      hipLaunchKernelGGL((attend_wide_kernel<DT, D, 2>), grid, block, 0, stream, a);
    } else {
      hipLaunchKernelGGL((attend_kernel<DT, D, 2>), grid, block, 0, stream, a);
    }
  }
}

template <int DT, int D>
void launch_join(const AttendArgs& a, hipStream_t stream) {
  const int64_t n = static_cast<int64_t>(a.rows.B) * a.rows.rmax * a.q_heads;
  hipLaunchKernelGGL((attend_join_kernel<DT, D>), dim3(static_cast<unsigned>((n + kWaves - 1) / kWaves)),
                     dim3(kThreads), 0, stream, a);
}

int query_tiles(const wf_page_cache& cache, const RowsArgs& rows, int32_t q_heads) {
  return static_cast<int>((static_cast<int64_t>(rows.rmax) * (q_heads / cache.heads) + 15) / 16);
}

int query_groups(const wf_page_cache& cache, const RowsArgs& rows, int32_t q_heads) {
  const int tiles = query_tiles(cache, rows, q_heads);
  const Shape s = attend_shape(tiles, cache.dtype);
  const int each = s.mt * (s.wide ? kWaves : 1);
  return (tiles + each - 1) / each;
}

}  // namespace

AttendPlan attend_plan(const wf_page_cache& cache, const RowsArgs& rows, int32_t q_heads,
                       int32_t max_context) {
  int64_t most = static_cast<int64_t>(max_context) + rows.rmax;
  const int64_t room = static_cast<int64_t>(cache.max_pages) * cache.page_size;
  most = most < room ? most : room;
  const int64_t one =
      static_cast<int64_t>(rows.B) * cache.heads * query_groups(cache, rows, q_heads);
  // Rounds of workgroups that the card's slots hold at a time, each as long as a piece's
  // positions, its start and end, and its part written and read again (all in positions).
  const Shape shape = attend_shape(query_tiles(cache, rows, q_heads), cache.dtype);
  const int64_t queries = 16 * shape.mt * (shape.wide ? kWaves : 1);
  const int64_t part = queries * 8 / (cache.dtype == WF_BF16 ? 4 : 8);
  int64_t splits = 1, best = INT64_MAX;
  for (int64_t rounds = 1; rounds <= kMaxRounds; ++rounds) {
    // The most pieces that take no more rounds.
    int64_t s = rounds * kSlots / one;
    const int64_t cap = most / kMinSpan < kMaxSplits ? most / kMinSpan : kMaxSplits;
    s = s > cap ? cap : s;
    if (s < 1) s = 1;
    const int64_t need = (one * s + kSlots - 1) / kSlots;
    const int64_t cost = need * (most / s + kStart + (s > 1 ? part : 0));
    if (cost < best) {
      best = cost;
      splits = s;
    }
  }
  int64_t span = (most + splits - 1) / splits;
  span = (span + kMinSpan - 1) / kMinSpan * kMinSpan;
  span = span < kMinSpan ? kMinSpan : span;
  splits = (most + span - 1) / span;
  return AttendPlan{static_cast<int32_t>(splits < 1 ? 1 : splits), static_cast<int32_t>(span)};
}

int64_t attend_blocks(const wf_page_cache& cache, const RowsArgs& rows, int32_t q_heads,
                      int32_t max_context) {
  const AttendPlan p = attend_plan(cache, rows, q_heads, max_context);
  const int64_t pieces = static_cast<int64_t>(rows.B) * p.splits;
  return (pieces + 7) / 8 * 8 * cache.heads * query_groups(cache, rows, q_heads);
}

size_t attend_workspace(const wf_page_cache& cache, const RowsArgs& rows, int32_t q_heads,
                        int32_t max_context, int64_t total_rows) {
  const AttendPlan p = attend_plan(cache, rows, q_heads, max_context);
  if (p.splits == 1) return 0;
  return static_cast<size_t>(p.splits) * total_rows * q_heads * (cache.head_dim + 2) * sizeof(float);
}

hipError_t launch_attend(const void* q, int64_t q_stride, int32_t q_heads,
                         const wf_page_cache& cache, int32_t layer, const RowsArgs& rows,
                         const int32_t* seq, int32_t max_context, float scale, void* out,
                         void* workspace, int64_t total_rows, hipStream_t stream) {
  const int bytes = cache.dtype == WF_BF16 ? 2 : 4;
  const AttendPlan plan = attend_plan(cache, rows, q_heads, max_context);
  AttendArgs a{};
  a.rows = rows;
  a.q = static_cast<const unsigned char*>(q);
  a.q_bytes = q_stride * bytes;
  a.q_heads = q_heads;
  a.group = q_heads / cache.heads;
  a.k = static_cast<const unsigned char*>(cache.k) + layer * cache.layer_stride * bytes;
  a.v = static_cast<const unsigned char*>(cache.v) + layer * cache.layer_stride * bytes;
  a.page_bytes = cache.page_stride * bytes;
  a.pages = cache.pages;
  a.heads = cache.heads;
  a.page_log = __builtin_ctz(static_cast<unsigned>(cache.page_size));
  a.seqs = cache.seqs;
  a.max_pages = cache.max_pages;
  a.table = cache.table;
  a.context = cache.context;
  a.seq = seq;
  a.max_context = max_context;
  // Above zero, so that a score of -inf stays one: 1e-30 makes all weights equal too.
  a.scale_log2 = fmaxf(fabsf(scale) * kLog2E, 1e-30f);
  a.flip = scale < 0.f ? (cache.dtype == WF_BF16 ? 0x80008000u : 0x80000000u) : 0u;
  a.out = static_cast<unsigned char*>(out);
  a.splits = plan.splits;
  a.span = plan.span;
  a.mgroups = query_groups(cache, rows, q_heads);
  a.row_heads = total_rows * q_heads;
  a.part_o = static_cast<float*>(workspace);
  if (plan.splits > 1)
    a.part_ml = reinterpret_cast<float2*>(a.part_o + plan.splits * a.row_heads * cache.head_dim);
  const Shape shape = attend_shape(query_tiles(cache, rows, q_heads), cache.dtype);
  const int64_t blocks = attend_blocks(cache, rows, q_heads, max_context);
  const bool bf16 = cache.dtype == WF_BF16, wide = cache.head_dim == 128;
  if (bf16 && wide) launch_typed<WF_BF16, 128>(a, shape, blocks, stream);
  if (bf16 && !wide) launch_typed<WF_BF16, 64>(a, shape, blocks, stream);
  if (!bf16 && wide) launch_typed<WF_F32, 128>(a, shape, blocks, stream);
  if (!bf16 && !wide) launch_typed<WF_F32, 64>(a, shape, blocks, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || plan.splits == 1) return e;
  if (bf16 && wide) launch_join<WF_BF16, 128>(a, stream);
  if (bf16 && !wide) launch_join<WF_BF16, 64>(a, stream);
  if (!bf16 && wide) launch_join<WF_F32, 128>(a, stream);
  if (!bf16 && !wide) launch_join<WF_F32, 64>(a, stream);
  return hipGetLastError();
}

}  // namespace wf
