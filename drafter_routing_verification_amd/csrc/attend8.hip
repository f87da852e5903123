// Attention of a round's rows over the paged cache of 8 bits (whiflash_attend8).
//
// Per sequence and key-value head, the rows x (q_heads / heads) queries that share its keys form
// tiles of 16; a workgroup takes up to five of them over a piece of the positions, its four waves
// a share of the piece each, with a one-pass softmax in registers (attend_body.h), and joins them
// in LDS.  Pieces are joined by a second launch.
//
// An e4m3 number under a power-of-two scale is a bfloat16 number, so keys and values go to the
// matrix units as bfloat16 without loss, each widened with its own position's scale by one
// instruction for two.  Float32 queries and weights are cut into three bfloat16 parts of eight
// bits, which hold them exactly: three products of bfloat16 (48 cycles for 32 positions or
// dimensions) where those of float32 take 256.
//
// Keys need no LDS: the order of the dimensions in the first product is free if the queries take
// the same, and lane (n, g) takes bytes [64 i + 16 g, + 16) of row n, which are 64 bytes of a row
// for the four lanes of a load.
#include "attend_body.h"
#include "decode.h"
#include "dpp.h"
#include "e4m3.h"

namespace wf {
namespace {

constexpr int kTile = 32;          // positions per product
constexpr int kMinSpan = 4 * kTile;
constexpr int kMaxSplits = 512;

struct Attend8Args : AttendArgs {
  const unsigned char *k_scale, *v_scale;  // the layer
  int64_t scale_page;
  int block_log;
};

// Two e4m3 numbers of a word's half under a scale, as bfloat16.
template <bool HI>
__device__ inline unsigned widen(unsigned w, float scale) {
  return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, HI));
}

// The first eight bits of a float32 number's fraction, as a bfloat16 number in the upper half.
__device__ inline float upper(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }
__device__ inline unsigned uppers(float lo, float hi) {
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}

template <int DT, int D>
struct Ops8 {
  static constexpr int kD = D;
  static constexpr int kSub = 2;
  static constexpr bool kSums = DT == WF_BF16;
  static constexpr int kParts = DT == WF_BF16 ? 1 : 3;
  static constexpr int kFrags = D / 32;
  static constexpr int kQ = kParts * kFrags;
  static constexpr int kOut = D / 16;
  static constexpr int kBytes = DT == WF_BF16 ? 2 : 4;
  static constexpr int kWords = D / 32;     // bfloat16 pairs of a lane's share of a row of V
  struct V {
    unsigned w[8][kWords];                  // [position][dimension pairs]
  };
  // A lane's share of a tile as it lies in memory.
  struct Raw {
    u32x4 k[2][D / 64];
    unsigned v[8][D / 64];
    unsigned scale;                         // lanes 0 - 31: the keys' byte of a position, then the values'
  };

  // Fragment f: dimensions 64 (f / 2) + 16 g + 8 (f % 2) and the seven behind it.
  __device__ static inline u32x4 q_fragment(const unsigned char* p, int f, int g, unsigned flip) {
    const int part = f / kFrags, at = 64 * (f % kFrags / 2) + 16 * g + 8 * (f % 2);
    const u32x4* from = reinterpret_cast<const u32x4*>(p + at * kBytes);
    if constexpr (DT == WF_BF16) return from[0] ^ flip;
    const u32x4 a = from[0] ^ flip, b = from[1] ^ flip;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = __uint_as_float(e < 4 ? a[e] : b[e - 4]);
      if (part > 0) x[e] -= upper(x[e]);
      if (part > 1) x[e] -= upper(x[e]);
    }
    return u32x4{uppers(x[0], x[1]), uppers(x[2], x[3]), uppers(x[4], x[5]), uppers(x[6], x[7])};
  }

  __device__ static inline f32x4 scores(const u32x4* k, const u32x4* q) {
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int part = kParts - 1; part >= 0; --part)
#pragma unroll
      for (int f = 0; f < kFrags; ++f)
        s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k[f]),
                                                    __builtin_bit_cast(bf16x8, q[part * kFrags + f]), s, 0, 0, 0);
    return s;
  }

  // The keys of sub-tile t, under the scale of the lane's position.
  __device__ static inline void keys(u32x4* k, const Raw& raw, int t, float scale) {
#pragma unroll
    for (int f = 0; f < kFrags; ++f) {
      const unsigned lo = raw.k[t][f / 2][2 * (f % 2)], hi = raw.k[t][f / 2][2 * (f % 2) + 1];
      k[f] = u32x4{widen<false>(lo, scale), widen<true>(lo, scale), widen<false>(hi, scale), widen<true>(hi, scale)};
    }
  }
  // The values, under the scales of the positions (bytes of scale[t]: those of 4 g + i).
  __device__ static inline void values(V& v, const Raw& raw, const unsigned* scale) {
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const float s = __uint_as_float((r % 4 < 3 ? scale[r / 4] << (23 - 8 * (r % 4) < 0 ? 0 : 23 - 8 * (r % 4))
                                                 : scale[r / 4] >> 1) & 0x7f800000u);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        v.w[r][2 * c] = widen<false>(raw.v[r][c], s);
        v.w[r][2 * c + 1] = widen<true>(raw.v[r][c], s);
      }
    }
  }
  __device__ static inline void zero_v(V& v, int t, int i) {
#pragma unroll
    for (int x = 0; x < kWords; ++x) v.w[4 * t + i][x] = 0;
  }

  // o += V^T P^T for MT query tiles.  bfloat16: the weights rounded as the matrix units take them
  // (a part in 2^8 each), and summed as rounded, so that equal values come out as they are.
  // float32: in three parts, exactly.
  template <int MT>
  __device__ static inline void outputs(f32x4 (*o)[kOut], f32x4* sum, const V& v,
                                        const float (*p)[kSub][4]) {
    bf16x8 pb[MT][kParts];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if constexpr (kParts == 1) {
        pb[m][0] = __builtin_bit_cast(bf16x8, (u32x4{pack_bf16(p[m][0][0], p[m][0][1]), pack_bf16(p[m][0][2], p[m][0][3]),
                                                     pack_bf16(p[m][1][0], p[m][1][1]), pack_bf16(p[m][1][2], p[m][1][3])}));
      } else {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = p[m][e / 4][e % 4];
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          pb[m][part] = __builtin_bit_cast(bf16x8, (u32x4{uppers(x[0], x[1]), uppers(x[2], x[3]), uppers(x[4], x[5]), uppers(x[6], x[7])}));
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] -= upper(x[e]);
        }
      }
    }
    if constexpr (kSums) {
      const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u});
#pragma unroll
      for (int m = 0; m < MT; ++m)
        sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, pb[m][0], sum[m], 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kOut; ++j) {
      // Element j of each position's dimensions, two positions a word.
      unsigned w[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
        w[x] = __builtin_amdgcn_perm(v.w[2 * x + 1][j >> 1], v.w[2 * x][j >> 1],
                                     (j & 1) ? 0x07060302u : 0x05040100u);
      const bf16x8 a = __builtin_bit_cast(bf16x8, (u32x4{w[0], w[1], w[2], w[3]}));
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int part = kParts - 1; part >= 0; --part)
          o[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, pb[m][part], o[m][j], 0, 0, 0);
    }
  }

  __device__ static inline bool odd(const V& v) {
    bool x = false;
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int c = 0; c < kWords; ++c)
        x = x || (v.w[r][c] & 0x7f80u) == 0x7f80u || (v.w[r][c] & 0x7f800000u) == 0x7f800000u;
    return x;
  }
  // NaN among the values that not every query sees go apart from the product, where they would
  // meet the weights of zero of those queries too: they make NaN of the outputs that see them,
  // and zeros take their place.
  template <int MT>
  __device__ static inline void poison(f32x4 (*o)[kOut], V& v, const unsigned* see) {
    const int g = (threadIdx.x & 63) >> 4;
    bf16x8 pb[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      unsigned w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int r = 0; r < 8; ++r)
        w[r / 2] |= see[m] >> (16 * (r / 4) + 4 * g + r % 4) & 1u ? 0x3f80u << (r % 2 * 16) : 0u;
      pb[m] = __builtin_bit_cast(bf16x8, (u32x4{w[0], w[1], w[2], w[3]}));
    }
#pragma unroll
    for (int j = 0; j < kOut; ++j) {
      unsigned w[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const unsigned mask = (j & 1) ? 0x7f800000u : 0x7f80u;
        w[x] = (v.w[2 * x][j >> 1] & mask) == mask ? 0x3f80u : 0u;
        w[x] |= (v.w[2 * x + 1][j >> 1] & mask) == mask ? 0x3f800000u : 0u;
      }
      const bf16x8 a = __builtin_bit_cast(bf16x8, (u32x4{w[0], w[1], w[2], w[3]}));
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f32x4 n = {0.f, 0.f, 0.f, 0.f};
        n = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, pb[m], n, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[m][j][i] += n[i] > 0.f ? NAN : 0.f;
      }
    }
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int c = 0; c < kWords; ++c) {
        const unsigned x = v.w[r][c];
        v.w[r][c] = ((x & 0x7f80u) == 0x7f80u ? 0u : x & 0xffffu) |
                    ((x & 0x7f800000u) == 0x7f800000u ? 0u : x & 0xffff0000u);
      }
  }

  // Element i of every output tile of one query (dimensions (4 g + i) D / 16 and on), times f.
  __device__ static inline void store_out(unsigned char* out, const f32x4* o, int g, float f) {
    if constexpr (DT == WF_BF16) {
      store_query<WF_BF16, D>(out, o, g, f);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < kOut; j += 4)
          *reinterpret_cast<f32x4*>(out + ((4 * g + i) * kOut + j) * 4) =
              f32x4{o[j][i] * f, o[j + 1][i] * f, o[j + 2][i] * f, o[j + 3][i] * f};
    }
  }
  __device__ static inline void store_part(float* out, const f32x4* o, int g) {
    store_partial<WF_BF16, D>(out, o, g);
  }
};

struct Unit {
  int split, b, kvh, mg;
  bool ok;
};

// Workgroup -> (sequence, piece, key-value head, query group), such that the query groups of a
// head's piece, which read the same keys and values, go to the same XCD (every eighth workgroup
// does), and all else is spread over the XCDs.
__device__ inline Unit unit_of(const AttendArgs& a) {
  Unit x;
  const int y = blockIdx.x / 8;
  x.mg = y % a.mgroups;
  const int64_t part = static_cast<int64_t>(y / a.mgroups) * 8 + blockIdx.x % 8;
  x.kvh = static_cast<int>(part % a.heads);
  const int64_t piece = part / a.heads;
  x.split = static_cast<int>(piece % a.splits);
  x.b = static_cast<int>(piece / a.splits);
  x.ok = x.b < a.rows.B;
  return x;
}

template <int DT, int D, int MT, int PER_SIMD>
__global__ __launch_bounds__(kThreads, PER_SIMD) void attend8_kernel(Attend8Args a) {
  using X = Ops8<DT, D>;
  __shared__ int16_t par_s[kMaxSeqRows];
  __shared__ struct {
    f32x4 o[kWaves / 2][MT * X::kOut][64];
    float2 ml[kWaves / 2][MT][64];
  } join_s;
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

  const int64_t head_bytes = static_cast<int64_t>(x.kvh) * D << a.page_log;
  const int64_t head_scale = static_cast<int64_t>(x.kvh) << (a.page_log - a.block_log);
  const int in_page = (1 << a.page_log) - 1;
  const unsigned k_lane = n * D + 16 * g, v_lane = 4 * g * D + n * (D / 16);
  const unsigned char* scales = lane < 32 ? a.k_scale : a.v_scale;
  typename X::Raw raw;
  int id[2];
  // Places the tile from j on; its bits that have a page.
  auto place = [&](int j) {
    walk.reach(j, kTile);
    unsigned pages = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      id[t] = walk.at(j + 16 * t);
      pages |= id[t] >= 0 ? 0xffffu << (16 * t) : 0u;
    }
    return pages;
  };
  auto load_k = [&](int j) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const unsigned char* p = a.k + max(id[t], 0) * a.page_bytes + head_bytes +
                               static_cast<int64_t>((j + 16 * t) & in_page) * D;
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
        raw.k[t][i] = load16(reinterpret_cast<const u32x4*>(p + k_lane + 64 * i));
    }
    const int mine = lane & 16 ? id[1] : id[0];
    raw.scale = scales[max(mine, 0) * a.scale_page + head_scale + (((j + (lane & 31)) & in_page) >> a.block_log)];
  };
  auto load_v = [&](int j) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const unsigned char* p = a.v + max(id[t], 0) * a.page_bytes + head_bytes +
                               static_cast<int64_t>((j + 16 * t) & in_page) * D;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (D == 128) {
          typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
          const u32x2 y = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p + v_lane + i * D));
          raw.v[4 * t + i][0] = y.x;
          raw.v[4 * t + i][1] = y.y;
        } else {
          raw.v[4 * t + i][0] = __builtin_nontemporal_load(reinterpret_cast<const unsigned*>(p + v_lane + i * D));
        }
      }
    }
  };
  // Scales to the lanes that use them: keys' of position n, values' of positions 4 g + i (a byte each).
  auto spread = [&](float* ks, unsigned* vs) {
    const unsigned byte = raw.scale;
    unsigned four = byte << (8 * (lane & 3));
    four |= static_cast<unsigned>(dpp_mov<kDppQuadXor1>(static_cast<int>(four)));
    four |= static_cast<unsigned>(dpp_mov<kDppQuadXor2>(static_cast<int>(four)));
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      ks[t] = __uint_as_float(static_cast<unsigned>(__builtin_amdgcn_ds_bpermute(4 * (16 * t + n), static_cast<int>(byte << 23))));
      vs[t] = static_cast<unsigned>(__builtin_amdgcn_ds_bpermute(4 * (32 + 16 * t + 4 * g), static_cast<int>(four)));
    }
  };
  unsigned pages = 0;
  if (w0 < w1) {
    pages = place(w0);
    load_k(w0);
    load_v(w0);
  }
  using Weights = typename Queries<X, MT>::Weights;
  // The products of the tile at hand with the queries; its values; the loads of the next tile.
  auto take = [&](Weights& p, typename X::V& v, int next) {
    float ks[2];
    unsigned vs[2];
    spread(ks, vs);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      u32x4 k[X::kFrags];
      X::keys(k, raw, t, ks[t]);
      Q.score(p, t, k);
    }
    X::values(v, raw, vs);
    const unsigned here = pages;
    if (next < w1) {
      pages = place(next);
      load_k(next);
      load_v(next);
    }
    return here;
  };
  // Tiles that every query sees, then those that some do not.
  int j0 = w0;
  for (; j0 + kTile <= min(sight.all, w1); j0 += kTile) {
    Weights p;
    typename X::V v;
    const unsigned here = take(p, v, j0 + kTile);
    if (here != ~0u) Q.hide(p, v, here);
    Q.soften(p, a.scale_log2);
    X::template outputs<MT>(Q.o, Q.sum, v, p);
  }
#pragma unroll 1
  for (; j0 < w1; j0 += kTile) {
    Weights p;
    typename X::V v;
    const unsigned any = Q.visible(j0, sight.end, take(p, v, j0 + kTile));
    Q.hide(p, v, any);
    unsigned see[MT];
    Q.mask(p, see, j0, any, a, call, par_s);
    Q.soften(p, a.scale_log2);
    if (__any(X::odd(v))) X::template poison<MT>(Q.o, v, see);
    X::template outputs<MT>(Q.o, Q.sum, v, p);
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
        join_s.ml[wave - half][m][lane] = make_float2(Q.mx[m], Q.sum[m][0]);
#pragma unroll
        for (int j = 0; j < X::kOut; ++j) join_s.o[wave - half][m * X::kOut + j][lane] = Q.o[m][j];
      }
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float2 y = join_s.ml[wave][m][lane];
        const float now = fmaxf(Q.mx[m], y.x);
        const float fa = __builtin_amdgcn_exp2f(Q.mx[m] - now);
        const float fb = __builtin_amdgcn_exp2f(y.x - now);
        Q.mx[m] = now;
        Q.sum[m][0] = Q.sum[m][0] * fa + y.y * fb;
#pragma unroll
        for (int j = 0; j < X::kOut; ++j)
          Q.o[m][j] = Q.o[m][j] * fa + join_s.o[wave][m * X::kOut + j][lane] * fb;
      }
    }
  }
  if (wave == 0) Q.store(a, call, x.kvh, x.split);
}

// Query tiles of a workgroup, and workgroups of a CU.
struct Shape {
  int mt, per_cu;
};

Shape shape_of(int tiles, int dtype) {
  if (dtype == WF_F32) return tiles <= 1 ? Shape{1, 2} : Shape{2, 1};
  if (tiles <= 1) return Shape{1, 2};
  if (tiles <= 2) return Shape{2, 2};
  return Shape{3, 1};
}

template <int DT, int D>
void launch_typed(const Attend8Args& a, Shape s, int64_t blocks, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(blocks)), block(kThreads);
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
  if constexpr (DT == WF_F32) {
    s.mt == 1 ? go(attend8_kernel<DT, D, 1, 2>) : go(attend8_kernel<DT, D, 2, 1>);
  } else {
    if (s.mt == 1) go(attend8_kernel<DT, D, 1, 2>);
    if (s.mt == 2) go(attend8_kernel<DT, D, 2, 2>);
    if (s.mt == 3) go(attend8_kernel<DT, D, 3, 1>);
  }
}

template <int DT, int D>
void launch_join(const AttendArgs& a, hipStream_t stream) {
  const int64_t n = static_cast<int64_t>(a.rows.B) * a.rows.rmax * a.q_heads;
  hipLaunchKernelGGL((attend_join_kernel<DT, D>), dim3(static_cast<unsigned>((n + kWaves - 1) / kWaves)),
                     dim3(kThreads), 0, stream, a);
}

// How a call is cut: `splits` pieces of `span` positions a sequence, `groups` query groups a head.
struct Plan8 {
  Shape shape;
  int groups, splits, span;
};

Plan8 plan_of(const wf_page_cache8& cache, const RowsArgs& rows, int dtype, int32_t q_heads,
              int32_t max_context) {
  const wf_page_cache& c = cache.pages;
  Plan8 p;
  const int tiles = static_cast<int>((static_cast<int64_t>(rows.rmax) * (q_heads / c.heads) + 15) / 16);
  p.shape = shape_of(tiles, dtype);
  p.groups = (tiles + p.shape.mt - 1) / p.shape.mt;
  int64_t most = static_cast<int64_t>(max_context) + rows.rmax;
  const int64_t room = static_cast<int64_t>(c.max_pages) * c.page_size;
  most = most < room ? most : room;
  const int64_t one = static_cast<int64_t>(rows.B) * c.heads * p.groups;
  const int64_t slots = 256 * p.shape.per_cu;
  int64_t best = INT64_MAX, splits = 1;
  for (int64_t rounds = 1; rounds <= 8; ++rounds) {
    int64_t s = rounds * slots / one;
    const int64_t cap = most / kMinSpan < kMaxSplits ? most / kMinSpan : kMaxSplits;
    s = s > cap ? cap : s;
    s = s < 1 ? 1 : s;
    const int64_t need = (one * s + slots - 1) / slots;
    const int64_t cost = need * (most / s + 256 + (s > 1 ? 32 * p.shape.mt : 0));
    if (cost < best) {
      best = cost;
      splits = s;
    }
  }
  int64_t span = (most + splits - 1) / splits;
  span = (span + kMinSpan - 1) / kMinSpan * kMinSpan;
  span = span < kMinSpan ? kMinSpan : span;
  splits = (most + span - 1) / span;
  p.splits = static_cast<int>(splits < 1 ? 1 : splits);
  p.span = static_cast<int>(span);
  return p;
}

int64_t blocks_of(const wf_page_cache8& cache, const RowsArgs& rows, const Plan8& p) {
  const int64_t parts = static_cast<int64_t>(rows.B) * p.splits * cache.pages.heads;
  return (parts + 7) / 8 * 8 * p.groups;
}

}  // namespace

int64_t attend8_blocks(const wf_page_cache8& cache, const RowsArgs& rows, int dtype, int32_t q_heads,
                       int32_t max_context) {
  return blocks_of(cache, rows, plan_of(cache, rows, dtype, q_heads, max_context));
}

size_t attend8_workspace(const wf_page_cache8& cache, const RowsArgs& rows, int dtype,
                         int32_t q_heads, int32_t max_context, int64_t total_rows) {
  const Plan8 p = plan_of(cache, rows, dtype, q_heads, max_context);
  if (p.splits == 1) return 0;
  return static_cast<size_t>(p.splits) * total_rows * q_heads * (cache.pages.head_dim + 2) * sizeof(float);
}

hipError_t launch_attend8(const void* q, int64_t q_stride, int32_t q_heads, int dtype,
                          const wf_page_cache8& cache, int32_t layer, const RowsArgs& rows,
                          const int32_t* seq, int32_t max_context, float scale, void* out,
                          void* workspace, int64_t total_rows, hipStream_t stream) {
  const Plan8 plan = plan_of(cache, rows, dtype, q_heads, max_context);
  const bool bf16 = dtype == WF_BF16, wide = cache.pages.head_dim == 128;
  Attend8Args a{};
  a.rows = rows;
  a.q = static_cast<const unsigned char*>(q);
  a.q_bytes = q_stride * (bf16 ? 2 : 4);
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
  // Above zero, so that a score of -inf stays one: 1e-30 makes all weights equal too.
  a.scale_log2 = fmaxf(fabsf(scale) * kLog2E, 1e-30f);
  a.flip = scale < 0.f ? (bf16 ? 0x80008000u : 0x80000000u) : 0u;
  a.out = static_cast<unsigned char*>(out);
  a.splits = plan.splits;
  a.span = plan.span;
  a.mgroups = plan.groups;
  a.row_heads = total_rows * q_heads;
  a.part_o = static_cast<float*>(workspace);
  if (plan.splits > 1)
    a.part_ml = reinterpret_cast<float2*>(a.part_o + plan.splits * a.row_heads * cache.pages.head_dim);
  const int64_t blocks = blocks_of(cache, rows, plan);
  if (bf16 && wide) launch_typed<WF_BF16, 128>(a, plan.shape, blocks, stream);
  if (bf16 && !wide) launch_typed<WF_BF16, 64>(a, plan.shape, blocks, stream);
  if (!bf16 && wide) launch_typed<WF_F32, 128>(a, plan.shape, blocks, stream);
  if (!bf16 && !wide) launch_typed<WF_F32, 64>(a, plan.shape, blocks, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || plan.splits == 1) return e;
  if (bf16 && wide) launch_join<WF_BF16, 128>(a, stream);
  if (bf16 && !wide) launch_join<WF_BF16, 64>(a, stream);
  if (!bf16 && wide) launch_join<WF_F32, 128>(a, stream);
  if (!bf16 && !wide) launch_join<WF_F32, 64>(a, stream);
  return hipGetLastError();
}

}  // namespace wf
