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

// All bits, or none: bit i of x.
__device__ inline unsigned all_of(unsigned x, int i) {
  return static_cast<unsigned>(static_cast<int>(x << (31 - i)) >> 31);
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
  // The scale of position r (4 t + i) out of the bytes of sub-tile t's.
  __device__ static inline float value_scale(const unsigned* bytes, int r) {
    const unsigned w = bytes[r / 4];
    const int up = 23 - 8 * (r % 4);
    return __uint_as_float((up >= 0 ? w << (up >= 0 ? up : 0) : w >> 1) & 0x7f800000u);
  }
  // Takes the values of positions without their bit out: 0 under a scale of 1.  any: a lane's
  // positions 4 g + i of sub-tile t at bit 16 t + i.
  __device__ static inline void hide(Raw& raw, unsigned* bytes, unsigned any) {
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const unsigned in = all_of(any, 16 * (r / 4) + r % 4);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) raw.v[r][c] &= in;
      const unsigned place = 0xffu << (8 * (r % 4));
      bytes[r / 4] = (bytes[r / 4] & (in | ~place)) | (127u << (8 * (r % 4)) & ~in);
    }
  }

  // o += V^T P^T for MT query tiles.  bfloat16: the weights rounded as the matrix units take them
  // (a part in 2^8 each), and summed as rounded, so that equal values come out as they are.
  // float32: in three parts, exactly.
  template <int MT>
  __device__ static inline void outputs(f32x4 (*o)[kOut], f32x4* sum, const Raw& raw,
                                        const unsigned* bytes, const float (*p)[kSub][4]) {
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
    float scale[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) scale[r] = value_scale(bytes, r);
    // The values are widened two dimensions at a time, so that few of them need registers.
#pragma unroll
    for (int c = 0; c < kOut / 2; ++c) {
      unsigned v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        v[r] = c % 2 ? widen<true>(raw.v[r][c / 2], scale[r]) : widen<false>(raw.v[r][c / 2], scale[r]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // Dimension 2 c + h of each position, two positions a word.
        unsigned w[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          w[x] = __builtin_amdgcn_perm(v[2 * x + 1], v[2 * x], h ? 0x07060302u : 0x05040100u);
        const bf16x8 a = __builtin_bit_cast(bf16x8, (u32x4{w[0], w[1], w[2], w[3]}));
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int part = kParts - 1; part >= 0; --part)
            o[m][2 * c + h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, pb[m][part], o[m][2 * c + h], 0, 0, 0);
      }
    }
  }

  // Whether the lane's values hold NaN (0x7f but for the sign).
  __device__ static inline bool odd(const Raw& raw) {
    unsigned x = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int c = 0; c < D / 64; ++c) x |= (raw.v[r][c] & 0x7f7f7f7fu) + 0x01010101u;
    return (x & 0x80808080u) != 0;
  }
  // Zeros in the place of NaN.
  __device__ static inline void clean(Raw& raw) {
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const unsigned is = ((raw.v[r][c] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
        raw.v[r][c] &= ~(is | (is - (is >> 7)));  // (0x80 and 0x7f of every such byte)
      }
  }
  // Makes NaN of the outputs that see one among the values.
  template <int MT>
  __device__ static inline void poison(f32x4 (*o)[kOut], const Raw& raw, const unsigned* see) {
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
      const unsigned mask = 0x7fu << (8 * (j % 4));
      unsigned w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int r = 0; r < 8; ++r)
        w[r / 2] |= (raw.v[r][j / 4] & mask) == mask ? 0x3f80u << (r % 2 * 16) : 0u;
      const bf16x8 a = __builtin_bit_cast(bf16x8, (u32x4{w[0], w[1], w[2], w[3]}));
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f32x4 n = {0.f, 0.f, 0.f, 0.f};
        n = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, pb[m], n, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[m][j][i] += n[i] > 0.f ? NAN : 0.f;
      }
      __builtin_amdgcn_sched_barrier(0);  // (one at a time: their results would all need registers)
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

// Products to weights 2^(scale q . k - m).  The reference m of a query is a maximum of its row that
// is raised only when a product exceeds it by more than kSlack8: bfloat16 and float32 hold weights
// up to 2^16 and their sums as well as those up to 1, and so most tiles need no maximum over the
// lanes and no rescaling.
constexpr float kSlack8 = 16.f;

template <class X, int MT>
__device__ inline void soften8(Queries<X, MT>& Q, typename Queries<X, MT>::Weights& p, float scale) {
  bool grown = false;
  float top[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    float x = p[m][0][0];
#pragma unroll
    for (int t = 0; t < X::kSub; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) x = fmaxf(x, p[m][t][i]);
    top[m] = x * scale;
    grown = grown || top[m] > Q.mx[m] + kSlack8;
  }
  if (__any(grown)) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const float now = fmaxf(Q.mx[m], rows_max(top[m]));
      const float f = __builtin_amdgcn_exp2f(Q.mx[m] - now);
      Q.mx[m] = now;
      Q.sum[m] *= f;
#pragma unroll
      for (int j = 0; j < X::kOut; ++j) Q.o[m][j] *= f;
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < X::kSub; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[m][t][i] = __builtin_amdgcn_exp2f(fmaf(p[m][t][i], scale, -Q.mx[m]));
        if constexpr (!X::kSums) Q.sum[m][0] += p[m][t][i];
      }
}

// Of the 32 positions from j0 on, of which `any` can be seen at all, those that the lane's query of
// tile m sees.
template <class X, int MT>
__device__ inline unsigned seen_of(const Queries<X, MT>& Q, int m, int j0, unsigned any,
                                   const AttendArgs& a, const SeqCall& call, const int16_t* par) {
  const int old = min(max(call.c - j0, 0), 32);
  unsigned bits = old >= 32 ? ~0u : (1u << old) - 1u;
  const int x0 = Q.query(a, call, m);
  const int own = x0 < 0 ? -1 : x0 / a.group, last = call.c + own - j0;
  if (!call.q.tree) {
    if (own >= 0 && last >= 0) bits = last >= 31 ? ~0u : (2u << last) - 1u;
  } else {
    for (int u = own; u >= 0 && call.c + u >= j0; u = u == 0 ? -1 : par[u]) {
      const int x = call.c + u - j0;
      if (x < 32) bits |= 1u << x;
    }
  }
  return bits & any;
}

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

// GS query groups a workgroup: its waves take a group each and 4 / GS shares of the piece.  The waves
// of a share read the same keys and values, from memory once and else from the CU's cache.
template <int DT, int D, int MT, int GS>
__global__ __launch_bounds__(kThreads, 2) void attend8_kernel(Attend8Args a) {
  using X = Ops8<DT, D>;
  constexpr int kShares = kWaves / GS;
  __shared__ int16_t par_s[kMaxSeqRows];
  __shared__ struct {
    f32x4 o[kShares > 1 ? kWaves / 2 : 1][MT * X::kOut][64];
    float2 ml[kShares > 1 ? kWaves / 2 : 1][MT][64];
  } join_s;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = lane & 15, g = lane >> 4;
  const Unit x = unit_of(a);
  if (!x.ok) return;
  const SeqCall call = seq_call(a, x.b);
  const int rows = call.q.n;
  const int all_first = x.mg * GS * MT * 16;
  if (all_first >= rows * a.group) return;
  const int k0 = x.split * a.span;
  const Sight all = sight_of(a, call, all_first, GS * MT * 16);
  if (x.split > 0 && k0 >= all.end) return;
  const int first = all_first + wave % GS * MT * 16;
  const bool work = first < rows * a.group;
  const Sight sight = sight_of(a, call, work ? first : all_first, MT * 16);
  const int k1 = work ? min(k0 + a.span, sight.end) : k0;
  // The wave's positions [w0, w1), in whole tiles of the piece.
  const int share = (a.span / kTile + kShares - 1) / kShares * kTile;
  const int w0 = min(k0 + wave / GS * share, k1), w1 = min(w0 + share, k1);
  PageWalk walk(a, call, w0, w1);
  if (call.q.tree && k0 + a.span > call.c && call.c >= 0) {
    for (int u = 1 + tid; u < rows; u += kThreads)
      par_s[u] = static_cast<int16_t>(node_parent(a.rows, x.b, true, u));
    __syncthreads();
  }
  // Three tiles of queries do not fit the registers beside their outputs: they stay in LDS.
  constexpr bool kInLds = MT * X::kQ > 8;
  __shared__ u32x4 q_s[kInLds ? GS : 1][kInLds ? MT * X::kQ : 1][64];
  Queries<X, MT> Q;
  Q.load(a, call, x.kvh, first);
  if constexpr (kInLds) {
    if (wave < GS)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int f = 0; f < X::kQ; ++f) q_s[wave][m * X::kQ + f][lane] = Q.q[m][f];
    __syncthreads();
  }

  const int64_t head_bytes = static_cast<int64_t>(x.kvh) * D << a.page_log;
  const int64_t head_scale = static_cast<int64_t>(x.kvh) << (a.page_log - a.block_log);
  const int in_page = (1 << a.page_log) - 1;
  const unsigned k_lane = n * D + 16 * g, v_lane = 4 * g * D + n * (D / 16);
  const unsigned char* scales = lane < 32 ? a.k_scale : a.v_scale;
  typename X::Raw raw;
  int id[2] = {-1, -1};
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
  // Loads that stay in the caches only where another wave wants them too.
  auto fetch = [&](auto* p) {
    if constexpr (GS > 1) return *p;
    return __builtin_nontemporal_load(p);
  };
  auto load_k = [&](int j) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const unsigned char* p = a.k + max(id[t], 0) * a.page_bytes + head_bytes +
                               static_cast<int64_t>((j + 16 * t) & in_page) * D;
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
        raw.k[t][i] = fetch(reinterpret_cast<const u32x4*>(p + k_lane + 64 * i));
    }
    // (A choice between the elements of an array would put it into memory.)
    const int mine = id[0] ^ ((id[0] ^ id[1]) & static_cast<int>(all_of(lane, 4)));
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
          const u32x2 y = fetch(reinterpret_cast<const u32x2*>(p + v_lane + i * D));
          raw.v[4 * t + i][0] = y.x;
          raw.v[4 * t + i][1] = y.y;
        } else {
          raw.v[4 * t + i][0] = fetch(reinterpret_cast<const unsigned*>(p + v_lane + i * D));
        }
      }
    }
  };
  unsigned pages = 0;
  if (w0 < w1) {
    pages = place(w0);
    load_k(w0);
    load_v(w0);
  }
  using Weights = typename Queries<X, MT>::Weights;
  // The products of the tile's keys with the queries, the scales of its values (a byte for each of
  // the positions 4 g + i), and the loads of the next tile's keys; the bits that have a page.
  auto scores = [&](Weights& p, unsigned* vs, int next) {
    const unsigned byte = raw.scale;
    unsigned four = byte << (8 * (lane & 3));
    four |= static_cast<unsigned>(dpp_mov<kDppQuadXor1>(static_cast<int>(four)));
    four |= static_cast<unsigned>(dpp_mov<kDppQuadXor2>(static_cast<int>(four)));
    float ks[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      ks[t] = __uint_as_float(static_cast<unsigned>(__builtin_amdgcn_ds_bpermute(4 * (16 * t + n), static_cast<int>(byte << 23))));
      vs[t] = static_cast<unsigned>(__builtin_amdgcn_ds_bpermute(4 * (32 + 16 * t + 4 * g), static_cast<int>(four)));
    }
    if constexpr (kInLds) {
      u32x4 k[2][X::kFrags];
      X::keys(k[0], raw, 0, ks[0]);
      X::keys(k[1], raw, 1, ks[1]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f32x4 sum[2] = {};
#pragma unroll
        for (int f = X::kQ - 1; f >= 0; --f) {
          const u32x4 q = q_s[wave % GS][m * X::kQ + f][lane];
#pragma unroll
          for (int t = 0; t < 2; ++t)
            sum[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k[t][f % X::kFrags]),
                                                             __builtin_bit_cast(bf16x8, q), sum[t], 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) p[m][t][i] = sum[t][i];
      }
    } else {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        u32x4 k[X::kFrags];
        X::keys(k, raw, t, ks[t]);
        Q.score(p, t, k);
      }
    }
    const unsigned here = pages;
    if (next < w1) {
      pages = place(next);
      load_k(next);
    }
    return here;
  };
  int odd_from = -1;  // the first tile with NaN that were taken out
#pragma unroll 1
  for (int j0 = w0; j0 < w1; j0 += kTile) {
    Weights p;
    unsigned vs[2];
    const unsigned here = scores(p, vs, j0 + kTile);
    if (here != ~0u || j0 + kTile > min(sight.all, w1)) {
      // Some query does not see all of the tile.
      const unsigned any = Q.visible(j0, sight.end, here);
      X::hide(raw, vs, any >> (4 * g));
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const unsigned see = seen_of(Q, m, j0, any, a, call, par_s) >> (4 * g);
        __builtin_amdgcn_sched_barrier(0);
        // (By masks of bits: comparisons would take two scalar registers for each product.)
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const unsigned in = all_of(see, 16 * (r / 4) + r % 4);
          float& x = p[m][r / 4][r % 4];
          x = __uint_as_float((__float_as_uint(x) & in) | (0xff800000u & ~in));
        }
      }
      // NaN among values that not every query sees would meet weights of zero: they go apart.
      if (__any(X::odd(raw))) {
        if (odd_from < 0) odd_from = j0;
        X::clean(raw);
      }
    }
    soften8<X, MT>(Q, p, a.scale_log2);
    X::template outputs<MT>(Q.o, Q.sum, raw, vs, p);
    if (j0 + kTile < w1) load_v(j0 + kTile);
  }
  if (odd_from >= 0) {
    // Once more over the tiles that some query does not see, for their NaN.
    walk.fetch(odd_from);
#pragma unroll 1
    for (int j0 = odd_from; j0 < w1; j0 += kTile) {
      const unsigned here = place(j0);
      if (here == ~0u && j0 + kTile <= min(sight.all, w1)) continue;
      const unsigned any = Q.visible(j0, sight.end, here);
      unsigned see[MT], none[2] = {0u, 0u};
      load_v(j0);
      X::hide(raw, none, any >> (4 * g));
#pragma unroll
      for (int m = 0; m < MT; ++m) see[m] = seen_of(Q, m, j0, any, a, call, par_s);
      X::template poison<MT>(Q.o, raw, see);
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
    if constexpr (!X::kSums) Q.sum[m][0] = rows_sum(Q.sum[m][0]);

  // The shares of a group join, halves at a time.
  const int mine = wave / GS;
#pragma unroll
  for (int half = kShares / 2; half > 0; half /= 2) {
    __syncthreads();
    if (mine >= half && mine < 2 * half) {
      const int to = wave - half * GS;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        join_s.ml[to][m][lane] = make_float2(Q.mx[m], Q.sum[m][0]);
#pragma unroll
        for (int j = 0; j < X::kOut; ++j) join_s.o[to][m * X::kOut + j][lane] = Q.o[m][j];
      }
    }
    __syncthreads();
    if (mine < half) {
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
  if (mine == 0 && work) Q.store(a, call, x.kvh, x.split);
}

// Query tiles of a wave, and query groups of a workgroup.
struct Shape {
  int mt, gs;
};

Shape shape_of(int tiles, int dtype) {
  const int mt = dtype == WF_F32 ? 1 : tiles <= 1 ? 1 : tiles <= 2 ? 2 : 3;
  const int groups = (tiles + mt - 1) / mt;
  return Shape{mt, groups > 2 ? 4 : groups > 1 ? 2 : 1};
}

template <int DT, int D, int MT>
void launch_groups(const Attend8Args& a, int gs, int64_t blocks, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(blocks)), block(kThreads);
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
  if (gs == 1) go(attend8_kernel<DT, D, MT, 1>);
  if (gs == 2) go(attend8_kernel<DT, D, MT, 2>);
  if (gs == 4) go(attend8_kernel<DT, D, MT, 4>);
}

template <int DT, int D>
void launch_typed(const Attend8Args& a, Shape s, int64_t blocks, hipStream_t stream) {
  if (s.mt == 1) launch_groups<DT, D, 1>(a, s.gs, blocks, stream);
  if constexpr (DT == WF_BF16) {
    if (s.mt == 2) launch_groups<DT, D, 2>(a, s.gs, blocks, stream);
    if (s.mt == 3) launch_groups<DT, D, 3>(a, s.gs, blocks, stream);
  }
}

template <int DT, int D>
void launch_join(const AttendArgs& a, hipStream_t stream) {
  const int64_t n = static_cast<int64_t>(a.rows.B) * a.rows.rmax * a.q_heads;
  hipLaunchKernelGGL((attend_join_kernel<DT, D>), dim3(static_cast<unsigned>((n + kWaves - 1) / kWaves)),
                     dim3(kThreads), 0, stream, a);
}

// How a call is cut: `splits` pieces of `span` positions a sequence, `groups` workgroups a piece and head.
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
  const int each = p.shape.mt * p.shape.gs;
  p.groups = (tiles + each - 1) / each;
  int64_t most = static_cast<int64_t>(max_context) + rows.rmax;
  const int64_t room = static_cast<int64_t>(c.max_pages) * c.page_size;
  most = most < room ? most : room;
  const int64_t one = static_cast<int64_t>(rows.B) * c.heads * p.groups;
  const int64_t slots = 512;
  int64_t best = INT64_MAX, splits = 1;
  for (int64_t rounds = 1; rounds <= 8; ++rounds) {
    int64_t s = rounds * slots / one;
    const int64_t cap = most / kMinSpan < kMaxSplits ? most / kMinSpan : kMaxSplits;
    s = s > cap ? cap : s;
    s = s < 1 ? 1 : s;
    const int64_t need = (one * s + slots - 1) / slots;
    const int64_t cost = need * (most / s + 256 + (s > 1 ? 32 * each : 0));
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
