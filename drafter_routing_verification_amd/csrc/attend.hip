// Attention of a round's rows over the paged cache (whiflash_attend).
//
// Per sequence and key-value head, the M = rows x (q_heads / heads) queries that share
// its keys form tiles of 16, and a wave walks its share of the positions in tiles of
// 16 or 32, keeping each query's running maximum m, sum l and output O in registers:
//   S^T = K Q^T           (MFMA; a lane holds one query's scores of four positions)
//   p = 2^(s - m), l += p (the softmax in base 2, one pass)
//   O^T += V^T P^T        (MFMA)
// The transposed products keep everything in registers.  A lane's scores all belong to
// query lane % 16, so m, l and the rescaling of O are one value a lane, and the scores'
// layout is the second product's operand layout if V's positions take the same order.
// K and V are loaded in rows: K takes its operand layout through LDS, V is transposed by
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

#include "elem.h"
#include "rounds.h"

namespace wf {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2E = 1.44269504088896340736f;
constexpr float kLowest = -3.0e38f;  // a maximum of nothing: finite, so that no inf - inf arises
// O is rescaled only when a maximum grows by more than this (base 2): the weights then
// stay below 2^8, and most tiles need no rescaling.
constexpr float kSlack = 8.f;
constexpr int kMinSpan = 128;
// The plan of pieces: workgroups that run at a time (two a CU; with head_dim 64 three or four
// would fit, which the plan does not use), and the time of a workgroup's start and end, in
// positions.  64 sequences of up to 8,192 positions: one piece
// 256 us, two rounds 270, four 269, sixteen 272.
constexpr int kSlots = 512;
constexpr int kStart = 256;
constexpr int kMaxSplits = 512;
constexpr int kMaxRounds = 8;
constexpr int kJoinAhead = 8;      // pieces whose outputs are fetched at once

struct AttendArgs {
  RowsArgs rows;
  const unsigned char* q;
  int64_t q_bytes;
  int q_heads, group;
  const unsigned char* k;  // the layer
  const unsigned char* v;
  int64_t page_bytes;
  int pages, heads, page_log, seqs, max_pages;
  const int32_t* table;
  const int32_t* context;
  const int32_t* seq;
  int max_context;
  float scale_log2;  // |scale| log2(e)
  unsigned flip;     // the sign bits to flip in q (scale < 0)
  unsigned char* out;
  int splits, span, mgroups;
  float* part_o;     // [splits][rows x q_heads][D]
  float2* part_ml;   // [splits][rows x q_heads]
  int64_t row_heads;
};

// One sequence's part of a launch: its rows, cache sequence and committed length
// (-1: its rows get zeros).
struct SeqCall {
  SeqRows q;
  int s, c;
};

__device__ inline SeqCall seq_call(const AttendArgs& a, int b) {
  SeqCall x;
  x.q = seq_rows(a.rows, b);
  x.s = slot_of(a.seq, b, a.seqs);
  x.c = x.s < 0 ? -1 : a.context[x.s];
  if (x.c > a.max_context ||
      static_cast<int64_t>(x.c) + x.q.n > static_cast<int64_t>(a.max_pages) << a.page_log)
    x.c = -1;
  if (x.c < 0) x.c = -1;
  return x;
}

// Max over the four 16-lane rows of a wave, for each of their 16 places.
__device__ inline float rows_max(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

__device__ inline float rows_sum(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Two float32 values as bfloat16, rounded to nearest even.
__device__ inline unsigned pack_bf16(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const bf16x2 r = __builtin_convertvector((f32x2{lo, hi}), bf16x2);
  return __builtin_bit_cast(unsigned, r);
}

// Infinities and NaN among values that not every query sees go apart from the product, where
// they would meet the weights of zero of those queries too.  What they make of sum p v, in
// four rounds, each the count of the seen positions whose value is of a kind: infinities
// of either sign add theirs, NaN make NaN, and so do infinities whose weight is zero itself.
constexpr int kOddRounds = 4;

// Float32 bits x are of the round's kind if (x & mask) - low <= span.
struct OddKind {
  unsigned mask, low, span;
  float effect;
};

__device__ inline OddKind odd_kind(int round) {
  if (round == 0) return OddKind{0xffffffffu, 0x7f800000u, 0u, INFINITY};
  if (round == 1) return OddKind{0xffffffffu, 0xff800000u, 0u, -INFINITY};
  if (round == 2) return OddKind{0x7fffffffu, 0x7f800001u, 0x7ffffeu, NAN};
  return OddKind{0x7fffffffu, 0x7f800000u, 0u, NAN};
}

// Operand fragment f of group g is the piece of sixteen bytes 4 f + g of a query or key.
// What differs between the types: operand fragments, the two products and their tiles.
// Lane l is place n = l % 16 of group g = l / 16.  kSub positions sub-tiles of 16 make
// a tile; a lane's scores of sub-tile t are positions 16 t + 4 g + i, i < 4.  The
// output tile j, element i is dimension dim(g, i, j) of query n.
template <int DT, int D>
struct Ops;

template <int D>
struct Ops<WF_BF16, D> {
  static constexpr int kSub = 2;
  static constexpr bool kSums = true;    // outputs() adds up the weights too
  static constexpr int kFrags = D / 32;  // 16-byte operand vectors of a query or key
  static constexpr int kOut = D / 16;    // output tiles
  static constexpr int kBytes = 2;
  static constexpr int kVecV = D / 64;   // 8-byte pieces of a lane's share of a row of V
  struct V {
    unsigned w[2 * 4][kVecV * 2];        // [position][dimension pairs]
  };

  __device__ static inline f32x4 scores(const u32x4* k, const u32x4* q) {
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int f = 0; f < kFrags; ++f)
      s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k[f]),
                                                  __builtin_bit_cast(bf16x8, q[f]), s, 0, 0, 0);
    return s;
  }
  // Rows 4 g + i of sub-tile t, dimensions [n D / 16, (n + 1) D / 16).
  template <bool STREAM>
  __device__ static inline void load_v(V& v, int t, const unsigned char* p, unsigned lane_off) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (D == 128) {
        const u32x4 x = STREAM ? load16(reinterpret_cast<const u32x4*>(p + lane_off + i * D * 2))
                               : *reinterpret_cast<const u32x4*>(p + lane_off + i * D * 2);
        v.w[4 * t + i][0] = x.x;
        v.w[4 * t + i][1] = x.y;
        v.w[4 * t + i][2] = x.z;
        v.w[4 * t + i][3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(p + lane_off + i * D * 2);
        v.w[4 * t + i][0] = x.x;
        v.w[4 * t + i][1] = x.y;
      }
    }
  }
  __device__ static inline unsigned v_lane(int n, int g) { return (4 * g * D + n * (D / 16)) * 2; }
  __device__ static inline void zero_v(V& v, int t, int i) {
#pragma unroll
    for (int x = 0; x < kVecV * 2; ++x) v.w[4 * t + i][x] = 0;
  }
  // o += V^T P^T for MT query tiles; p[m][t][i] the weights, rounded to bfloat16 as the matrix
  // units take them (a part in 2^8 each), and summed as rounded, so that equal values come out
  // as they are.  Against 64 bits the outputs are then off by 0.0022-0.0024 (root mean square,
  // relative) where their own rounding alone gives 0.0017.  Weights as two bfloat16 halves give
  // 0.0017, in the same time for one row a sequence (256 us), but 88 us against 77 for the trees
  // and 223 against 188 for the long chains, and an infinity among the values would meet lower
  // halves of zero: not taken.
  template <int MT>
  __device__ static inline void outputs(f32x4 (*o)[kOut], f32x4* sum, const V& v,
                                        const float (*p)[kSub][4]) {
    bf16x8 pb[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const u32x4 x = {pack_bf16(p[m][0][0], p[m][0][1]), pack_bf16(p[m][0][2], p[m][0][3]),
                       pack_bf16(p[m][1][0], p[m][1][1]), pack_bf16(p[m][1][2], p[m][1][3])};
      pb[m] = __builtin_bit_cast(bf16x8, x);
    }
    // The sums of the rounded weights: a product with ones, in place of 8 additions.
    const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u});
#pragma unroll
    for (int m = 0; m < MT; ++m)
      sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, pb[m], sum[m], 0, 0, 0);
#pragma unroll
    for (int j = 0; j < kOut; ++j) {
      // Element j of each position's dimensions, two positions a word.
      u32x4 a;
      unsigned w[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
        w[x] = __builtin_amdgcn_perm(v.w[2 * x + 1][j >> 1], v.w[2 * x][j >> 1],
                                     (j & 1) ? 0x07060302u : 0x05040100u);
      a = u32x4{w[0], w[1], w[2], w[3]};
#pragma unroll
      for (int m = 0; m < MT; ++m)
        o[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), pb[m],
                                                          o[m][j], 0, 0, 0);
    }
  }
  __device__ static inline u32x4 flip_sign(u32x4 x, unsigned bits) { return x ^ bits; }

  // Whether the lane's values hold infinities or NaN.
  __device__ static inline bool odd(const V& v) {
    bool x = false;
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int c = 0; c < kVecV * 2; ++c)
        x = x || (v.w[r][c] & 0x7f80u) == 0x7f80u || (v.w[r][c] & 0x7f800000u) == 0x7f800000u;
    return x;
  }
  // Adds to the outputs what infinities and NaN among the values make of them (odd_kind), and
  // puts zeros in their place.  see[m]: the positions that the lane's query of tile m sees,
  // a bit each.
  template <int MT>
  __device__ static inline void poison(f32x4 (*o)[kOut], V& v, const float (*p)[kSub][4],
                                       const unsigned* see) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll 1
    for (int round = 0; round < kOddRounds; ++round) {
      const OddKind kind = odd_kind(round);
      bf16x8 pb[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        unsigned w[4] = {0u, 0u, 0u, 0u}, bits = see[m] >> (4 * g);
        asm volatile("" : "+v"(bits));  // (worked out in each round: it would take registers)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool seen = bits >> (16 * t + i) & 1u;
            const bool on = seen && (round < kOddRounds - 1 || !(p[m][t][i] > 0.f));
            w[2 * t + i / 2] |= on ? 0x3f80u << (i % 2 * 16) : 0u;
          }
        pb[m] = __builtin_bit_cast(bf16x8, (u32x4{w[0], w[1], w[2], w[3]}));
      }
#pragma unroll
      for (int j = 0; j < kOut; ++j) {
        unsigned w[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          // (A half is compared where it lies: in the lower one everything is shifted.)
          const int down = (j & 1) ? 0 : 16;
          const unsigned mask = (kind.mask & 0xffff0000u) >> down;
          const unsigned low = ((kind.low + 0xffffu) & 0xffff0000u) >> down, span = kind.span >> down;
          w[x] = (v.w[2 * x][j >> 1] & mask) - low <= span ? 0x3f80u : 0u;
          w[x] |= (v.w[2 * x + 1][j >> 1] & mask) - low <= span ? 0x3f800000u : 0u;
        }
        const bf16x8 a = __builtin_bit_cast(bf16x8, (u32x4{w[0], w[1], w[2], w[3]}));
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          f32x4 n = {0.f, 0.f, 0.f, 0.f};
          n = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, pb[m], n, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[m][j][i] += n[i] > 0.f ? kind.effect : 0.f;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int c = 0; c < kVecV * 2; ++c) {
        const unsigned x = v.w[r][c];
        v.w[r][c] = ((x & 0x7f80u) == 0x7f80u ? 0u : x & 0xffffu) |
                    ((x & 0x7f800000u) == 0x7f800000u ? 0u : x & 0xffff0000u);
      }
  }
};

template <int D>
struct Ops<WF_F32, D> {
  static constexpr int kSub = 1;
  static constexpr bool kSums = false;
  static constexpr int kFrags = D / 16;
  static constexpr int kOut = D / 16;
  static constexpr int kBytes = 4;
  struct V {
    f32x4 w[4][D / 64];
  };
  __device__ static inline f32x4 scores(const u32x4* k, const u32x4* q) {
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int f = 0; f < kFrags; ++f) {
      const f32x4 kf = __builtin_bit_cast(f32x4, k[f]), qf = __builtin_bit_cast(f32x4, q[f]);
#pragma unroll
      for (int e = 0; e < 4; ++e) s = __builtin_amdgcn_mfma_f32_16x16x4f32(kf[e], qf[e], s, 0, 0, 0);
    }
    return s;
  }
  // Rows 4 g + i, dimensions 64 h + 4 n + [0, 4).
  template <bool STREAM>
  __device__ static inline void load_v(V& v, int, const unsigned char* p, unsigned lane_off) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
        v.w[i][h] = __builtin_bit_cast(
            f32x4, STREAM ? load16(reinterpret_cast<const u32x4*>(p + lane_off + i * D * 4 + h * 256))
                          : *reinterpret_cast<const u32x4*>(p + lane_off + i * D * 4 + h * 256));
  }
  __device__ static inline unsigned v_lane(int n, int g) { return (4 * g * D + n * 4) * 4; }
  __device__ static inline void zero_v(V& v, int, int i) {
#pragma unroll
    for (int h = 0; h < D / 64; ++h) v.w[i][h] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  template <int MT>
  __device__ static inline void outputs(f32x4 (*o)[kOut], f32x4*, const V& v,
                                        const float (*p)[kSub][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int m = 0; m < MT; ++m)
            o[m][4 * h + e] = __builtin_amdgcn_mfma_f32_16x16x4f32(v.w[i][h][e], p[m][0][i],
                                                                   o[m][4 * h + e], 0, 0, 0);
  }
  __device__ static inline u32x4 flip_sign(u32x4 x, unsigned bits) { return x ^ bits; }

  __device__ static inline bool is_odd(float x) {
    return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u;
  }
  __device__ static inline bool odd(const V& v) {
    bool x = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) x = x || is_odd(v.w[i][h][e]);
    return x;
  }
  template <int MT>
  __device__ static inline void poison(f32x4 (*o)[kOut], V& v, const float (*p)[kSub][4],
                                       const unsigned* see) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll 1
    for (int round = 0; round < kOddRounds; ++round) {
      const OddKind kind = odd_kind(round);
      unsigned bits[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        bits[m] = see[m] >> (4 * g);
        asm volatile("" : "+v"(bits[m]));
      }
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            f32x4 n = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool seen = bits[m] >> i & 1u;
              const bool on = seen && (round < kOddRounds - 1 || !(p[m][0][i] > 0.f));
              const bool is = (__float_as_uint(v.w[i][h][e]) & kind.mask) - kind.low <= kind.span;
              n = __builtin_amdgcn_mfma_f32_16x16x4f32(is ? 1.f : 0.f, on ? 1.f : 0.f, n, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) o[m][4 * h + e][i] += n[i] > 0.f ? kind.effect : 0.f;
          }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) v.w[i][h][e] = is_odd(v.w[i][h][e]) ? 0.f : v.w[i][h][e];
  }
};

// Writes a lane's outputs of one query tile (element i of every output tile) scaled by
// `f`: to out in the call's type, or float32.
template <int DT, int D>
__device__ inline void store_query(unsigned char* out, const f32x4* o, int g, float f) {
  constexpr int kOut = Ops<DT, D>::kOut;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == WF_BF16) {
      unsigned w[kOut / 2];
#pragma unroll
      for (int j = 0; j < kOut / 2; ++j) w[j] = pack_bf16(o[2 * j][i] * f, o[2 * j + 1][i] * f);
      unsigned char* p = out + (4 * g + i) * kOut * 2;
      if constexpr (kOut == 8) {
        *reinterpret_cast<u32x4*>(p) = u32x4{w[0], w[1], w[2], w[3]};
      } else {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
      }
    } else {
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
        *reinterpret_cast<f32x4*>(out + (64 * h + (4 * g + i) * 4) * 4) =
            f32x4{o[4 * h][i] * f, o[4 * h + 1][i] * f, o[4 * h + 2][i] * f, o[4 * h + 3][i] * f};
    }
  }
}

// ... the partial output, float32 in the order of the dimensions.
template <int DT, int D>
__device__ inline void store_partial(float* out, const f32x4* o, int g) {
  constexpr int kOut = Ops<DT, D>::kOut;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == WF_BF16) {
#pragma unroll
      for (int j = 0; j < kOut; j += 4)
        *reinterpret_cast<f32x4*>(out + (4 * g + i) * kOut + j) =
            f32x4{o[j][i], o[j + 1][i], o[j + 2][i], o[j + 3][i]};
    } else {
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
        *reinterpret_cast<f32x4*>(out + 64 * h + (4 * g + i) * 4) =
            f32x4{o[4 * h][i], o[4 * h + 1][i], o[4 * h + 2][i], o[4 * h + 3][i]};
    }
  }
}

// Orders a wave's LDS accesses: what a lane wrote before, every lane reads after.
__device__ inline void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// What a wave keeps of MT tiles of 16 queries: the queries in operand layout, and for
// query place n of each tile m, l and O.
template <int DT, int D, int MT>
struct Queries {
  using X = Ops<DT, D>;
  u32x4 q[MT][X::kFrags];
  f32x4 o[MT][X::kOut];
  float mx[MT];
  f32x4 sum[MT];  // element 0: l, where kSums; else this lane's part of it
  int first;       // the first query

  // The lane's query of tile m, or -1 past the last one.
  __device__ inline int query(const AttendArgs& a, const SeqCall& call, int m) const {
    const int x = first + 16 * m + static_cast<int>(threadIdx.x & 15);
    return x < call.q.n * a.group ? x : -1;
  }

  __device__ inline void load(const AttendArgs& a, const SeqCall& call, int kvh, int from) {
    const int g = (threadIdx.x & 63) >> 4;
    first = from;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int x = query(a, call, m);
      const int h = kvh * a.group + max(x, 0) % a.group;
      const int64_t r = static_cast<int64_t>(call.q.row0) + max(x, 0) / a.group;
      const unsigned char* p = a.q + r * a.q_bytes + h * D * X::kBytes;
#pragma unroll
      for (int f = 0; f < X::kFrags; ++f) {
        q[m][f] = u32x4{0u, 0u, 0u, 0u};
        if (x >= 0)
          q[m][f] = X::flip_sign(*reinterpret_cast<const u32x4*>(p + (4 * f + g) * 16), a.flip);
      }
      mx[m] = kLowest;
      sum[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < X::kOut; ++j) o[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }

  using Weights = float[MT][X::kSub][4];

  // The products q . k of sub-tile t.
  __device__ inline void score(Weights& p, int t, const u32x4* k) const {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const f32x4 s = X::scores(k, q[m]);
#pragma unroll
      for (int i = 0; i < 4; ++i) p[m][t][i] = s[i];
    }
  }

  // Of the 32 positions from j0 on, those that can be seen at all: before `end` and with
  // a page (`pages`: a bit each).
  __device__ static inline unsigned visible(int j0, int end, unsigned pages) {
    const int have = min(max(end - j0, 0), 32);
    return pages & (have >= 32 ? ~0u : (1u << have) - 1u);
  }

  // Takes positions that no query sees out of a tile's scores and values: whatever lies
  // there must not meet a weight of zero, it may be NaN.
  __device__ static inline void hide(Weights& p, typename X::V& v, unsigned any) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int t = 0; t < X::kSub; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!(any >> (16 * t + 4 * g + i) & 1u)) {
          X::zero_v(v, t, i);
#pragma unroll
          for (int m = 0; m < MT; ++m) p[m][t][i] = -INFINITY;
        }
  }

  // Takes out of a tile's scores what its query does not see: positions outside `any`,
  // and of the round's own positions those of rows that are not on its path.  see[m] gets the
  // positions that the lane's query of tile m sees.
  __device__ inline void mask(Weights& p, unsigned* see, int j0, unsigned any, const AttendArgs& a,
                              const SeqCall& call, const int16_t* par) const {
    const int g = (threadIdx.x & 63) >> 4;
    const int old = min(max(call.c - j0, 0), 32);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      see[m] = old >= 32 ? ~0u : (1u << old) - 1u;
      const int x0 = query(a, call, m);
      const int own = x0 < 0 ? -1 : x0 / a.group, last = call.c + own - j0;
      if (!call.q.tree) {
        if (own >= 0 && last >= 0) see[m] = last >= 31 ? ~0u : (2u << last) - 1u;
      } else {
        for (int u = own; u >= 0 && call.c + u >= j0; u = u == 0 ? -1 : par[u]) {
          const int x = call.c + u - j0;
          if (x < 32) see[m] |= 1u << x;
        }
      }
      see[m] &= any;
#pragma unroll
      for (int t = 0; t < X::kSub; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!(see[m] >> (16 * t + 4 * g + i) & 1u)) p[m][t][i] = -INFINITY;
    }
  }

  // Products to weights 2^(scale q . k - m), with the running maxima (of the scaled
  // products; scale > 0, its sign is in q) and, where the output product does not give
  // them, the sums.
  __device__ inline void soften(Weights& p, float scale) {
    bool grown = false;
    float top[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float x = p[m][0][0];
#pragma unroll
      for (int t = 0; t < X::kSub; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) x = fmaxf(x, p[m][t][i]);
      top[m] = rows_max(x) * scale;
      grown = grown || top[m] > mx[m] + kSlack;
    }
    if (__any(grown)) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float now = fmaxf(mx[m], top[m]);
        const float f = __builtin_amdgcn_exp2f(mx[m] - now);
        mx[m] = now;
        sum[m] *= f;
#pragma unroll
        for (int j = 0; j < X::kOut; ++j) o[m][j] *= f;
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int t = 0; t < X::kSub; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[m][t][i] = __builtin_amdgcn_exp2f(fmaf(p[m][t][i], scale, -mx[m]));
          if constexpr (!X::kSums) sum[m][0] += p[m][t][i];
        }
    }
  }

  // The result of a piece: the output if it is the only one, else its part.
  __device__ inline void store(const AttendArgs& a, const SeqCall& call, int kvh, int split) const {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int x = query(a, call, m);
      if (x < 0) continue;
      const int64_t to = (static_cast<int64_t>(call.q.row0) + x / a.group) * a.q_heads +
                         kvh * a.group + x % a.group;
      if (a.splits == 1) {
        store_query<DT, D>(a.out + to * D * X::kBytes, o[m], g, sum[m][0] > 0.f ? 1.f / sum[m][0] : 0.f);
      } else {
        const int64_t at = split * a.row_heads + to;
        store_partial<DT, D>(a.part_o + at * D, o[m], g);
        if (g == 0) a.part_ml[at] = make_float2(mx[m], sum[m][0]);
      }
    }
  }
};

// The pages of one sequence as a wave walks it: the ids of 64 sub-tiles at a time, one a
// lane (-1: none).
struct PageWalk {
  const int32_t* table;
  int log, pages, stop, base, ids;

  __device__ inline void fetch(int from) {
    const int j = from + 16 * static_cast<int>(threadIdx.x & 63);
    base = from;
    ids = j < stop ? table[j >> log] : -1;
    if (ids >= pages) ids = -1;
  }
  __device__ inline PageWalk(const AttendArgs& a, const SeqCall& call, int from, int to)
      : table(a.table + static_cast<int64_t>(max(call.s, 0)) * a.max_pages), log(a.page_log),
        pages(a.pages), stop(to), base(from), ids(-1) {
    if (from < to) fetch(from);
  }
  // The tile from j0 on (j0 grows by no more than 1,024 between calls).
  __device__ inline void reach(int j0, int tile) {
    if (j0 + tile - base > 64 * 16) fetch(j0);
  }
  // The page of sub-tile j, uniform, or -1.
  __device__ inline int at(int j) const {
    return __builtin_amdgcn_readlane(ids, ((j - base) >> 4) & 63);
  }
};

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

// What `count` queries from `first` on see of a sequence: positions before `all` are seen by
// every one of them, positions from `end` on by none.
struct Sight {
  int all, end;
};

__device__ inline Sight sight_of(const AttendArgs& a, const SeqCall& call, int first, int count) {
  if (call.c < 0) return Sight{-1, 0};
  if (call.q.tree) return Sight{call.c, call.c + call.q.n};
  const int last = min(call.q.n * a.group, first + count) - 1;
  return Sight{call.c + first / a.group + 1, call.c + last / a.group + 1};
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
  Queries<DT, D, MT> Q;
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
  using Weights = typename Queries<DT, D, MT>::Weights;
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
  Queries<DT, D, MT> Q;
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
  using Weights = typename Queries<DT, D, MT>::Weights;
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

// Joins the pieces of every row and head: one wave each, in the pieces' order.
template <int DT, int D>
__global__ __launch_bounds__(kThreads) void attend_join_kernel(AttendArgs a) {
  constexpr int kPer = D / 64;
  const int lane = threadIdx.x & 63;
  const int64_t x = static_cast<int64_t>(blockIdx.x) * kWaves + (threadIdx.x >> 6);
  const int h = static_cast<int>(x % a.q_heads);
  const int64_t bi = x / a.q_heads;
  const int b = static_cast<int>(bi / a.rows.rmax), i = static_cast<int>(bi % a.rows.rmax);
  if (b >= a.rows.B) return;
  const SeqCall call = seq_call(a, b);
  if (i >= call.q.n) return;
  const int64_t r = (static_cast<int64_t>(call.q.row0) + i) * a.q_heads + h;
  // A chain's row is not in the pieces past its own position.
  const int end = call.c < 0 ? 0 : call.c + (call.q.tree ? call.q.n : i + 1);
  const int used = end > 0 ? (end + a.span - 1) / a.span : 0;
  // Lane s holds piece s's maximum and sum, 64 pieces at a time, so that the loads of
  // the outputs depend on nothing.
  float m = kLowest, l = 0.f, o[kPer] = {};
  for (int s0 = 0; s0 < used; s0 += 64) {
    const int many = min(used - s0, 64);
    float2 y = make_float2(kLowest, 0.f);
    if (lane < many) y = a.part_ml[(s0 + lane) * a.row_heads + r];
    float top = y.x;
    for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    const float now = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - now);
    const float w = __builtin_amdgcn_exp2f(y.x - now);
    float sum = y.y * w;
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
    m = now;
    l = l * f + sum;
#pragma unroll
    for (int t = 0; t < kPer; ++t) o[t] *= f;
    for (int s = 0; s < many; s += kJoinAhead) {
      float p[kJoinAhead][kPer];
#pragma unroll
      for (int e = 0; e < kJoinAhead; ++e) {
        const float* from = a.part_o + ((s0 + min(s + e, many - 1)) * a.row_heads + r) * D + lane * kPer;
#pragma unroll
        for (int t = 0; t < kPer; ++t) p[e][t] = from[t];
      }
#pragma unroll
      for (int e = 0; e < kJoinAhead; ++e) {
        const float ws = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), (s + e) & 63));
#pragma unroll
        for (int t = 0; t < kPer; ++t) o[t] += s + e < many ? p[e][t] * ws : 0.f;
      }
    }
  }
  const float f = l > 0.f ? 1.f / l : 0.f;
  if constexpr (DT == WF_F32) {
#pragma unroll
    for (int t = 0; t < kPer; ++t)
      reinterpret_cast<float*>(a.out)[r * D + lane * kPer + t] = o[t] * f;
  } else if constexpr (kPer == 2) {
    reinterpret_cast<unsigned*>(a.out)[r * (D / 2) + lane] = pack_bf16(o[0] * f, o[1] * f);
  } else {
    reinterpret_cast<uint16_t*>(a.out)[r * D + lane] = static_cast<uint16_t>(pack_bf16(o[0] * f, 0.f));
  }
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
