// The rules of decoding applied to the logits of a round's rows: written out
// (whiflash_process_logits), or folded into the greedy argmax
// (whiflash_verify_constrained), whose chunk partials the acceptance then merges.
#include <math.h>

#include "accept.h"
#include "elem.h"
#include "rounds.h"
#include "rules_math.h"

namespace wf {
namespace {

constexpr int kVecsPer = 4;                       // 16-byte vectors of a row per thread
constexpr int kChunkVecs = kVecsPer * kThreads;   // vectors of a row per workgroup
constexpr int kBiasLds = 256;                     // biases of a chunk that are kept in LDS
constexpr int kMaxGroup = 64;                     // rows per workgroup
constexpr int kListMax = 256;                     // special elements of a wave that are listed
constexpr int kArgmax = -1;
// Workgroups of a large launch.  More make shorter groups (every group reads its history
// words and works out its special elements anew), fewer leave an uneven end.  128 sequences
// (half chains of 17 rows, half trees of 61) x 151,936 bf16, and 64 chains x 17 written out, three
// passes of each in turn: 8,192 369-383 / 146 us, 12,288 343-355 / 148, 16,384 343-358 / 148;
// 4,096 and 24,576, in another session, 397 / 158 and 377 / 174.
constexpr int64_t kRulesBlocks = 12288;

struct RulesArgs {
  RowsArgs rows;
  wf_logit_rules rules;
  const unsigned char* logits;
  int64_t row_bytes;
  int V, nvec, chunks, groups, group;
  Partial* part;       // argmax: [B * rmax][chunks]
  unsigned char* out;  // written form
  int64_t out_bytes;
};

// A round's drafted tokens that lie in one chunk, and the paths of its rows.
struct PathLds {
  int tok[kMaxSeqRows];                // target token of node u, -1 for none
  int16_t par[kMaxSeqRows];            // parent of node u, -1 where its path ends
  unsigned long long rows[64];         // rows that have node u on their path (up to 64 rows)
  int16_t node[kMaxSeqRows];           // nodes whose token lies in the chunk, any order
  int count;
  unsigned node_bits[kChunkVecs / 4];  // one byte a vector: elements that some node drafted
  unsigned bias_bits[kChunkVecs / 4];  // ... and that have a bias
  int bias_id[kBiasLds];
  float bias_value[kBiasLds];
};

// Element k of a vector of history words (8 or 4 of them).
template <int DT>
__device__ inline unsigned word_at(const u32x4& h, int k) {
  const unsigned w = k < 2 ? h.x : k < 4 ? h.y : k < 6 ? h.z : h.w;
  return (w >> ((k & 1) * 16)) & 0xffffu;
}

// Orders a wave's LDS accesses: what a lane wrote before, every lane reads after.
__device__ inline void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <typename T>
__device__ inline T read_lane(T x, int lane) {
  return static_cast<T>(__builtin_amdgcn_readlane(static_cast<int>(x), lane));
}

// Equal for equal float32 values (-0 and +0 too).
__device__ inline unsigned float_key(unsigned bits) { return bits == 0x80000000u ? 0u : bits; }

// x if bit k of f is set, else -inf.
__device__ inline float masked(float x, unsigned f, int k) {
  const unsigned m = static_cast<unsigned>(static_cast<int>(f << (31 - k)) >> 31);
  return __uint_as_float((__float_as_uint(x) & m) | (~m & 0xff800000u));
}

// How often token t is among the path tokens of row i.
__device__ inline int times_on_path(const PathLds& L, bool tree, int n, int i, int t) {
  int c = 0;
  if (tree && n > 64) {
    for (int u = i; u > 0; u = L.par[u]) c += L.tok[u] == t;
    return c;
  }
  for (int j = 0; j < L.count; ++j) {
    const int u = L.node[j];
    const bool on = n <= 64 ? (L.rows[u] >> i) & 1ull : u <= i;
    c += on && L.tok[u] == t;
  }
  return c;
}

// Maximum over the 64 lanes of a wave, in every lane.
__device__ inline float wave_max_f32(float x) {
  x = fmaxf(x, dpp_mov<kDppQuadXor1>(x));
  x = fmaxf(x, dpp_mov<kDppQuadXor2>(x));
  x = fmaxf(x, dpp_mov<kDppHalfMirror>(x));
  x = fmaxf(x, dpp_mov<kDppMirror>(x));
  x = fmaxf(x, dpp_mov<kDppBcast15, 0xa>(x));
  x = fmaxf(x, dpp_mov<kDppBcast31, 0xc>(x));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}

// The first n of a vector's PER values, at vector v of an output row.
template <int OUT, int PER>
__device__ inline void store_vec(unsigned char* row, int v, const float* x, int n) {
  if constexpr (OUT == WF_F32) {
    float* p = reinterpret_cast<float*>(row) + static_cast<int64_t>(v) * PER;
    if (n == PER) {
#pragma unroll
      for (int k = 0; k < PER; k += 4)
        *reinterpret_cast<float4*>(p + k) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
    } else {
#pragma unroll
      for (int k = 0; k < PER; ++k)
        if (k < n) p[k] = x[k];
    }
  } else {
    uint16_t* p = reinterpret_cast<uint16_t*>(row) + static_cast<int64_t>(v) * PER;
    if (n == PER) {
      unsigned w[PER / 2];
#pragma unroll
      for (int k = 0; k < PER / 2; ++k) w[k] = bf16_bits(x[2 * k]) | bf16_bits(x[2 * k + 1]) << 16;
      if constexpr (PER == 8) {
        *reinterpret_cast<u32x4*>(p) = u32x4{w[0], w[1], w[2], w[3]};
      } else {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < PER; ++k)
        if (k < n) p[k] = static_cast<uint16_t>(bf16_bits(x[k]));
    }
  }
}

// One workgroup per (sequence, group of rows, chunk of the vocabulary), the group's rows
// one after the other: a chunk's history words stay in registers for all of them.
//
// Streaming of the logits.  Nearly all tokens have neither history nor bias and were not
// drafted in this round, so every element has one "special" bit, worked out once a
// workgroup: elements without it take the plain path (a masked maximum, or a copy).  The
// argmax lists a wave's special elements, so that its lanes share them evenly: the row's
// vectors pass through LDS, and each lane, which decoded its element once for all rows,
// picks its logit.  Written out, each lane handles the special elements of its vectors in a
// loop of its own.  The path's tokens differ from row to row; only elements that some node
// drafted look them up.  The maximum is reduced over the wave, and its first place found by
// ballots and in scalar registers.
//
// The next row's mask and vectors are fetched before this row is worked on, the mask first:
// loads return in order, and the mask is needed first.
//
// Measured (MI355X, 151,936 entries): 64 chains x 17 rows written out in bf16 148 us, 4.7 TB/s
// read and written together, the rate of a large copy; in float32 269 us.  The whole
// verification of 128 sequences (4,992 rows, 1.65 GB of bf16) 324-344 us, 5 TB/s: bound by its
// instructions, some 310 vector and 220 scalar ones a wave and row, and by having only 4 waves
// a SIMD to cover their latencies (105 registers, and 35,344 bytes of LDS a workgroup, of which
// a CU holds four); without any rule it takes 243 us, against 209 us of the plain call.
// Registers cut for five waves, which spills (and LDS still holds four): 430 us; bit masks
// that keep the special elements out of an unmasked maximum (137 registers, 3 waves) 416 us.
template <int DT, int OUT>
__global__ __launch_bounds__(kThreads) void rules_kernel(RulesArgs a) {
  using E = Elem<DT>;
  constexpr int kPer = E::kPerVec;
  constexpr unsigned kAll = (1u << kPer) - 1u;
  __shared__ PathLds L;
  __shared__ Partial best_s[OUT == kArgmax ? kMaxGroup : 1][kWaves];
  __shared__ u32x4 stage_s[kWaves][OUT == kArgmax ? kVecsPer * 64 : 1];
  __shared__ unsigned list_s[kWaves][OUT == kArgmax ? kListMax : 1];
  const int tid = threadIdx.x;
  const int c = blockIdx.x % a.chunks;
  const int bg = blockIdx.x / a.chunks;
  const int b = bg / a.groups, g = bg - b * a.groups;
  const SeqRows q = seq_rows(a.rows, b);
  // Of a sequence shorter than the longest, as few groups as hold it, evenly.
  const int used = (q.n + a.group - 1) / a.group;
  if (g >= used) return;
  const int i0 = g * q.n / used, i1 = (g + 1) * q.n / used;
  const wf_logit_rules& R = a.rules;
  const int v0 = c * kChunkVecs + tid;  // the thread's vectors: v0 + u * kThreads
  const int tail = a.V - a.nvec * kPer;

  const unsigned char* rowp = a.logits + (static_cast<int64_t>(q.row0) + i0) * a.row_bytes;
  // Lanes past the row's whole vectors read its last one and mask it.
  const bool has_tail = tail && a.nvec / kChunkVecs == c;
  unsigned off[kVecsPer];
#pragma unroll
  for (int u = 0; u < kVecsPer; ++u) off[u] = 16u * max(min(v0 + u * kThreads, a.nvec - 1), 0);
  auto load_row = [&](const unsigned char* p, u32x4* d) {
    if (a.nvec > 0) {
#pragma unroll
      for (int u = 0; u < kVecsPer; ++u) d[u] = load16(reinterpret_cast<const u32x4*>(p + off[u]));
    }
    if (has_tail) {
#pragma unroll
      for (int u = 0; u < kVecsPer; ++u) {
        if (v0 + u * kThreads != a.nvec) continue;
        // The entries past the last whole vector, one by one.
        unsigned w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          if (k < tail) {
            if constexpr (DT == WF_BF16) {
              const unsigned x = reinterpret_cast<const uint16_t*>(p)[a.nvec * kPer + k];
              w[k >> 1] |= x << ((k & 1) * 16);
            } else {
              w[k] = reinterpret_cast<const unsigned*>(p)[a.nvec * kPer + k];
            }
          }
        }
        d[u] = u32x4{w[0], w[1], w[2], w[3]};
      }
    }
  };
  // The byte of a row's mask that holds each vector's bits (a row has ceil(V / 8) at least).
  auto load_mask = [&](int64_t r, unsigned* m) {
    if (!R.allow) return;
    const unsigned char* p = reinterpret_cast<const unsigned char*>(R.allow + r * R.allow_stride);
#pragma unroll
    for (int u = 0; u < kVecsPer; ++u) {
      const int v = min(v0 + u * kThreads, (a.V - 1) / kPer);
      m[u] = p[kPer == 8 ? v : v >> 1];
    }
  };
  u32x4 d[kVecsPer] = {};
  unsigned mask[kVecsPer] = {};
  load_mask(static_cast<int64_t>(q.row0) + i0, mask);
  load_row(rowp, d);

  // What the chunk's elements need beyond a mask.
  Penalties pen{1.f, 0.f, 0.f};
  const bool penal = R.penalties != nullptr;
  if (penal) pen = Penalties{R.penalties[3 * b], R.penalties[3 * b + 1], R.penalties[3 * b + 2]};
  const int slot = penal && R.history ? slot_of(R.slot, b, R.slots) : -1;
  u32x4 hw[kVecsPer] = {};
  unsigned valid = 0, special = 0;
  const uint16_t* hist = slot >= 0 ? R.history + slot * R.history_stride : nullptr;
#pragma unroll
  for (int u = 0; u < kVecsPer; ++u) {
    const int v = v0 + u * kThreads;
    const unsigned have = v < a.nvec ? kAll : v == a.nvec ? (1u << tail) - 1u : 0u;
    valid |= have << (8 * u);
    if (hist && have) {
      if (have == kAll) {
        if constexpr (DT == WF_BF16) {
          hw[u] = reinterpret_cast<const u32x4*>(hist)[v];
        } else {
          const uint2 h = reinterpret_cast<const uint2*>(hist)[v];
          hw[u].x = h.x;
          hw[u].y = h.y;
        }
      } else {
        unsigned w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          if (k < tail) w[k >> 1] |= static_cast<unsigned>(hist[v * kPer + k]) << ((k & 1) * 16);
        hw[u] = u32x4{w[0], w[1], w[2], w[3]};
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kVecsPer; ++u) {
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      special |= word_at<DT>(hw[u], k) ? 1u << (8 * u + k) : 0u;
  }
  int blo = 0, bhi = 0;
  if (R.bias_offsets) {
    blo = min(max(R.bias_offsets[b], 0), R.bias_count);
    bhi = min(max(R.bias_offsets[b + 1], blo), R.bias_count);
    const int t0 = c * kChunkVecs * kPer;
    blo = lower_bound(R.bias_ids, blo, bhi, t0);
    bhi = lower_bound(R.bias_ids, blo, bhi, min(t0 + kChunkVecs * kPer, a.V));
  }
  const bool paths = penal && q.n > 1;
  unsigned node_bits = 0, bias_bits = 0;
  if (paths || blo < bhi) {
    if (tid == 0) L.count = 0;
    L.node_bits[tid] = 0;
    L.bias_bits[tid] = 0;
    __syncthreads();
    if (paths) {
      for (int u = 1 + tid; u < q.n; u += kThreads) {
        const int t = node_token(a.rows, b, q.tree, u, a.V);
        L.tok[u] = t;
        if (q.tree) L.par[u] = static_cast<int16_t>(node_parent(a.rows, b, true, u));
        const int v = t / kPer - c * kChunkVecs;
        if (t >= 0 && v >= 0 && v < kChunkVecs) {
          L.node[atomicAdd(&L.count, 1)] = static_cast<int16_t>(u);
          atomicOr(&L.node_bits[v >> 2], 1u << ((v & 3) * 8 + t % kPer));
        }
      }
    }
    for (int k = blo + tid; k < bhi; k += kThreads) {
      const int t = R.bias_ids[k];
      const int v = t / kPer - c * kChunkVecs;
      // (ids out of order may lie outside the chunk)
      if (t >= 0 && v >= 0 && v < kChunkVecs)
        atomicOr(&L.bias_bits[v >> 2], 1u << ((v & 3) * 8 + t % kPer));
      if (k - blo < kBiasLds) {
        L.bias_id[k - blo] = t;
        L.bias_value[k - blo] = R.bias_values[k];
      }
    }
    __syncthreads();
    if (paths && q.n <= 64 && L.count > 0) {
      if (tid < q.n) L.rows[tid] = q.tree ? 0ull : ~0ull << tid;
      __syncthreads();
      if (q.tree && tid < q.n)
        for (int u = tid; u > 0; u = L.par[u]) atomicOr(&L.rows[u], 1ull << tid);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kVecsPer; ++u) {
      const int v = u * kThreads + tid;
      node_bits |= ((L.node_bits[v >> 2] >> ((v & 3) * 8)) & 0xffu) << (8 * u);
      bias_bits |= ((L.bias_bits[v >> 2] >> ((v & 3) * 8)) & 0xffu) << (8 * u);
    }
    special |= node_bits | bias_bits;
  }
  const int nb = bhi - blo;
  auto bias_of = [&](int t) {
    if (nb <= kBiasLds) {
      int lo = 0, hi = nb;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (L.bias_id[mid] < t) {
          lo = mid + 1;
        } else {
          hi = mid;
        }
      }
      return lo < nb && L.bias_id[lo] == t ? L.bias_value[lo] : 0.f;
    }
    const int j = lower_bound(R.bias_ids, blo, bhi, t);
    return j < bhi && R.bias_ids[j] == t ? R.bias_values[j] : 0.f;
  };
  // The processed value of a special element: logit x of token t with history word
  // `word`, in row i.
  auto value = [&](float x, unsigned word, bool node, bool biased, int t, int i) {
    if (penal) {
      const int extra = node ? times_on_path(L, q.tree, q.n, i, t) : 0;
      x = apply_penalties(x, word, extra, pen);
    }
    if (biased) x += bias_of(t);
    return x;
  };
  // The same for element k of the lane's own vector u.
  auto own_value = [&](const u32x4& dv, const u32x4& h, int u, int k, int i) {
    const unsigned bit = 1u << (8 * u + k);
    return value(E::at(dv, k), word_at<DT>(h, k), node_bits & bit, bias_bits & bit,
                 (v0 + u * kThreads) * kPer + k, i);
  };
  // Up to kListMax special elements of a wave are listed, so that its lanes share them
  // evenly: bits 0-15 the history word, 16-26 the place in the wave's vectors, 27 and 28
  // whether some node drafted it and whether it has a bias.
  const int lane = tid & 63, wave = tid >> 6;
  int listed = 0;
  if constexpr (OUT == kArgmax) {
    int before = __popc(special);
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(before, off);
      before += lane >= off ? o : 0;
    }
    listed = __shfl(before, 63);
    if (listed <= kListMax) {
      unsigned* p = list_s[wave] + before - __popc(special);
#pragma unroll
      for (int u = 0; u < kVecsPer; ++u) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const unsigned bit = 1u << (8 * u + k);
          if (special & bit)
            *p++ = word_at<DT>(hw[u], k) | ((u * 64 + lane) * kPer + k) << 16 |
                   ((node_bits & bit) ? 1u << 27 : 0u) | ((bias_bits & bit) ? 1u << 28 : 0u);
        }
      }
    }
  }

  // The lane's first listed element, decoded once for all rows: its place and token, its
  // bias, and the rows that have its node on their path (one node drafted it, of up to
  // 64 rows; else `ask` has them looked up in each row).
  int first_at = 0, first_t = 0;
  unsigned first_word = 0;
  float first_bias = 0.f;
  unsigned long long first_rows = 0;
  bool first = false, first_biased = false, ask = false;
  if constexpr (OUT == kArgmax) {
    wave_sync();
    first = listed <= kListMax && lane < listed;
    if (first) {
      const unsigned e = list_s[wave][lane];
      first_at = (e >> 16) & 0x7ffu;
      first_word = e & 0xffffu;
      first_t = (c * kChunkVecs + first_at / (64 * kPer) * kThreads + wave * 64) * kPer +
                first_at % (64 * kPer);
      first_biased = e >> 28 & 1u;
      if (first_biased) first_bias = bias_of(first_t);
      if (e >> 27 & 1u) {
        int times = 0;
        for (int j = 0; j < L.count; ++j) {
          const int u = L.node[j];
          if (L.tok[u] != first_t) continue;
          ++times;
          if (q.n <= 64) first_rows = L.rows[u];
        }
        ask = times > 1 || q.n > 64;
      }
    }
  }

  for (int i = i0; i < i1; ++i) {
    const int64_t r = static_cast<int64_t>(q.row0) + i;
    // The next row's mask and vectors are on their way while this one is worked on.
    u32x4 next[kVecsPer];
    unsigned next_mask[kVecsPer];
    if (i + 1 < i1) {
      load_mask(r + 1, next_mask);
      load_row(rowp + a.row_bytes, next);
    }
    unsigned allowed = valid;
    if (R.allow) {
      unsigned bits = 0;
#pragma unroll
      for (int u = 0; u < kVecsPer; ++u) {
        const unsigned f = kPer == 8 ? mask[u] : mask[u] >> ((tid & 1) * 4) & 0xfu;
        bits |= f << (8 * u);
      }
      allowed &= bits;
    }
    const unsigned plain = allowed & ~special;
    const unsigned hits = allowed & special;
    if constexpr (OUT == kArgmax) {
      float top[kVecsPer];
      float best = -INFINITY;
#pragma unroll
      for (int u = 0; u < kVecsPer; ++u) {
        const unsigned f = (plain >> (8 * u)) & 0xffu;
        if (__all(f == kAll)) {
          top[u] = E::vmax(d[u]);
        } else {
          top[u] = -INFINITY;
#pragma unroll
          for (int k = 0; k < kPer; ++k)
            top[u] = fmaxf(top[u], masked(E::at(d[u], k), f, k));
        }
        best = fmaxf(best, top[u]);
      }
      // The lane's special elements: (value, lowest index).
      float hv = -INFINITY;
      int hi = INT_MAX;
      if (listed > 0) {
        // The wave's vectors through LDS, read back by whichever lane has the element.
#pragma unroll
        for (int u = 0; u < kVecsPer; ++u) stage_s[wave][u * 64 + lane] = d[u];
        wave_sync();
        const unsigned char* stage = reinterpret_cast<const unsigned char*>(stage_s[wave]);
        const bool list = listed <= kListMax;
        if (list) {
          const unsigned theirs = __shfl(allowed, first_at / kPer & 63);
          if (first && (theirs >> (first_at / (64 * kPer) * 8 + first_at % kPer) & 1u)) {
            float x = E::scalar(stage, first_at);
            if (penal) {
              const int extra = ask ? times_on_path(L, q.tree, q.n, i, first_t)
                                    : static_cast<int>(first_rows >> (i & 63)) & 1;
              x = apply_penalties(x, first_word, extra, pen);
            }
            if (first_biased) x += first_bias;
            hv = fmaxf(hv, x);  // (a NaN never wins)
            hi = first_t;
          }
        }
        // The others of a list, 64 at a time; without one each lane takes its own elements.
        unsigned h = hits;
        for (int j0 = 64; list ? j0 < listed : __any(h != 0); j0 += 64) {
          int owner = lane, u = 0, k = 0;
          unsigned word = 0;
          bool node = false, biased = false, on;
          if (list) {
            on = j0 + lane < listed;
            const unsigned e = list_s[wave][on ? j0 + lane : 0];
            const int at = (e >> 16) & 0x7ffu;
            owner = (at / kPer) & 63;
            u = at / (64 * kPer);
            k = at % kPer;
            const unsigned theirs = __shfl(allowed, owner);
            on = on && ((theirs >> (8 * u + k)) & 1u);
            word = e & 0xffffu;
            node = e >> 27 & 1u;
            biased = e >> 28 & 1u;
          } else {
            on = h != 0;
            const int bit = on ? __ffs(h) - 1 : 0;
            h &= h - 1;
            u = bit >> 3;
            k = bit & 7;
            node = node_bits >> bit & 1u;
            biased = bias_bits >> bit & 1u;
          }
          if (on) {
            const int t = (c * kChunkVecs + u * kThreads + wave * 64 + owner) * kPer + k;
            if (!list && hist) word = hist[t];
            const float x = value(E::scalar(stage, (u * 64 + owner) * kPer + k), word, node, biased,
                                  t, i);
            if (x > hv || (x == hv && t < hi)) {
              hv = x;
              hi = t;
            }
          }
        }
        wave_sync();
      }
      const float wave_top = wave_max_f32(fmaxf(best, hv));
      // The first plain element that holds it: its vector and lane by ballots, then the
      // element in scalar registers.  (Places ascend with u, then the lane, then k.)
      int idx = INT_MAX;
      if (wave_top > -INFINITY) {
#pragma unroll
        for (int u = 0; u < kVecsPer; ++u) {
          if (idx == INT_MAX) {
            const unsigned long long who = __ballot(top[u] == wave_top);
            if (who) {
              const int from = __builtin_ctzll(who);
              const unsigned f = read_lane(plain, from) >> (8 * u);
              const unsigned w[4] = {read_lane(d[u].x, from), read_lane(d[u].y, from),
                                     read_lane(d[u].z, from), read_lane(d[u].w, from)};
              const unsigned want = float_key(__float_as_uint(wave_top));
              int k = 0;
#pragma unroll
              for (int j = kPer - 1; j >= 0; --j) {
                const unsigned x = kPer == 4 ? w[j] : j & 1 ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16;
                if ((f >> j & 1u) && float_key(x) == want) k = j;
              }
              idx = (c * kChunkVecs + u * kThreads + wave * 64 + from) * kPer + k;
            }
          }
        }
        if (__any(hv == wave_top)) {
          const int mine = hv == wave_top ? hi : INT_MAX;
          idx = min(idx, read_lane(~wave_max_to_lane63(~mine), 63));
        }
      }
      if (lane == 0) best_s[i - i0][wave] = Partial{wave_top, idx == INT_MAX ? -1 : idx};
    } else {
      unsigned char* o = a.out + r * a.out_bytes;
#pragma unroll
      for (int u = 0; u < kVecsPer; ++u) {
        const int v = v0 + u * kThreads;
        float x[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          x[k] = (allowed >> (8 * u + k)) & 1u ? E::at(d[u], k) : -INFINITY;
        unsigned h = (hits >> (8 * u)) & 0xffu;
        while (h) {
          const int k = __ffs(h) - 1;
          h &= h - 1;
          const float y = own_value(d[u], hw[u], u, k, i);
#pragma unroll
          for (int j = 0; j < kPer; ++j) x[j] = j == k ? y : x[j];
        }
        store_vec<OUT, kPer>(o, v, x, v < a.nvec ? kPer : v == a.nvec ? tail : 0);
      }
    }
    rowp += a.row_bytes;
#pragma unroll
    for (int u = 0; u < kVecsPer; ++u) {
      d[u] = next[u];
      mask[u] = next_mask[u];
    }
  }
  if constexpr (OUT == kArgmax) {
    __syncthreads();
    for (int k = tid; k < i1 - i0; k += kThreads) {
      float bv = best_s[k][0].val;
      int bi = best_s[k][0].idx;
#pragma unroll
      for (int w = 1; w < kWaves; ++w) better_partial(bv, bi, best_s[k][w].val, best_s[k][w].idx);
      a.part[(static_cast<int64_t>(b) * a.rows.rmax + i0 + k) * a.chunks + c] = Partial{bv, bi};
    }
  }
}

// The acceptance over partials [B * rmax][chunks], one workgroup per sequence.
struct ConstrainedAccept {
  RowsArgs rows;
  const Partial* part;
  int splits, V;
  int32_t* accept_len;
  int32_t* bonus;
  int32_t* best_node;
  int32_t* row_argmax;
};

__global__ __launch_bounds__(kThreads) void constrained_accept_kernel(ConstrainedAccept a) {
  __shared__ AcceptLds L;
  const int b = blockIdx.x;
  const RowsArgs& rows = a.rows;
  const SeqRows q = seq_rows(rows, b);
  int32_t* best = a.best_node ? a.best_node + b : nullptr;
  if (q.n == 0) {
    if (threadIdx.x == 0) {
      a.accept_len[b] = 0;
      a.bonus[b] = -1;
      if (best) *best = -1;
    }
    return;
  }
  const Partial* part = a.part + static_cast<int64_t>(b) * rows.rmax * a.splits;
  int32_t* argmax = a.row_argmax ? a.row_argmax + q.row0 : nullptr;
  MergeIn mi;
  merge_load(mi, part, a.splits, 0, q.n);
  if (q.tree) {
    const int64_t o = static_cast<int64_t>(b) * rows.N;
    TreeIn ti;
    tree_load_ids(ti, rows.N, rows.parent + o, rows.draft_ids + o);
    tree_load_tokens(ti, rows.d2t, rows.Vd, a.V);
    merge_finish(mi, part, a.splits, 0, q.n, L.t_s, argmax);
    __syncthreads();
    tree_accept(ti, L.t_s, rows.N, L.anc, L.dep, L.ok, L.red, a.accept_len + b, a.bonus + b, best);
  } else {
    const int32_t* draft = rows.chain_draft + static_cast<int64_t>(b) * rows.K;
    const int draft0 = rows.K > 0 ? chain_load(draft, rows.K) : -1;
    merge_finish(mi, part, a.splits, 0, q.n, L.t_s, argmax);
    __syncthreads();
    chain_accept(draft0, L.t_s, rows.K, draft, a.accept_len + b, a.bonus + b, best);
  }
}

RulesArgs rules_args(const RowsArgs& rows, const wf_logit_rules& rules, const void* logits,
                     int dtype, int32_t V, int64_t row_stride) {
  RulesArgs a{};
  a.rows = rows;
  a.rules = rules;
  a.logits = static_cast<const unsigned char*>(logits);
  a.row_bytes = row_stride * (dtype == WF_BF16 ? 2 : 4);
  a.V = V;
  a.nvec = V / (dtype == WF_BF16 ? 8 : 4);
  const RulesPlan p = rules_plan(dtype, rows.B, rows.rmax, V);
  a.chunks = p.chunks;
  a.groups = p.groups;
  a.group = p.group;
  return a;
}

template <int DT>
void launch_written(const RulesArgs& a, int out_dtype, dim3 grid, hipStream_t stream) {
  if (out_dtype == WF_BF16) {
    hipLaunchKernelGGL((rules_kernel<DT, WF_BF16>), grid, dim3(kThreads), 0, stream, a);
  } else {
    hipLaunchKernelGGL((rules_kernel<DT, WF_F32>), grid, dim3(kThreads), 0, stream, a);
  }
}

}  // namespace

RulesPlan rules_plan(int dtype, int32_t B, int32_t rmax, int32_t V) {
  const int32_t per = kChunkVecs * (dtype == WF_BF16 ? 8 : 4);
  const int32_t chunks = V / per + (V % per != 0);
  // As many workgroups as fill the card a few times over; beyond that, longer groups.
  const int64_t one = static_cast<int64_t>(B) * chunks;
  int64_t groups = one > 0 ? (kRulesBlocks + one - 1) / one : 1;
  const int32_t least = (rmax + kMaxGroup - 1) / kMaxGroup;
  groups = groups > rmax ? rmax : groups;
  groups = groups < least ? least : groups;
  const int32_t group = static_cast<int32_t>((rmax + groups - 1) / groups);
  return RulesPlan{chunks, (rmax + group - 1) / group, group};
}

hipError_t launch_process(const RowsArgs& rows, const wf_logit_rules& rules, const void* logits,
                          int dtype, int32_t V, int64_t row_stride, void* out, int out_dtype,
                          int64_t out_stride, hipStream_t stream) {
  RulesArgs a = rules_args(rows, rules, logits, dtype, V, row_stride);
  a.out = static_cast<unsigned char*>(out);
  a.out_bytes = out_stride * (out_dtype == WF_BF16 ? 2 : 4);
  const dim3 grid(static_cast<unsigned>(rows.B) * a.groups * a.chunks);
  if (dtype == WF_BF16) {
    launch_written<WF_BF16>(a, out_dtype, grid, stream);
  } else {
    launch_written<WF_F32>(a, out_dtype, grid, stream);
  }
  return hipGetLastError();
}

hipError_t launch_constrained(const RowsArgs& rows, const wf_logit_rules& rules,
                              const void* logits, int dtype, int32_t V, int64_t row_stride,
                              Partial* part, int32_t* accept_len, int32_t* bonus,
                              int32_t* best_node, int32_t* row_argmax, hipStream_t stream) {
  RulesArgs a = rules_args(rows, rules, logits, dtype, V, row_stride);
  a.part = part;
  const dim3 grid(static_cast<unsigned>(rows.B) * a.groups * a.chunks);
  if (dtype == WF_BF16) {
    hipLaunchKernelGGL((rules_kernel<WF_BF16, kArgmax>), grid, dim3(kThreads), 0, stream, a);
  } else {
    hipLaunchKernelGGL((rules_kernel<WF_F32, kArgmax>), grid, dim3(kThreads), 0, stream, a);
  }
  if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
  const ConstrainedAccept f{rows,       part,  a.chunks,  V,
                            accept_len, bonus, best_node, row_argmax};
  hipLaunchKernelGGL(constrained_accept_kernel, dim3(rows.B), dim3(kThreads), 0, stream, f);
  return hipGetLastError();
}

}  // namespace wf
