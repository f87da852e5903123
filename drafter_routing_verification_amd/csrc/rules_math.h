// The rules of decoding on one logit (wf_logit_rules).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace wf {

struct Penalties {
  float repetition, frequency, presence;
};

// Every operation rounded once, as the definition states it: no contraction into
// fused multiply-adds, and an IEEE division.
__device__ inline float apply_penalties(float x, unsigned word, int extra, const Penalties& p) {
#pragma clang fp contract(off)
  const int count = static_cast<int>(word & 0x7fffu) + extra;
  const bool put_out = count > 0;
  if (!put_out && !(word & 0x8000u)) return x;
  x = x > 0.f ? x / p.repetition : x * p.repetition;
  const float f = p.frequency * static_cast<float>(count);
  x = x - f;
  x = x - (put_out ? p.presence : 0.f);
  return x;
}

// First index in [lo, hi) of ascending ids with ids[i] >= v.
__device__ inline int lower_bound(const int32_t* __restrict__ ids, int lo, int hi, int v) {
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (ids[mid] < v) {
      lo = mid + 1;
    } else {
      hi = mid;
    }
  }
  return lo;
}

// bfloat16 of x, rounded to nearest even (NaN stays NaN).
__device__ inline unsigned bf16_bits(float x) {
  const unsigned u = __float_as_uint(x);
  if ((u & 0x7fffffffu) > 0x7f800000u) return (u >> 16) | 0x40u;
  return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}

}  // namespace wf
