// Device helpers of the token scores: running statistics of one row of scaled
// logits and the total order of its alternatives.
#pragma once

#include <cmath>
#include <cstdint>

namespace vce {

// Maximum m, S = sum exp(l - m) and U = sum exp(l - m) (l - m) of part of a row.
struct ScoreStat {
  float m, S, U;
};
__device__ __forceinline__ ScoreStat score_stat_empty() { return ScoreStat{-INFINITY, 0.0f, 0.0f}; }

// Multiplying U's exponent term by a difference clamped at -200 keeps
// exp(-inf) * -inf from becoming NaN; exp(-200) is 0 in fp32 anyway.
__device__ __forceinline__ void score_stat_add(ScoreStat& a, float l) {
  if (l > a.m) {
    const float d = a.m == -INFINITY ? 0.0f : a.m - l;   // nothing summed yet: S and U are 0 or NaN
    const float c = expf(d);
    a.U = c * fmaf(d, a.S, a.U);
    a.S = c * a.S;
    a.m = l;
  }
  const float d = l - (a.m == -INFINITY ? 0.0f : a.m);
  const float e = expf(d);
  a.S += e;
  a.U = fmaf(e, fmaxf(d, -200.0f), a.U);
}

__device__ __forceinline__ ScoreStat score_stat_join(const ScoreStat& a, const ScoreStat& b) {
  const float M = fmaxf(a.m, b.m);
  const float ref = M == -INFINITY ? 0.0f : M;
  // a part that has seen nothing finite holds S = U = 0, or NaN, under any scale
  const float da = a.m == -INFINITY ? 0.0f : a.m - ref, db = b.m == -INFINITY ? 0.0f : b.m - ref;
  const float ca = expf(da), cb = expf(db);
  return ScoreStat{M, ca * a.S + cb * b.S, ca * fmaf(da, a.S, a.U) + cb * fmaf(db, b.S, b.U)};
}

__device__ __forceinline__ float score_lse(const ScoreStat& a) { return a.m + logf(a.S); }
__device__ __forceinline__ float score_entropy(const ScoreStat& a) { return logf(a.S) - a.U / a.S; }

// Monotone map of fp32 to unsigned (both zeros to the same word).
__device__ __forceinline__ uint32_t ordered_bits(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float ordered_value(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o ^ 0x80000000u : ~o);
}
// Larger logit first, lower class first between equal ones; 0 (less than every
// class's key) for NaN, which is never listed.
__device__ __forceinline__ uint64_t top_key(float z, uint32_t col) {
  return z == z ? (static_cast<uint64_t>(ordered_bits(z)) << 32) | (0xFFFFFFFFu - col) : 0;
}
__device__ __forceinline__ void write_top(uint64_t key, int64_t at, float scale, float lse,
                                          int64_t* __restrict__ top_ids, float* __restrict__ top_logp) {
  const bool have = key != 0;
  top_ids[at] = have ? static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(key)) : -1;
  top_logp[at] = have ? fmaf(ordered_value(static_cast<uint32_t>(key >> 32)), scale, -lse) : NAN;
}

}  // namespace vce
