// Token scores: per-token log probability of a given class, entropy and the
// top alternatives, from rows of fp32 logits.
//
// With l = s z the scaled logits of one token (s > 0), m their maximum,
//     S = sum exp(l - m),   U = sum exp(l - m) (l - m),
//     lse = m + log S,   logp_v = l_v - lse,   entropy = log S - U / S.
// U is a sum of terms of one sign (l - m <= 0), so the entropy loses nothing
// to cancellation however large the logits are. S and U of two parts of a row
// join under the larger maximum M: with c = exp(m - M),
//     S -> c S,   U -> c (U + (m - M) S).
//
// The alternatives are ordered by (unscaled logit, lower class first), held as
// one 64-bit key a class, so every order is total and ties never depend on
// the schedule.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "internal.h"
#include "score.cuh"

namespace vce {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowCand = 1024;   // candidates kept in shared memory

// One block per row of logits. First pass: running (m, S, U) and the largest
// key of each thread's columns. The K-th largest of the 256 thread maxima
// bounds the K-th largest key of the row from below, since they are K distinct
// elements of it; the second pass collects what reaches the bound and ranks it
// by counting. Rows where more than kRowCand keys reach the bound (their
// largest logits all in a few threads' columns) take K scans instead.
__global__ void __launch_bounds__(kRowThreads)
    score_rows_kernel(const float* __restrict__ Z, int64_t ldz, int V, int64_t t0, const int64_t* __restrict__ targets,
                      int64_t ignore_index, float scale, int K, float* __restrict__ logp, float* __restrict__ entropy,
                      float* __restrict__ lse, int64_t* __restrict__ top_ids, float* __restrict__ top_logp,
                      int32_t* status) {
  __shared__ float sm[kRowThreads / 32], sS[kRowThreads / 32], sU[kRowThreads / 32];
  __shared__ uint64_t skey[kRowThreads];
  __shared__ uint64_t cand[kRowCand];
  __shared__ uint64_t best[kMaxTop];
  __shared__ uint64_t s_bound;
  __shared__ int s_n;
  grid_dep_launch();
  grid_dep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float* z = Z + static_cast<int64_t>(blockIdx.x) * ldz;
  const int64_t t = t0 + blockIdx.x;
  const uint32_t Vu = static_cast<uint32_t>(V);
  ScoreStat a = score_stat_empty();
  uint64_t kmax = 0;
  for (uint32_t v = 4 * tid; v < Vu; v += 4 * kRowThreads) {
    const float4 q = *reinterpret_cast<const float4*>(z + v);   // rows are padded to a multiple of 4
    const float x[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (v + j < Vu) {
        score_stat_add(a, x[j] * scale);
        const uint64_t k = top_key(x[j], v + j);
        kmax = k > kmax ? k : kmax;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ScoreStat b{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.S, o),
                __shfl_xor_sync(0xffffffffu, a.U, o)};
    a = (lane & o) == 0 ? score_stat_join(a, b) : score_stat_join(b, a);
  }
  if (lane == 0) {
    sm[warp] = a.m;
    sS[warp] = a.S;
    sU[warp] = a.U;
  }
  skey[tid] = kmax;
  if (tid == 0) {
    s_n = 0;
    s_bound = 0;
  }
  __syncthreads();
  a = ScoreStat{sm[0], sS[0], sU[0]};
  for (int w = 1; w < kRowThreads / 32; ++w) a = score_stat_join(a, ScoreStat{sm[w], sS[w], sU[w]});
  const float l = score_lse(a);
  if (tid == 0) {
    if (lse) lse[t] = l;
    const int64_t y = targets ? targets[t] : -1;
    const bool valid = targets && y >= 0 && y < V;
    if (targets && !valid && y != ignore_index && status) atomicCAS(status, 0, static_cast<int>(VCE_ERR_BAD_INDEX));
    if (logp) logp[t] = valid ? fmaf(z[y], scale, -l) : 0.0f;
    if (entropy) entropy[t] = (!targets || valid) ? score_entropy(a) : 0.0f;
  }
  if (K == 0) return;
  int rank = 0;
  if (kmax)
    for (int i = 0; i < kRowThreads; ++i) rank += skey[i] > kmax ? 1 : 0;
  if (kmax && rank == K - 1) s_bound = kmax;   // stays 0 when fewer than K threads hold a key
  if (tid < K) best[tid] = 0;
  __syncthreads();
  const uint64_t bound = s_bound;
  for (uint32_t v = 4 * tid; v < Vu; v += 4 * kRowThreads) {
    const float4 q = *reinterpret_cast<const float4*>(z + v);
    const float x[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t k = v + j < Vu ? top_key(x[j], v + j) : 0;
      if (k != 0 && k >= bound) {
        const int at = atomicAdd(&s_n, 1);
        if (at < kRowCand) cand[at] = k;
      }
    }
  }
  __syncthreads();
  const int n = s_n;
  if (n <= kRowCand) {
    for (int i = tid; i < n; i += kRowThreads) {
      const uint64_t k = cand[i];
      int r = 0;
      for (int j = 0; j < n; ++j) r += cand[j] > k ? 1 : 0;
      if (r < K) best[r] = k;
    }
    __syncthreads();
  } else {
    uint64_t below = ~uint64_t(0);
    for (int i = 0; i < K; ++i) {   // the largest key below the last one taken
      uint64_t k = 0;
      for (uint32_t v = tid; v < Vu; v += kRowThreads) {
        const uint64_t kv = top_key(z[v], v);
        if (kv < below && kv > k) k = kv;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t k2 = __shfl_xor_sync(0xffffffffu, k, o);
        k = k2 > k ? k2 : k;
      }
      __syncthreads();
      if (lane == 0) skey[warp] = k;
      __syncthreads();
      below = skey[0];
      for (int w = 1; w < kRowThreads / 32; ++w) below = skey[w] > below ? skey[w] : below;
      if (tid == 0) best[i] = below;
    }
    __syncthreads();
  }
  if (tid < K) write_top(best[tid], t * K + tid, scale, l, top_ids, top_logp);
}

// Rows of h whose token takes part in the gradient, zeros for the others: the
// product G^T h then never multiplies a zero of G by what an ignored token's
// row holds (which may be infinite or NaN). Targets that are neither a real
// class nor ignored are reported.
__global__ void __launch_bounds__(256) mask_rows_kernel(const uint4* __restrict__ h, const int64_t* __restrict__ targets,
                                                        int V, int64_t ignore_index, int row16, int64_t n16, uint4* __restrict__ out,
                                                        int32_t* status) {
  grid_dep_launch();
  grid_dep_wait();
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n16;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t y = targets[i / row16];
    const bool valid = y >= 0 && y < V;
    if (!valid && y != ignore_index && status) atomicCAS(status, 0, static_cast<int>(VCE_ERR_BAD_INDEX));
    out[i] = valid ? h[i] : make_uint4(0, 0, 0, 0);
  }
}

}  // namespace

cudaError_t launch_score_rows(const float* Z, int64_t ldz, int64_t rows, int V, int64_t t0, const int64_t* targets,
                              int64_t ignore_index, float scale, int K, float* logp, float* entropy, float* lse,
                              int64_t* top_ids, float* top_logp, int32_t* status, cudaStream_t st) {
  const cudaError_t e = launch_dependent(score_rows_kernel, dim3(static_cast<unsigned>(rows)), dim3(kRowThreads), 0, st,
                                         Z, ldz, V, t0, targets, ignore_index, scale, K, logp, entropy, lse, top_ids,
                                         top_logp, status);
  note_launch(VCE_K_SCORE_ROWS, st);
  return e;
}

cudaError_t launch_mask_rows(const void* h, const int64_t* targets, int64_t T, int V, int64_t ignore_index,
                             int64_t row_bytes, void* out, int32_t* status, cudaStream_t st) {
  const int64_t n16 = T * (row_bytes / 16);
  const int64_t cap = static_cast<int64_t>(current_device_info().num_sms) * 8;
  const int64_t want = ceil_div(n16, 256);
  const cudaError_t e = launch_dependent(mask_rows_kernel, dim3(static_cast<unsigned>(want < cap ? want : cap)),
                                         dim3(256), 0, st, static_cast<const uint4*>(h), targets, V,
                                         ignore_index, static_cast<int>(row_bytes / 16), n16,
                                         static_cast<uint4*>(out), status);
  note_launch(VCE_K_MASK_ROWS, st);
  return e;
}

}  // namespace vce
