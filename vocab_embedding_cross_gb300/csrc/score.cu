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
constexpr int kListThreads = 128;

// One block per row of logits (the fp32 path): the statistics and, for
// alternatives, the largest key of each thread's classes in a first pass over
// the row, then the keys that reach the bound.
__global__ void __launch_bounds__(kRowThreads)
    score_rows_kernel(const float* __restrict__ Z, int64_t ldz, int V, const int64_t* __restrict__ targets,
                      int64_t ignore_index, float scale, int K, float* __restrict__ logp, float* __restrict__ entropy,
                      float* __restrict__ lse, int64_t* __restrict__ top_ids, float* __restrict__ top_logp,
                      int32_t* status) {
  __shared__ TopShared top;
  __shared__ ScoreStat sh[32];
  grid_dep_launch();
  top_init(top);
  grid_dep_wait();
  const float* z = Z + static_cast<int64_t>(blockIdx.x) * ldz;
  const int64_t t = blockIdx.x;
  const uint32_t n = static_cast<uint32_t>(V);
  ScoreStat a = score_stat_empty();
  uint64_t kmax = 0;
  for (uint32_t v = threadIdx.x; v < n; v += kRowThreads) {
    const float x = z[v];
    score_stat_add(a, x * scale);
    const uint64_t k = top_key(x, v);
    kmax = k > kmax ? k : kmax;
  }
  if (K) top_raise(top, kmax);
  a = block_join(a, sh);
  const float l = score_lse(a);
  if (threadIdx.x == 0) {
    const int64_t y = targets ? targets[t] : -1;
    write_scores(a, l, t, V, targets, ignore_index, z + (y >= 0 && y < V ? y : 0), scale, logp, entropy, lse, status);
  }
  if (K == 0) return;
  const uint64_t bound = top_bound(top, K);
  for (uint32_t v = threadIdx.x; v < n; v += kRowThreads) top_collect(top, top_key(z[v], v), bound);
  if (!top_rank(top, K)) top_scan(top, n, K, [&](uint32_t v) { return top_key(z[v], v); });
  if (threadIdx.x < K) write_top(top.best[threadIdx.x], t * K + threadIdx.x, scale, l, top_ids, top_logp);
}

// One block per token: joins the tensor-core scores' unit statistics and takes
// the alternatives from the row's list, which holds every logit that can be one
// (a few hundred entries of 150000, so 128 threads; T blocks of them take 3 us a
// thousand tokens beside the 330 us of their product at H = 2048, V = 151936).
__global__ void __launch_bounds__(kListThreads)
    score_lists_kernel(ScoreLists sl, int V, int n_units, const float* __restrict__ ztgt,
                       const int64_t* __restrict__ targets, int64_t ignore_index, float* __restrict__ logp,
                       float* __restrict__ entropy, float* __restrict__ lse, int64_t* __restrict__ top_ids,
                       float* __restrict__ top_logp, int32_t* status) {
  __shared__ TopShared top;
  __shared__ ScoreStat sh[32];
  grid_dep_launch();
  top_init(top);
  grid_dep_wait();
  const int64_t t = blockIdx.x;
  const int K = sl.K;
  ScoreStat a = score_stat_empty();
  for (int i = threadIdx.x; i < n_units; i += kListThreads) {
    const float4 p = sl.part[t * n_units + i];
    a = score_stat_join(a, ScoreStat{p.x, p.y, p.z});
  }
  const uint32_t n = K ? static_cast<uint32_t>(sl.row_count[t]) : 0;
  const uint2* list = sl.row_list + t * sl.row_cap;
  auto key_at = [&](uint32_t i) { return (static_cast<uint64_t>(list[i].x) << 32) | list[i].y; };
  uint64_t kmax = 0;
  for (uint32_t i = threadIdx.x; i < n; i += kListThreads) {
    const uint64_t k = key_at(i);
    kmax = k > kmax ? k : kmax;
  }
  if (K) top_raise(top, kmax);
  a = block_join(a, sh);
  const float l = score_lse(a);
  if (threadIdx.x == 0) write_scores(a, l, t, V, targets, ignore_index, ztgt + t, sl.scale, logp, entropy, lse, status);
  if (K == 0) return;
  const uint64_t bound = top_bound(top, K);
  for (uint32_t i = threadIdx.x; i < n; i += kListThreads) top_collect(top, key_at(i), bound);
  if (!top_rank(top, K)) top_scan(top, n, K, key_at);
  if (threadIdx.x < K) write_top(top.best[threadIdx.x], t * K + threadIdx.x, sl.scale, l, top_ids, top_logp);
}

// Zeroes n words (a kernel and not a memset: the kernel after it can set itself up meanwhile).
__global__ void __launch_bounds__(256) zero_words_kernel(uint4* __restrict__ p, int64_t n16) {
  grid_dep_launch();
  grid_dep_wait();
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n16;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x)
    p[i] = make_uint4(0, 0, 0, 0);
}

}  // namespace

cudaError_t launch_score_rows(const float* Z, int64_t ldz, int64_t rows, int V, const int64_t* targets,
                              int64_t ignore_index, float scale, int K, float* logp, float* entropy, float* lse,
                              int64_t* top_ids, float* top_logp, int32_t* status, cudaStream_t st) {
  const cudaError_t e = launch_dependent(score_rows_kernel, dim3(static_cast<unsigned>(rows)), dim3(kRowThreads), 0, st,
                                         Z, ldz, V, targets, ignore_index, scale, K, logp, entropy, lse, top_ids,
                                         top_logp, status);
  note_launch(VCE_K_SCORE_ROWS, st);
  return e;
}

cudaError_t launch_score_lists(const ScoreLists& sl, int64_t T, int V, int n_units, const float* ztgt,
                               const int64_t* targets, int64_t ignore_index, float* logp, float* entropy, float* lse,
                               int64_t* top_ids, float* top_logp, int32_t* status, cudaStream_t st) {
  const cudaError_t e = launch_dependent(score_lists_kernel, dim3(static_cast<unsigned>(T)), dim3(kListThreads), 0, st,
                                         sl, V, n_units, ztgt, targets, ignore_index, logp, entropy, lse, top_ids,
                                         top_logp, status);
  note_launch(VCE_K_SCORE_LISTS, st);
  return e;
}

cudaError_t launch_zero_words(void* p, size_t bytes, cudaStream_t st) {
  const int64_t n16 = static_cast<int64_t>(bytes / 16), want = ceil_div(n16, 256);
  const int64_t cap = static_cast<int64_t>(current_device_info().num_sms) * 4;
  const cudaError_t e = launch_dependent(zero_words_kernel, dim3(static_cast<unsigned>(want < cap ? want : cap)),
                                         dim3(256), 0, st, static_cast<uint4*>(p), n16);
  note_launch(VCE_K_SCORE_ZERO, st);
  return e;
}

}  // namespace vce
