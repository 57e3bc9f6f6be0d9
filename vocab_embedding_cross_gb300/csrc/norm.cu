// Layer and root-mean-square normalisation of the hidden states that enter the
// head, forward and backward.
//
//   forward    xhat = (x - mean) rstd,  y = xhat w + b,
//              rstd = 1 / sqrt(mean((x - mean)^2) + eps); mean = 0 for RMS
//   backward   g = dy w;  dx = rstd (g - mean(g) - xhat mean(g xhat))
//              (without the mean(g) term for RMS);
//              dw = sum_t dy xhat,  db = sum_t dy
// Every sum is fp32 and taken in an order fixed by the sizes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "internal.h"

namespace vce {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormParts = 128;   // row groups of the weight gradient

__device__ __forceinline__ float load_f(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p, int64_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ void store_f(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store_f(__nv_bfloat16* p, int64_t i, float v) { p[i] = __float2bfloat16_rn(v); }

__device__ __forceinline__ float block_sum(float v, float* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) s += sh[w];
  return s;
}

template <typename E>
__global__ void __launch_bounds__(kNormThreads)
    norm_fwd_kernel(int H, int rms, const E* __restrict__ x, const E* __restrict__ w, const E* __restrict__ b, float eps,
                    E* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ float sh[kNormThreads / 32];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * H;
  float mu = 0.0f;
  if (!rms) {
    float s = 0.0f;
    for (int i = threadIdx.x; i < H; i += kNormThreads) s += load_f(x, row + i);
    mu = block_sum(s, sh) / static_cast<float>(H);
  }
  float q = 0.0f;
  for (int i = threadIdx.x; i < H; i += kNormThreads) {
    const float d = load_f(x, row + i) - mu;
    q = fmaf(d, d, q);
  }
  const float r = 1.0f / sqrtf(block_sum(q, sh) / static_cast<float>(H) + eps);
  for (int i = threadIdx.x; i < H; i += kNormThreads) {
    float v = (load_f(x, row + i) - mu) * r;
    if (w) v *= load_f(w, i);
    if (b) v += load_f(b, i);
    store_f(y, row + i, v);
  }
  if (threadIdx.x == 0) {
    if (mean) mean[blockIdx.x] = mu;
    if (rstd) rstd[blockIdx.x] = r;
  }
}

template <typename E, typename D>
__global__ void __launch_bounds__(kNormThreads)
    norm_dx_kernel(int H, int rms, const E* __restrict__ x, const E* __restrict__ w, const D* __restrict__ dy,
                   const float* __restrict__ mean, const float* __restrict__ rstd, E* __restrict__ dx) {
  __shared__ float sh[kNormThreads / 32];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * H;
  const float mu = rms ? 0.0f : mean[blockIdx.x], r = rstd[blockIdx.x];
  float sg = 0.0f, sgx = 0.0f;
  for (int i = threadIdx.x; i < H; i += kNormThreads) {
    const float g = load_f(dy, row + i) * (w ? load_f(w, i) : 1.0f);
    sg += g;
    sgx = fmaf(g, (load_f(x, row + i) - mu) * r, sgx);
  }
  const float mg = rms ? 0.0f : block_sum(sg, sh) / static_cast<float>(H);
  const float mgx = block_sum(sgx, sh) / static_cast<float>(H);
  for (int i = threadIdx.x; i < H; i += kNormThreads) {
    const float g = load_f(dy, row + i) * (w ? load_f(w, i) : 1.0f);
    store_f(dx, row + i, r * (g - mg - (load_f(x, row + i) - mu) * r * mgx));
  }
}

// part[p][0][i] = sum over rows t = p, p + gridDim.y, ... of dy xhat; part[p][1][i] of dy.
template <typename E, typename D>
__global__ void __launch_bounds__(kNormThreads)
    norm_dw_kernel(int T, int H, int rms, const E* __restrict__ x, const D* __restrict__ dy,
                   const float* __restrict__ mean, const float* __restrict__ rstd, float* __restrict__ part) {
  const int i = blockIdx.x * kNormThreads + threadIdx.x;
  if (i >= H) return;
  float a = 0.0f, b = 0.0f;
  for (int64_t t = blockIdx.y; t < T; t += gridDim.y) {
    const float d = load_f(dy, t * H + i);
    a = fmaf(d, (load_f(x, t * H + i) - (rms ? 0.0f : mean[t])) * rstd[t], a);
    b += d;
  }
  part[(static_cast<int64_t>(blockIdx.y) * 2) * H + i] = a;
  part[(static_cast<int64_t>(blockIdx.y) * 2 + 1) * H + i] = b;
}

__global__ void __launch_bounds__(kNormThreads)
    norm_dw_sum_kernel(int H, int parts, int accumulate, const float* __restrict__ part, float* __restrict__ dw,
                       float* __restrict__ db) {
  const int i = blockIdx.x * kNormThreads + threadIdx.x;
  if (i >= H) return;
  float a = 0.0f, b = 0.0f;
  for (int p = 0; p < parts; ++p) {
    a += part[(static_cast<int64_t>(p) * 2) * H + i];
    b += part[(static_cast<int64_t>(p) * 2 + 1) * H + i];
  }
  if (dw) dw[i] = accumulate ? dw[i] + a : a;
  if (db) db[i] = accumulate ? db[i] + b : b;
}

template <typename E, typename D>
cudaError_t bwd_typed(const vce_problem& p, bool rms, const void* x, const void* w, const void* dy, const float* mean,
                      const float* rstd, void* dx, float* dw, float* db, bool accumulate, float* part,
                      cudaStream_t st) {
  const int H = static_cast<int>(p.H), T = static_cast<int>(p.T);
  if (dx) {
    norm_dx_kernel<E, D><<<static_cast<unsigned>(T), kNormThreads, 0, st>>>(
        H, rms, static_cast<const E*>(x), static_cast<const E*>(w), static_cast<const D*>(dy), mean, rstd,
        static_cast<E*>(dx));
    note_launch(VCE_K_NORM_BWD, st);
  }
  if (dw || db) {
    const int parts = norm_parts(p);
    const dim3 grid(static_cast<unsigned>(ceil_div(H, kNormThreads)), static_cast<unsigned>(parts));
    norm_dw_kernel<E, D><<<grid, kNormThreads, 0, st>>>(T, H, rms, static_cast<const E*>(x),
                                                        static_cast<const D*>(dy), mean, rstd, part);
    note_launch(VCE_K_NORM_BWD, st);
    norm_dw_sum_kernel<<<static_cast<unsigned>(ceil_div(H, kNormThreads)), kNormThreads, 0, st>>>(
        H, parts, accumulate, part, dw, db);
    note_launch(VCE_K_NORM_SUM, st);
  }
  return cudaGetLastError();
}

}  // namespace

int norm_parts(const vce_problem& p) { return static_cast<int>(p.T < kNormParts ? p.T : kNormParts); }
size_t norm_ws_bytes(const vce_problem& p) {
  return align_up(static_cast<size_t>(norm_parts(p)) * 2 * static_cast<size_t>(p.H) * sizeof(float), kWsAlign);
}

cudaError_t launch_norm_fwd(const vce_problem& p, bool rms, const void* x, const void* w, const void* b, float eps,
                            void* y, float* mean, float* rstd, cudaStream_t st) {
  const unsigned T = static_cast<unsigned>(p.T);
  const int H = static_cast<int>(p.H);
  if (p.dtype == VCE_BF16) {
    using E = __nv_bfloat16;
    norm_fwd_kernel<E><<<T, kNormThreads, 0, st>>>(H, rms, static_cast<const E*>(x), static_cast<const E*>(w),
                                                   static_cast<const E*>(b), eps, static_cast<E*>(y), mean, rstd);
  } else {
    norm_fwd_kernel<float><<<T, kNormThreads, 0, st>>>(H, rms, static_cast<const float*>(x),
                                                       static_cast<const float*>(w), static_cast<const float*>(b), eps,
                                                       static_cast<float*>(y), mean, rstd);
  }
  note_launch(VCE_K_NORM_FWD, st);
  return cudaGetLastError();
}

cudaError_t launch_norm_bwd(const vce_problem& p, bool rms, const void* x, const void* w, const void* dy, bool dy_bf16,
                            const float* mean, const float* rstd, void* dx, float* dw, float* db, bool accumulate,
                            void* ws, cudaStream_t st) {
  float* part = static_cast<float*>(ws);
  if (p.dtype != VCE_BF16 && dy_bf16)
    return bwd_typed<float, __nv_bfloat16>(p, rms, x, w, dy, mean, rstd, dx, dw, db, accumulate, part, st);
  if (p.dtype != VCE_BF16)
    return bwd_typed<float, float>(p, rms, x, w, dy, mean, rstd, dx, dw, db, accumulate, part, st);
  if (dy_bf16)
    return bwd_typed<__nv_bfloat16, __nv_bfloat16>(p, rms, x, w, dy, mean, rstd, dx, dw, db, accumulate, part, st);
  return bwd_typed<__nv_bfloat16, float>(p, rms, x, w, dy, mean, rstd, dx, dw, db, accumulate, part, st);
}

}  // namespace vce
