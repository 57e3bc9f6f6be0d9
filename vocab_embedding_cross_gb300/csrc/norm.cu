// Layer and root-mean-square normalisation of the hidden states that enter the
// head, forward and backward.
//
//   forward    xhat = (x - mean) rstd,  y = xhat w + b,
//              rstd = 1 / sqrt(mean((x - mean)^2) + eps); mean = 0 for RMS
//   backward   g = dy w;  dx = rstd (g - mean(g) - xhat mean(g xhat))
//              (without the mean(g) term for RMS);
//              dw = sum_t dy xhat,  db = sum_t dy
// Every sum is fp32 and taken in an order fixed by the sizes and the number of SMs.
//
// Both directions are bound by memory: x (and dy) once in, y (or dx) once out.
// A row belongs to a group of 32 to 1024 threads that keeps it in registers
// between the statistics and the output, so each byte moves once; the groups of
// a persistent grid go through the rows with the next row's loads in flight
// while a row is worked on. In the backward each thread's columns are the same
// for every row, so the weight gradients are summed in its registers over all
// rows of the group and leave the CTA once, as one partial per CTA (2 H floats
// for each of at most 152), which a second small kernel adds up.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "internal.h"

namespace vce {
namespace {

// 16 bytes of E as floats (8 bf16 or 4 fp32).
template <typename E>
struct Row16;
template <>
struct Row16<float> {
  static constexpr int N = 4;
  float4 v;
  __device__ __forceinline__ void load(const float* p, int64_t i) { v = reinterpret_cast<const float4*>(p)[i]; }
  __device__ __forceinline__ void get(float (&f)[4]) const {
    f[0] = v.x;
    f[1] = v.y;
    f[2] = v.z;
    f[3] = v.w;
  }
  __device__ __forceinline__ static void store(float* p, int64_t i, const float (&f)[4]) {
    reinterpret_cast<float4*>(p)[i] = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <>
struct Row16<__nv_bfloat16> {
  static constexpr int N = 8;
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int64_t i) { v = reinterpret_cast<const uint4*>(p)[i]; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ static void store(__nv_bfloat16* p, int64_t i, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    reinterpret_cast<uint4*>(p)[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
// N elements of D beside N of another type (dy beside x).
template <typename D, int N>
struct RowN {
  static constexpr int kVecs = N / Row16<D>::N > 0 ? N / Row16<D>::N : 1;
  static constexpr bool kHalf = N < Row16<D>::N;   // 4 bf16: half a vector
  Row16<D> v[kVecs];
  __device__ __forceinline__ void load(const D* p, int64_t i) {
    if constexpr (kHalf) {
      const uint2 h = reinterpret_cast<const uint2*>(p)[i];
      v[0].v = make_uint4(h.x, h.y, 0, 0);
    } else {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) v[j].load(p, i * kVecs + j);
    }
  }
  __device__ __forceinline__ void get(float (&f)[N]) const {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      float g[Row16<D>::N];
      v[j].get(g);
#pragma unroll
      for (int k = 0; k < Row16<D>::N; ++k)
        if (j * Row16<D>::N + k < N) f[j * Row16<D>::N + k] = g[k];
    }
  }
};

// Sum over a group of G threads (a multiple of 32); every thread gets the same
// bits. The two halves of `sh` are used in turn, so one barrier a sum is enough.
struct GroupSum {
  float* sh;   // [2][32] of this group
  int G, id, buf;
  __device__ __forceinline__ float operator()(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (G == 32) return v;
    float* s = sh + 32 * buf;
    buf ^= 1;
    const int warp = static_cast<int>(threadIdx.x % G) >> 5;
    if ((threadIdx.x & 31) == 0) s[warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(G) : "memory");
    v = 0.0f;
    for (int w = 0; w < (G >> 5); ++w) v += s[w];
    return v;
  }
};

constexpr int kFwdThreads = 256;
constexpr int kBwdThreads = 512;
constexpr int kMaxGroups = 16;   // of one CTA (named barriers 1 to 15 serve groups of two warps and more)

// VPT vectors a thread. Up to two of them, the weights stay in registers over the
// rows and the next row is fetched ahead (64 registers, so that 1024 threads of an
// SM hold 32 KB of rows in flight); four (rows of over 2048 vectors) do without.
template <typename E, int VPT>
__global__ void __launch_bounds__(1024)
    norm_fwd_kernel(int64_t T, int H, int G, int rms, const E* __restrict__ x, const E* __restrict__ w,
                    const E* __restrict__ b, float eps, E* __restrict__ y, float* __restrict__ mean,
                    float* __restrict__ rstd) {
  constexpr int N = Row16<E>::N;
  constexpr bool kAhead = VPT <= 2;
  __shared__ float sh[kMaxGroups][64];
  grid_dep_launch();
  grid_dep_wait();
  const int nv = H / N, groups = static_cast<int>(blockDim.x) / G;
  const int g = static_cast<int>(threadIdx.x) / G, i0 = static_cast<int>(threadIdx.x) % G;
  GroupSum sum{sh[g], G, 1 + g, 0};
  const float inv = 1.0f / static_cast<float>(H);
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  Row16<E> wv[VPT], bv[VPT], xv[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = i0 + j * G;
    if (kAhead && i < nv && w) wv[j].load(w, i);
    if (kAhead && i < nv && b) bv[j].load(b, i);
  }
  int64_t t = static_cast<int64_t>(blockIdx.x) * groups + g;
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (row < T && i0 + j * G < nv) xv[j].load(x, row * nv + i0 + j * G);
  };
  if (kAhead) fetch(t);
  for (; t < T; t += step) {
    float f[VPT][N];
    float s = 0.0f;
    if (!kAhead) fetch(t);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (i0 + j * G < nv) xv[j].get(f[j]);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (i0 + j * G >= nv) f[j][k] = 0.0f;
        s += f[j][k];
      }
    }
    if (kAhead) fetch(t + step);
    const float mu = rms ? 0.0f : sum(s) * inv;
    float q = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        f[j][k] -= mu;
        if (i0 + j * G < nv) q = fmaf(f[j][k], f[j][k], q);
      }
    const float r = 1.0f / sqrtf(sum(q) * inv + eps);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = i0 + j * G;
      if (i >= nv) continue;
      float c[N];
      if (!kAhead && w) wv[j].load(w, i);
      if (!kAhead && b) bv[j].load(b, i);
      if (w) wv[j].get(c);
#pragma unroll
      for (int k = 0; k < N; ++k) f[j][k] *= w ? r * c[k] : r;
      if (b) {
        bv[j].get(c);
#pragma unroll
        for (int k = 0; k < N; ++k) f[j][k] += c[k];
      }
      Row16<E>::store(y, t * nv + i, f[j]);
    }
    if (i0 == 0) {
      if (mean) mean[t] = mu;
      if (rstd) rstd[t] = r;
    }
  }
}

template <typename E, typename D, int VPT>
__global__ void __launch_bounds__(kBwdThreads)
    norm_bwd_kernel(int64_t T, int H, int G, int rms, const E* __restrict__ x, const E* __restrict__ w,
                    const D* __restrict__ dy, const float* __restrict__ mean, const float* __restrict__ rstd,
                    E* __restrict__ dx, float* __restrict__ part) {
  constexpr int N = Row16<E>::N;
  __shared__ float sh[kMaxGroups][128];
  __shared__ float col[2][4096];   // used when the CTA has several groups (H <= 4096)
  grid_dep_launch();
  grid_dep_wait();
  const int nv = H / N, groups = static_cast<int>(blockDim.x) / G;
  const int g = static_cast<int>(threadIdx.x) / G, i0 = static_cast<int>(threadIdx.x) % G;
  const float inv = 1.0f / static_cast<float>(H);
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const int warp = i0 >> 5, lane = static_cast<int>(threadIdx.x & 31);
  int buf = 0;
  Row16<E> wv[VPT], xv[VPT];
  RowN<D, N> dv[VPT];
  float aw[VPT][N], ab[VPT][N];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if (w && i0 + j * G < nv) wv[j].load(w, i0 + j * G);
#pragma unroll
    for (int k = 0; k < N; ++k) aw[j][k] = ab[j][k] = 0.0f;
  }
  int64_t t = static_cast<int64_t>(blockIdx.x) * groups + g;
  float mu = 0.0f, r = 0.0f;
  auto fetch = [&](int64_t row) {
    if (row >= T) return;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (i0 + j * G < nv) {
        xv[j].load(x, row * nv + i0 + j * G);
        dv[j].load(dy, row * nv + i0 + j * G);
      }
    mu = rms ? 0.0f : mean[row];
    r = rstd[row];
  };
  fetch(t);
  for (; t < T; t += step) {
    float xh[VPT][N], gr[VPT][N];
    float sg = 0.0f, sx = 0.0f;
    const float rt = r;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (i0 + j * G >= nv) continue;
      float c[N];
      xv[j].get(xh[j]);
      dv[j].get(gr[j]);
      if (w) wv[j].get(c);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        xh[j][k] = (xh[j][k] - mu) * rt;
        aw[j][k] = fmaf(gr[j][k], xh[j][k], aw[j][k]);
        ab[j][k] += gr[j][k];
        if (w) gr[j][k] *= c[k];
        sg += gr[j][k];
        sx = fmaf(gr[j][k], xh[j][k], sx);
      }
    }
    fetch(t + step);
    if (!dx) continue;
    // both sums with one barrier
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sg += __shfl_xor_sync(0xffffffffu, sg, o);
      sx += __shfl_xor_sync(0xffffffffu, sx, o);
    }
    if (G > 32) {
      float* s = sh[g] + 64 * buf;
      buf ^= 1;
      if (lane == 0) {
        s[2 * warp] = sg;
        s[2 * warp + 1] = sx;
      }
      asm volatile("bar.sync %0, %1;" ::"r"(1 + g), "r"(G) : "memory");
      sg = sx = 0.0f;
      for (int i = 0; i < (G >> 5); ++i) {
        sg += s[2 * i];
        sx += s[2 * i + 1];
      }
    }
    const float mg = rms ? 0.0f : sg * inv, mx = sx * inv;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (i0 + j * G >= nv) continue;
#pragma unroll
      for (int k = 0; k < N; ++k) gr[j][k] = rt * (gr[j][k] - mg - xh[j][k] * mx);
      Row16<E>::store(dx, t * nv + i0 + j * G, gr[j]);
    }
  }
  if (!part) return;
  // The groups' column sums are added in group order. Element k of vector i is kept
  // at k * nv + i, so that a warp's accesses fall into different banks.
  float* out = part + static_cast<int64_t>(blockIdx.x) * 2 * H;
  for (int turn = 0; turn < groups; ++turn) {
    if (turn == g) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int i = i0 + j * G;
        if (i >= nv) continue;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          if (turn > 0) {
            aw[j][k] = col[0][k * nv + i] + aw[j][k];
            ab[j][k] = col[1][k * nv + i] + ab[j][k];
          }
          if (turn < groups - 1) {
            col[0][k * nv + i] = aw[j][k];
            col[1][k * nv + i] = ab[j][k];
          }
        }
        if (turn == groups - 1) {
#pragma unroll
          for (int k = 0; k < N; k += 4) {
            *reinterpret_cast<float4*>(out + i * N + k) = make_float4(aw[j][k], aw[j][k + 1], aw[j][k + 2], aw[j][k + 3]);
            *reinterpret_cast<float4*>(out + H + i * N + k) =
                make_float4(ab[j][k], ab[j][k + 1], ab[j][k + 2], ab[j][k + 3]);
          }
        }
      }
    }
    if (groups > 1) __syncthreads();
  }
}

// dw[i], db[i] (+)= the parts' sums: 32 columns a block, 16 threads a column that
// take every 16th part, then a fixed tree.
__global__ void __launch_bounds__(512)
    norm_sum_kernel(int H, int parts, int accumulate, const float* __restrict__ part, float* __restrict__ dw,
                    float* __restrict__ db) {
  __shared__ float sh[2][16][33];
  grid_dep_launch();
  grid_dep_wait();
  const int lane = static_cast<int>(threadIdx.x & 31), y = static_cast<int>(threadIdx.x >> 5);
  const int i = static_cast<int>(blockIdx.x) * 32 + lane;
  float a = 0.0f, b = 0.0f;
  if (i < H)
#pragma unroll 5
    for (int p = y; p < parts; p += 16) {
      a += part[static_cast<int64_t>(p) * 2 * H + i];
      b += part[(static_cast<int64_t>(p) * 2 + 1) * H + i];
    }
  sh[0][y][lane] = a;
  sh[1][y][lane] = b;
  __syncthreads();
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    if (y < o) {
      sh[0][y][lane] += sh[0][y + o][lane];
      sh[1][y][lane] += sh[1][y + o][lane];
    }
    __syncthreads();
  }
  if (y == 0 && i < H) {
    if (dw) dw[i] = accumulate ? dw[i] + sh[0][0][lane] : sh[0][0][lane];
    if (db) db[i] = accumulate ? db[i] + sh[1][0][lane] : sh[1][0][lane];
  }
}

// Rows too wide for registers (more than 4096 vectors forward, 1024 backward): one
// block a row that reads it again from L2, and the column sums by a thread a column.
__device__ __forceinline__ float load_f(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p, int64_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ void store_f(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store_f(__nv_bfloat16* p, int64_t i, float v) { p[i] = __float2bfloat16_rn(v); }

template <typename E>
__global__ void __launch_bounds__(kBwdThreads)
    norm_wide_fwd_kernel(int H, int rms, const E* __restrict__ x, const E* __restrict__ w, const E* __restrict__ b,
                         float eps, E* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ float sh[64];
  grid_dep_launch();
  grid_dep_wait();
  GroupSum sum{sh, kBwdThreads, 1, 0};
  const int64_t row = static_cast<int64_t>(blockIdx.x) * H;
  float mu = 0.0f, s = 0.0f;
  if (!rms) {
    for (int i = threadIdx.x; i < H; i += kBwdThreads) s += load_f(x, row + i);
    mu = sum(s) / static_cast<float>(H);
  }
  float q = 0.0f;
  for (int i = threadIdx.x; i < H; i += kBwdThreads) {
    const float d = load_f(x, row + i) - mu;
    q = fmaf(d, d, q);
  }
  const float r = 1.0f / sqrtf(sum(q) / static_cast<float>(H) + eps);
  for (int i = threadIdx.x; i < H; i += kBwdThreads) {
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
__global__ void __launch_bounds__(kBwdThreads)
    norm_wide_dx_kernel(int H, int rms, const E* __restrict__ x, const E* __restrict__ w, const D* __restrict__ dy,
                        const float* __restrict__ mean, const float* __restrict__ rstd, E* __restrict__ dx) {
  __shared__ float sh[64];
  grid_dep_launch();
  grid_dep_wait();
  GroupSum sum{sh, kBwdThreads, 1, 0};
  const int64_t row = static_cast<int64_t>(blockIdx.x) * H;
  const float mu = rms ? 0.0f : mean[blockIdx.x], r = rstd[blockIdx.x];
  float sg = 0.0f, sx = 0.0f;
  for (int i = threadIdx.x; i < H; i += kBwdThreads) {
    const float g = load_f(dy, row + i) * (w ? load_f(w, i) : 1.0f);
    sg += g;
    sx = fmaf(g, (load_f(x, row + i) - mu) * r, sx);
  }
  const float mg = rms ? 0.0f : sum(sg) / static_cast<float>(H);
  const float mx = sum(sx) / static_cast<float>(H);
  for (int i = threadIdx.x; i < H; i += kBwdThreads) {
    const float g = load_f(dy, row + i) * (w ? load_f(w, i) : 1.0f);
    store_f(dx, row + i, r * (g - mg - (load_f(x, row + i) - mu) * r * mx));
  }
}

template <typename E, typename D>
__global__ void __launch_bounds__(kFwdThreads)
    norm_wide_dw_kernel(int64_t T, int H, int rms, const E* __restrict__ x, const D* __restrict__ dy,
                        const float* __restrict__ mean, const float* __restrict__ rstd, float* __restrict__ part) {
  grid_dep_launch();
  grid_dep_wait();
  const int i = blockIdx.x * kFwdThreads + threadIdx.x;
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

// Threads per row: the least power of two that leaves at most `most` vectors a
// thread (up to `cap` threads).
int group_size(int64_t nv, int most, int cap) {
  int G = 32;
  while (G < cap && ceil_div(nv, G) > most) G *= 2;
  return G;
}

struct BwdShape {
  bool fused;
  int G, groups, vpt, parts;
};
BwdShape bwd_shape(const vce_problem& p) {
  BwdShape s{};
  const int64_t nv = p.H / (p.dtype == VCE_BF16 ? 8 : 4);
  const int sms = current_device_info().num_sms;
  s.fused = nv <= 2 * kBwdThreads;
  s.G = group_size(nv, 2, kBwdThreads);
  s.groups = kBwdThreads / s.G;
  s.vpt = nv <= s.G ? 1 : 2;
  const int64_t want = s.fused ? ceil_div(p.T, s.groups) : p.T;
  s.parts = static_cast<int>(want < sms ? want : sms);
  return s;
}

template <typename E>
cudaError_t fwd_typed(const vce_problem& p, bool rms, const void* x, const void* w, const void* b, float eps, void* y,
                      float* mean, float* rstd, cudaStream_t st) {
  const int64_t nv = p.H / Row16<E>::N;
  if (nv > 4096) {
    const cudaError_t e = launch_dependent(norm_wide_fwd_kernel<E>, dim3(static_cast<unsigned>(p.T)), dim3(kBwdThreads),
                                           0, st, static_cast<int>(p.H), rms ? 1 : 0, static_cast<const E*>(x),
                                           static_cast<const E*>(w), static_cast<const E*>(b), eps,
                                           static_cast<E*>(y), mean, rstd);
    note_launch(VCE_K_NORM_FWD, st);
    return e;
  }
  const int G = group_size(nv, 2, 1024);
  const int threads = G > kFwdThreads ? G : kFwdThreads, groups = threads / G;
  const int64_t want = ceil_div(p.T, groups);
  const int64_t cap = static_cast<int64_t>(current_device_info().num_sms) * (1024 / threads);   // resident at 64 registers
  const dim3 grid(static_cast<unsigned>(want < cap ? want : cap));
  const int64_t vpt = ceil_div(nv, G);
  auto go = [&](auto kern) {
    return launch_dependent(kern, grid, dim3(threads), 0, st, p.T, static_cast<int>(p.H), G, rms ? 1 : 0,
                            static_cast<const E*>(x), static_cast<const E*>(w), static_cast<const E*>(b), eps,
                            static_cast<E*>(y), mean, rstd);
  };
  const cudaError_t e = vpt <= 1   ? go(norm_fwd_kernel<E, 1>)
                        : vpt <= 2 ? go(norm_fwd_kernel<E, 2>)
                                   : go(norm_fwd_kernel<E, 4>);
  note_launch(VCE_K_NORM_FWD, st);
  return e;
}

template <typename E, typename D>
cudaError_t bwd_typed(const vce_problem& p, bool rms, const void* x_, const void* w_, const void* dy_,
                      const float* mean, const float* rstd, void* dx_, float* dw, float* db, bool accumulate,
                      float* part, cudaStream_t st) {
  const E* x = static_cast<const E*>(x_);
  const E* w = static_cast<const E*>(w_);
  const D* dy = static_cast<const D*>(dy_);
  E* dx = static_cast<E*>(dx_);
  const BwdShape s = bwd_shape(p);
  const int H = static_cast<int>(p.H);
  const bool sums = dw || db;
  cudaError_t e = cudaSuccess;
  if (s.fused) {
    auto go = [&](auto kern) {
      return launch_dependent(kern, dim3(static_cast<unsigned>(s.parts)), dim3(kBwdThreads), 0, st, p.T, H, s.G,
                              rms ? 1 : 0, x, w, dy, mean, rstd, dx, sums ? part : nullptr);
    };
    e = s.vpt == 1 ? go(norm_bwd_kernel<E, D, 1>) : go(norm_bwd_kernel<E, D, 2>);
    note_launch(VCE_K_NORM_BWD, st);
  } else {
    if (dx) {
      e = launch_dependent(norm_wide_dx_kernel<E, D>, dim3(static_cast<unsigned>(p.T)), dim3(kBwdThreads), 0, st, H,
                           rms ? 1 : 0, x, w, dy, mean, rstd, dx);
      note_launch(VCE_K_NORM_BWD, st);
    }
    if (e == cudaSuccess && sums) {
      e = launch_dependent(norm_wide_dw_kernel<E, D>,
                           dim3(static_cast<unsigned>(ceil_div(H, kFwdThreads)), static_cast<unsigned>(s.parts)),
                           dim3(kFwdThreads), 0, st, p.T, H, rms ? 1 : 0, x, dy, mean, rstd, part);
      note_launch(VCE_K_NORM_BWD, st);
    }
  }
  if (e != cudaSuccess || !sums) return e;
  e = launch_dependent(norm_sum_kernel, dim3(static_cast<unsigned>(ceil_div(H, 32))), dim3(512), 0, st, H, s.parts,
                       accumulate ? 1 : 0, static_cast<const float*>(part), dw, db);
  note_launch(VCE_K_NORM_SUM, st);
  return e;
}

}  // namespace

size_t norm_ws_bytes(const vce_problem& p) {
  return align_up(static_cast<size_t>(bwd_shape(p).parts) * 2 * static_cast<size_t>(p.H) * sizeof(float), kWsAlign);
}

cudaError_t launch_norm_fwd(const vce_problem& p, bool rms, const void* x, const void* w, const void* b, float eps,
                            void* y, float* mean, float* rstd, cudaStream_t st) {
  return p.dtype == VCE_BF16 ? fwd_typed<__nv_bfloat16>(p, rms, x, w, b, eps, y, mean, rstd, st)
                             : fwd_typed<float>(p, rms, x, w, b, eps, y, mean, rstd, st);
}

cudaError_t launch_norm_bwd(const vce_problem& p, bool rms, const void* x, const void* w, const void* dy, bool dy_bf16,
                            const float* mean, const float* rstd, void* dx, float* dw, float* db, bool accumulate,
                            void* ws, cudaStream_t st) {
  float* part = static_cast<float*>(ws);
  auto go = [&](auto f) { return f(p, rms, x, w, dy, mean, rstd, dx, dw, db, accumulate, part, st); };
  if (p.dtype == VCE_BF16)
    return dy_bf16 ? go(bwd_typed<__nv_bfloat16, __nv_bfloat16>) : go(bwd_typed<__nv_bfloat16, float>);
  return dy_bf16 ? go(bwd_typed<float, __nv_bfloat16>) : go(bwd_typed<float, float>);
}

}  // namespace vce
