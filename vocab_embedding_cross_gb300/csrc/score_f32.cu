// Token scores of fp32 problems, in fp32 FMA: the logits, their gradient and the
// gradient's two products are one tiled product kernel with four operand and
// epilogue forms,
//   LOGITS  Z  = h W^T
//   GRAD    G  = score gradient of (h W^T)
//   DH      dH = G W      (K, the classes, cut into parts where dH has few tiles)
//   DW      dW = G^T h    (rows of h without a real target read as zero)
// A block computes a 64 x 64 tile, 4 x 4 a thread, over slices of 32 along K; the
// next slice is fetched into registers while the current one is multiplied out of
// one of two shared-memory buffers. Small heads are bound by latency, so the
// parts of DH matter more than the inner loop: one 64 x 64 tile over K = 1000 as
// one block took 61 us. T = 64, H = 64, V = 1000: scores 13 us and gradient 20 us a
// call, launches and host included; T = 300, H = 512, V = 8000: gradient 267 us,
// 28 TFLOP/s of fp32 FMA, bound by shared-memory reads (two 16-byte loads for 16
// FMA). fp32 heads are kept for checks; the tensor cores have no fp32 form.
//
// The parts are joined, in a fixed order, by join_kernel, which also serves the
// tensor-core path's dH.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "internal.h"

namespace vce {
namespace {

constexpr int kTile = 64, kSlice = 32;
enum Form : int { LOGITS, GRAD, DH, DW };

struct F32Args {
  int M, N, K;
  const float* A;    // LOGITS, GRAD, DH: [M, K] row-major, lda; DW: [K, M] row-major, lda
  int64_t lda;
  const float* B;    // LOGITS, GRAD: [N, K] row-major, ldb; DH, DW: [K, N] row-major, ldb
  int64_t ldb;
  float* C;          // [M, N] row-major, ldc; DH: [parts][M][ldc]
  int64_t ldc;
  int add;           // C += instead of C =
  int m_tiles, k_part;   // K range of part z: [z k_part, (z + 1) k_part)
  const int64_t* targets;
  int V;             // classes; GRAD's columns start at class v0
  int v0;
  int64_t ignore_index;
  ScoreGrad sg;
  int32_t* status;
};

// Four neighbouring values along a row, zero past `n` of them.
__device__ __forceinline__ float4 row4(const float* p, int n) {
  if (n >= 4) return *reinterpret_cast<const float4*>(p);
  return make_float4(n > 0 ? p[0] : 0.0f, n > 1 ? p[1] : 0.0f, n > 2 ? p[2] : 0.0f, 0.0f);
}

template <int FORM>
__global__ void __launch_bounds__(256) f32_product_kernel(const F32Args a) {
  constexpr bool kATrans = FORM == DW;                       // A's tile comes along M
  constexpr bool kBTrans = FORM == LOGITS || FORM == GRAD;   // B's tile comes along K
  __shared__ float As[2][kSlice][kTile + 4];
  __shared__ float Bs[2][kSlice][kTile + 4];
  grid_dep_launch();
  grid_dep_wait();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int m0 = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.m_tiles)) * kTile;
  const int n0 = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.m_tiles)) * kTile;
  const int kb = static_cast<int>(blockIdx.z) * a.k_part;
  const int ke = kb + a.k_part < a.K ? kb + a.k_part : a.K;
  // Two quadruples of each operand a thread. Along K: rows tid / 8 and 32 on, four K
  // from 4 (tid % 8). Along M or N: K rows tid / 16 and 16 on, four columns from 4 (tid % 16).
  const int kr = tid >> 3, kc = (tid & 7) * 4, cr = tid >> 4, cc = (tid & 15) * 4;
  float4 fa[2], fb[2];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int r = kr + 32 * q, k = k0 + cr + 16 * q;
      if (kATrans)
        fa[q] = k < ke ? row4(a.A + k * a.lda + m0 + cc, a.M - m0 - cc) : make_float4(0, 0, 0, 0);
      else
        fa[q] = m0 + r < a.M ? row4(a.A + (m0 + r) * a.lda + k0 + kc, ke - k0 - kc) : make_float4(0, 0, 0, 0);
      if (kBTrans) {
        fb[q] = n0 + r < a.N ? row4(a.B + (n0 + r) * a.ldb + k0 + kc, ke - k0 - kc) : make_float4(0, 0, 0, 0);
      } else {
        bool take = k < ke;
        if (FORM == DW && take && a.targets) {   // a row of h takes part if its token does
          const int64_t y = a.targets[k];
          take = y >= 0 && y < a.V;
        }
        fb[q] = take ? row4(a.B + k * a.ldb + n0 + cc, a.N - n0 - cc) : make_float4(0, 0, 0, 0);
      }
    }
  };
  auto keep = [&](int buf) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float va[4] = {fa[q].x, fa[q].y, fa[q].z, fa[q].w}, vb[4] = {fb[q].x, fb[q].y, fb[q].z, fb[q].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (kATrans)
          As[buf][cr + 16 * q][cc + j] = va[j];
        else
          As[buf][kc + j][kr + 32 * q] = va[j];
        if (kBTrans)
          Bs[buf][kc + j][kr + 32 * q] = vb[j];
        else
          Bs[buf][cr + 16 * q][cc + j] = vb[j];
      }
    }
  };
  float acc[4][4] = {};
  fetch(kb);
  keep(0);
  __syncthreads();
  for (int k0 = kb, buf = 0; k0 < ke; k0 += kSlice, buf ^= 1) {
    const bool more = k0 + kSlice < ke;
    if (more) fetch(k0 + kSlice);
#pragma unroll
    for (int k = 0; k < kSlice; ++k) {
      const float4 x = *reinterpret_cast<const float4*>(&As[buf][k][4 * ty]);
      const float4 y = *reinterpret_cast<const float4*>(&Bs[buf][k][4 * tx]);
      const float xv[4] = {x.x, x.y, x.z, x.w}, yv[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xv[i], yv[j], acc[i][j]);
    }
    if (more) keep(buf ^ 1);
    __syncthreads();
  }
  float* C = a.C + (FORM == DH ? static_cast<int64_t>(blockIdx.z) * a.M * a.ldc : 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + 4 * ty + i;
    if (m >= a.M) continue;
    if constexpr (FORM == GRAD) {
      const int64_t y = a.targets ? a.targets[m] : -1;
      const bool valid = a.targets ? (y >= 0 && y < a.V) : true;
      if (tx == 0 && n0 == 0 && !valid && y != a.ignore_index && a.status)
        atomicCAS(a.status, 0, static_cast<int>(VCE_ERR_BAD_INDEX));
      const float lse = a.sg.lse[m];
      const float gl = a.sg.g_logp ? a.sg.g_logp[m] : 0.0f;
      const float ge = a.sg.g_entropy ? a.sg.g_entropy[m] : 0.0f;
      const float ent = a.sg.g_entropy ? a.sg.entropy[m] : 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + 4 * tx + j;
        const float lp = fmaf(acc[i][j], a.sg.scale, -lse);
        const float p = expf(lp);
        const float f = fmaxf(lp + ent, -200.0f);   // p is 0 below: a logit of -inf gives 0
        const float g = a.sg.scale * (gl * ((a.v0 + n == y ? 1.0f : 0.0f) - p) - ge * p * f);
        acc[i][j] = valid ? g : 0.0f;
      }
    }
    float* c = C + m * a.ldc + n0 + 4 * tx;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n0 + 4 * tx + j < a.N) c[j] = a.add ? c[j] + acc[i][j] : acc[i][j];
  }
}

// out[t, i] (+)= before + the sum of the parts, rounded once. A block takes 32
// quadruples of columns with eight threads each, which add every eighth part; their
// sums are added in order (one thread a quadruple took 13 us to add 76 parts).
// parts are P[part][rows][H], rows >= T; with lo4, each has a second summand that
// many quadruples further on (score_lo_rows).
constexpr int kJoinLanes = 8;
template <typename O>
__global__ void __launch_bounds__(32 * kJoinLanes)
    join_kernel(const float4* __restrict__ P, int64_t part4, int64_t lo4, int parts, const float4* __restrict__ before,
                int add, O* __restrict__ out, int64_t n4) {
  __shared__ float4 sh[kJoinLanes][32];
  grid_dep_launch();
  grid_dep_wait();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * 32; i0 < n4; i0 += static_cast<int64_t>(gridDim.x) * 32) {
    const int64_t i = i0 + x;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i < n4) {
#pragma unroll 4
      for (int p = y; p < parts; p += kJoinLanes) {
        float4 v = P[p * part4 + i];
        if (lo4) {
          const float4 l = P[p * part4 + lo4 + i];
          v = make_float4(v.x + l.x, v.y + l.y, v.z + l.z, v.w + l.w);
        }
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
      }
    }
    sh[y][x] = a;
    __syncthreads();
    if (y == 0 && i < n4) {
#pragma unroll
      for (int o = 1; o < kJoinLanes; ++o) {
        const float4 v = sh[o][x];
        a = make_float4(a.x + v.x, a.y + v.y, a.z + v.z, a.w + v.w);
      }
      if (before) {
        const float4 v = before[i];
        a = make_float4(v.x + a.x, v.y + a.y, v.z + a.z, v.w + a.w);
      }
      if constexpr (sizeof(O) == 16) {
        if (add) {
          const float4 o = out[i];
          a = make_float4(o.x + a.x, o.y + a.y, o.z + a.z, o.w + a.w);
        }
        out[i] = a;
      } else {
        if (add) {
          const uint2 o = out[i];
          a.x += __uint_as_float(o.x << 16);
          a.y += __uint_as_float(o.x & 0xFFFF0000u);
          a.z += __uint_as_float(o.y << 16);
          a.w += __uint_as_float(o.y & 0xFFFF0000u);
        }
        const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x, a.y), hi = __floats2bfloat162_rn(a.z, a.w);
        out[i] = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      }
    }
    __syncthreads();
  }
}

template <int FORM>
cudaError_t launch_form(F32Args a, int parts, int kind, cudaStream_t st) {
  a.m_tiles = static_cast<int>(ceil_div(a.M, kTile));
  a.k_part = static_cast<int>(ceil_div(ceil_div(a.K, kSlice), parts) * kSlice);
  const int64_t tiles = static_cast<int64_t>(a.m_tiles) * ceil_div(a.N, kTile);
  const cudaError_t e = launch_dependent(f32_product_kernel<FORM>,
                                         dim3(static_cast<unsigned>(tiles), 1, static_cast<unsigned>(parts)), dim3(256),
                                         0, st, a);
  note_launch(kind, st);
  return e;
}

}  // namespace

// One wave of two blocks an SM, a part being two slices at the least.
int f32_dh_parts(int64_t T, int64_t H, int64_t K) {
  const int64_t tiles = ceil_div(T, kTile) * ceil_div(H, kTile);
  int64_t parts = 2 * static_cast<int64_t>(current_device_info().num_sms) / (tiles > 0 ? tiles : 1);
  const int64_t most = ceil_div(K, 2 * kSlice);
  if (parts > most) parts = most;
  if (parts < 1) parts = 1;
  // no part empty
  const int64_t per = ceil_div(ceil_div(K, kSlice), parts);
  return static_cast<int>(ceil_div(ceil_div(K, kSlice), per));
}

cudaError_t launch_f32_logits(const ProbDev& pd, const float* h, const float* W, float* Z, int64_t ldz,
                              cudaStream_t st) {
  F32Args a{};
  a.M = pd.T;
  a.N = pd.V_real;
  a.K = pd.H;
  a.A = h;
  a.lda = pd.H;
  a.B = W;
  a.ldb = pd.H;
  a.C = Z;
  a.ldc = ldz;
  return launch_form<LOGITS>(a, 1, VCE_K_SIMT_LOGITS, st);
}

cudaError_t launch_f32_score_bwd(const ProbDev& pd, const float* h, const float* W, const int64_t* targets,
                                 const ScoreGrad& sg, int v0, int vc, float* G, int64_t ldg, float* P, int parts,
                                 float* dH, bool dH_add, float* dW, bool dW_add, int32_t* status, cudaStream_t st) {
  F32Args a{};
  a.targets = targets;
  a.V = pd.V_real;
  a.v0 = v0;
  a.ignore_index = pd.ignore_index;
  a.sg = sg;
  a.status = status;
  a.M = pd.T;
  a.N = vc;
  a.K = pd.H;
  a.A = h;
  a.lda = pd.H;
  a.B = W + static_cast<int64_t>(v0) * pd.H;
  a.ldb = pd.H;
  a.C = G;
  a.ldc = ldg;
  if (cudaError_t e = launch_form<GRAD>(a, 1, VCE_K_SIMT_SCORE_GRAD, st)) return e;
  a.N = pd.H;
  a.K = vc;
  a.A = G;
  a.lda = ldg;
  a.C = parts > 1 ? P : dH;
  a.ldc = pd.H;
  a.add = parts > 1 ? 0 : dH_add;
  if (cudaError_t e = launch_form<DH>(a, parts, VCE_K_SGEMM, st)) return e;
  a.M = vc;
  a.K = pd.T;
  a.B = h;
  a.C = dW + static_cast<int64_t>(v0) * pd.H;
  a.add = dW_add;
  return launch_form<DW>(a, 1, VCE_K_SGEMM, st);
}

cudaError_t launch_join(const float* P, int64_t part_elems, int64_t lo_elems, int parts, const float* before, bool add,
                        void* out, bool out_bf16, int64_t n, cudaStream_t st) {
  const int64_t n4 = n / 4, want = ceil_div(n4, 32), cap = static_cast<int64_t>(current_device_info().num_sms) * 8;
  const dim3 grid(static_cast<unsigned>(want < cap ? want : cap));
  auto go = [&](auto kern, auto* to) {
    return launch_dependent(kern, grid, dim3(32 * kJoinLanes), 0, st, reinterpret_cast<const float4*>(P),
                            part_elems / 4, lo_elems / 4, parts, reinterpret_cast<const float4*>(before), add ? 1 : 0, to, n4);
  };
  const cudaError_t e = out_bf16 ? go(join_kernel<uint2>, static_cast<uint2*>(out))
                                 : go(join_kernel<float4>, static_cast<float4*>(out));
  note_launch(VCE_K_DH_JOIN, st);
  return e;
}

}  // namespace vce
