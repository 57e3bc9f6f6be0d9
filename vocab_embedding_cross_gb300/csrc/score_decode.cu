// Token scores of a few tokens (a decoding step): one pass over W.
//
// With few tokens the head's product is bound by reading W once, so the roles
// of the operands are turned round: W's rows are the MMA's M side and the
// tokens its N side (16, 32, 64 or 128 wide), D[v, t] = <W_v, h_t>. A 128-row
// tile then costs N/128 of a full-width one in tensor time, and no row of W is
// multiplied by padding tokens. Every CTA owns a contiguous range of classes,
// equal to within 16 rows whatever V is (a range's last tile is fetched in
// 16-row boxes), and streams it through a ring of 16 KB tiles: about 190 KB in
// flight on each SM, several times what hiding the memory latency at full
// bandwidth takes.
//
// Epilogue (TMEM lane = class, column = token): the logits go to the workspace
// in fp32 where alternatives are asked for (4 T bytes a class beside the 2 H
// that were read; they stay in L2), and each warp reduces its 32 classes of 16
// tokens at a time to their maximum, S and U by butterfly exchanges that leave
// token j's sums in lane j, where its running statistics are kept. The merge
// kernel joins the CTAs' statistics and takes the alternatives from the
// 32-class groups whose maximum can reach the K-th largest one.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"
#include "score.cuh"

namespace vce {
namespace {

constexpr int kRows = 128;                 // classes per tile (the MMA's M)
constexpr int kBlockK = 64;
constexpr int kBatch = 16;                 // tokens reduced at a time
constexpr uint32_t kWBytes = kRows * kBlockK * 2;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int N>
struct Dec {
  static constexpr int epi_warps = N <= 32 ? 4 : N / 8;   // each warp: 32 classes, at most 32 tokens
  static constexpr int threads = 64 + 32 * epi_warps;
  static constexpr int tokens = N <= 32 ? N : 32;         // per epilogue warp
  static constexpr uint32_t stage_bytes = kWBytes + N * kBlockK * 2;
  static constexpr int stages = static_cast<int>((208 * 1024) / stage_bytes);
  static constexpr uint32_t tmem_cols = 2 * N < 32 ? 32 : 2 * N;
  static constexpr size_t smem = 1024 + static_cast<size_t>(stages) * stage_bytes + 512;
  static constexpr uint32_t idesc = idesc_bf16_f32(kRows, N, 0, 0);
};

struct DecArgs {
  int T, V, num_kb;
  int groups;          // 16-class groups of the vocabulary
  float scale;
  const int64_t* targets;
  float* Z;            // [T, ldz] logits, or null
  int64_t ldz;
  uint32_t* gmax;      // [T, n_cta * gpc] ordered maxima of 32-class groups, or null
  int gpc;
  float4* part;        // [T, n_cta * 4] (m, S, U)
  float* ztgt;         // [T] target logits, written by the class's owner
  int32_t* status;
  uint64_t limit_ns;
};

__host__ __device__ __forceinline__ int dec_row0(int groups, int n_cta, int cta) {
  return static_cast<int>(static_cast<int64_t>(groups) * cta / n_cta) * 16;
}

// Sums (or maxima) of v[0..15] over the warp: lane l ends with that of v[l & 15].
template <bool MAX>
__device__ __forceinline__ float butterfly16(float (&v)[kBatch], int lane) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float keep = up ? v[i + o] : v[i], send = up ? v[i] : v[i + o];
      const float got = __shfl_xor_sync(0xffffffffu, send, o);
      v[i] = MAX ? fmaxf(keep, got) : keep + got;
    }
  }
  const float got = __shfl_xor_sync(0xffffffffu, v[0], 16);
  return MAX ? fmaxf(v[0], got) : v[0] + got;
}

__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

template <int N>
__global__ void __launch_bounds__(Dec<N>::threads, 1)
    score_decode_kernel(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapW16,
                        const __grid_constant__ CUtensorMap mapH, const DecArgs a) {
  using D = Dec<N>;
  constexpr int kStages = D::stages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* tail = smem_raw + (base - raw) + kStages * D::stage_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(tail);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drain + 1);
  int* s_abort = reinterpret_cast<int*>(s_tmem + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x, n_cta = gridDim.x;
  grid_dep_launch();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tfull[s], 1);
      mbar_init(&tempty[s], D::epi_warps);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, D::tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const WaitCtx wc{s_abort, a.status, a.limit_ns};
  const int row_lo = dec_row0(a.groups, n_cta, cta), row_hi = dec_row0(a.groups, n_cta, cta + 1);
  const int n_tiles = (row_hi - row_lo + kRows - 1) / kRows;
  grid_dep_wait();

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&mapW);
      tma_prefetch_desc(&mapW16);
      tma_prefetch_desc(&mapH);
      int stage = 0;
      uint32_t phase = 0;
      int last_parity[kStages];
#pragma unroll
      for (int s = 0; s < kStages; ++s) last_parity[s] = -1;
      bool ok = true, issued = false;
      for (int tt = 0; ok && tt < n_tiles; ++tt) {
        const int r0 = row_lo + tt * kRows;
        const int rows = row_hi - r0 < kRows ? row_hi - r0 : kRows;   // a multiple of 16
        for (int kb = 0; kb < a.num_kb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, wc)) {
            ok = false;
            break;
          }
          const uint32_t sW = base + static_cast<uint32_t>(stage) * D::stage_bytes;
          mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(rows) * 128u + N * 128u);
          if (rows == kRows)
            tma_load_2d(sW, &mapW, &full[stage], kb * kBlockK, r0);
          else
            for (int r = 0; r < rows; r += 16)
              tma_load_2d(sW + static_cast<uint32_t>(r) * 128u, &mapW16, &full[stage], kb * kBlockK, r0 + r);
          tma_load_2d(sW + kWBytes, &mapH, &full[stage], kb * kBlockK, 0);
          issued = true;
          last_parity[stage] = static_cast<int>(phase);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && issued) {   // let the copies already issued land
        const uint64_t t0 = globaltimer_ns();
#pragma unroll
        for (int s = 0; s < kStages; ++s) {
          if (last_parity[s] < 0) continue;
          while (!mbar_try_wait(&full[s], static_cast<uint32_t>(last_parity[s])) &&
                 globaltimer_ns() - t0 < 100000000ull) {
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true, issued = false;
      for (int tt = 0; ok && tt < n_tiles; ++tt) {
        const int acc = tt & 1;
        if (!mbar_wait(&tempty[acc], ((tt >> 1) & 1) ^ 1, wc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(acc * N);
        for (int kb = 0; kb < a.num_kb; ++kb) {
          if (!mbar_wait(&full[stage], phase, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sW = base + static_cast<uint32_t>(stage) * D::stage_bytes;
          const uint64_t ad = smem_desc_sw128(sW, 16u, 1024u), bd = smem_desc_sw128(sW + kWBytes, 16u, 1024u);
#pragma unroll
          for (int kk = 0; kk < kBlockK / 16; ++kk)
            umma_f16(d, ad + static_cast<uint64_t>(kk * 2), bd + static_cast<uint64_t>(kk * 2), D::idesc,
                     (kb != 0 || kk != 0) ? 1u : 0u);
          issued = true;
          umma_commit(&empty[stage]);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) umma_commit(&tfull[acc]);
      }
      if (!ok && issued) {   // wait for the MMAs in flight before TMEM is released
        umma_commit(drain);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < 100000000ull) {
        }
      }
    }
  } else {
    const int e = warp - 2;
    const int q = warp & 3;                  // TMEM lane quarter this warp may read
    const int tok0 = (e >> 2) * D::tokens;   // its first token
    constexpr int kB = D::tokens / kBatch;
    float m_run[kB], s_run[kB], u_run[kB];   // of token tok0 + 16 b + (lane & 15)
    int64_t y[kB];
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      m_run[b] = -INFINITY;
      s_run[b] = u_run[b] = 0.0f;
      const int t = tok0 + b * kBatch + (lane & 15);
      y[b] = (a.targets && t < a.T) ? a.targets[t] : -1;
    }
    const float sL = a.scale * kLog2e;
    for (int tt = 0; tt < n_tiles; ++tt) {
      const int acc = tt & 1;
      if (!mbar_wait(&tfull[acc], (tt >> 1) & 1, wc)) break;
      tc_fence_after();
      const int r0 = row_lo + tt * kRows + q * 32;      // first class of this warp's 32
      const int v = r0 + lane;
      const bool row_ok = v < row_hi && v < a.V;
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        const int t0 = tok0 + b * kBatch;
        uint32_t x[kBatch];
        tmem_ld_x16(tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * N + t0), x);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < kBatch; ++j) asm volatile("" : "+r"(x[j]));
        if (b == kB - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[acc]);
        }
        if (t0 >= a.T || r0 >= row_hi) continue;        // the same for the whole warp
        float mx[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) mx[j] = row_ok ? __uint_as_float(x[j]) : -INFINITY;
        if (a.Z && row_ok) {
#pragma unroll
          for (int j = 0; j < kBatch; ++j)
            if (t0 + j < a.T) a.Z[static_cast<int64_t>(t0 + j) * a.ldz + v] = __uint_as_float(x[j]);
        }
        const float gm = butterfly16<true>(mx, lane);   // of token t0 + (lane & 15)
        const int64_t off = y[b] - r0;                  // the target, if it is one of the warp's classes
        if (__any_sync(0xffffffffu, off >= 0 && off < 32)) {
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int at = static_cast<int>(__shfl_sync(0xffffffffu, off >= 0 && off < 32 ? static_cast<int>(off) : -1, j));
            if (at == lane && row_ok) a.ztgt[t0 + j] = __uint_as_float(x[j]);
          }
        }
        const float ref = gm == -INFINITY ? 0.0f : gm;  // no finite logit: exp(-inf) = 0 against any reference
        float ex[kBatch], ux[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const float d = (__uint_as_float(x[j]) - __shfl_sync(0xffffffffu, ref, j)) * sL;
          ex[j] = row_ok ? ex2_approx(d) : 0.0f;
          ux[j] = row_ok ? ex[j] * fmaxf(d, -300.0f) : 0.0f;   // 2^-300 is 0: keeps 0 * -inf out
        }
        const float S = butterfly16<false>(ex, lane), U = butterfly16<false>(ux, lane) * kLn2;
        const ScoreStat r = score_stat_join(ScoreStat{m_run[b], s_run[b], u_run[b]}, ScoreStat{gm * a.scale, S, U});
        m_run[b] = r.m;
        s_run[b] = r.S;
        u_run[b] = r.U;
        if (a.gmax && lane < kBatch && t0 + lane < a.T)
          a.gmax[static_cast<int64_t>(t0 + lane) * n_cta * a.gpc + static_cast<int64_t>(cta) * a.gpc + tt * 4 + q] =
              gm == gm ? ordered_bits(gm) : 0u;
      }
    }
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      const int t = tok0 + b * kBatch + lane;
      if (lane < kBatch && t < a.T)
        a.part[(static_cast<int64_t>(t) * n_cta + cta) * 4 + q] = make_float4(m_run[b], s_run[b], u_run[b], 0.0f);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, D::tmem_cols);
  }
}

constexpr int kMergeThreads = 256;
constexpr int kMergeCand = 1024;

// One block per token. A group of 32 classes with maximum g holds a key of at
// least (g, its last class), so the K-th largest such key over the threads'
// best groups bounds the K-th largest key of the row from below; only groups
// that reach (g, first class) >= the bound are read. Equal logits do not widen
// the choice: an all-equal row reads the first K groups.
__global__ void __launch_bounds__(kMergeThreads)
    score_merge_kernel(int V, int groups, int n_cta, int gpc, const float4* __restrict__ part,
                       const uint32_t* __restrict__ gmax, const float* __restrict__ Z, int64_t ldz,
                       const float* __restrict__ ztgt, const int64_t* __restrict__ targets, int64_t ignore_index,
                       float scale, int K, float* __restrict__ logp, float* __restrict__ entropy,
                       float* __restrict__ lse, int64_t* __restrict__ top_ids, float* __restrict__ top_logp,
                       int32_t* status) {
  __shared__ ScoreStat sstat[kMergeThreads / 32];
  __shared__ uint64_t skey[kMergeThreads];
  __shared__ uint64_t cand[kMergeCand];
  __shared__ uint64_t best[kMaxTop];
  __shared__ uint64_t s_bound;
  __shared__ int s_n;
  grid_dep_launch();
  grid_dep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t t = blockIdx.x;
  ScoreStat a = score_stat_empty();
  for (int i = tid; i < 4 * n_cta; i += kMergeThreads) {
    const float4 p = part[t * 4 * n_cta + i];
    a = score_stat_join(a, ScoreStat{p.x, p.y, p.z});
  }
  // Group i of CTA c starts at dec_row0(c) + 32 i; slots past the CTA's range are never written.
  uint64_t kmax = 0;
  const uint32_t* gm = K ? gmax + t * n_cta * gpc : nullptr;
  for (int i = tid; K && i < n_cta * gpc; i += kMergeThreads) {
    const int c = i / gpc, v0 = dec_row0(groups, n_cta, c) + (i - c * gpc) * 32;
    const int hi = min(dec_row0(groups, n_cta, c + 1), V);
    const uint32_t g = v0 < hi ? gm[i] : 0;
    if (g) {
      const uint64_t k = (static_cast<uint64_t>(g) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(min(v0 + 32, hi) - 1));
      kmax = k > kmax ? k : kmax;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ScoreStat b{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.S, o),
                __shfl_xor_sync(0xffffffffu, a.U, o)};
    a = (lane & o) == 0 ? score_stat_join(a, b) : score_stat_join(b, a);
  }
  if (lane == 0) sstat[warp] = a;
  skey[tid] = kmax;
  if (tid < K) best[tid] = 0;
  if (tid == 0) {
    s_n = 0;
    s_bound = 0;
  }
  __syncthreads();
  a = sstat[0];
  for (int w = 1; w < kMergeThreads / 32; ++w) a = score_stat_join(a, sstat[w]);
  const float l = score_lse(a);
  if (tid == 0) {
    if (lse) lse[t] = l;
    const int64_t y = targets ? targets[t] : -1;
    const bool valid = targets && y >= 0 && y < V;
    if (targets && !valid && y != ignore_index) atomicCAS(status, 0, static_cast<int>(VCE_ERR_BAD_INDEX));
    if (logp) logp[t] = valid ? fmaf(ztgt[t], scale, -l) : 0.0f;
    if (entropy) entropy[t] = (!targets || valid) ? score_entropy(a) : 0.0f;
  }
  if (K == 0) return;
  if (kmax) {
    int rank = 0;
    for (int i = 0; i < kMergeThreads; ++i) rank += skey[i] > kmax ? 1 : 0;
    if (rank == K - 1) s_bound = kmax;   // stays 0 when fewer than K threads hold a group
  }
  __syncthreads();
  const uint64_t bound = s_bound;
  const float* z = Z + t * ldz;
  for (int i = tid; i < n_cta * gpc; i += kMergeThreads) {
    const int c = i / gpc, v0 = dec_row0(groups, n_cta, c) + (i - c * gpc) * 32;
    const int hi = min(dec_row0(groups, n_cta, c + 1), V);
    const uint32_t g = v0 < hi ? gm[i] : 0;
    if (!g || ((static_cast<uint64_t>(g) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(v0))) < bound) continue;
    for (int v = v0; v < min(v0 + 32, hi); ++v) {
      const uint64_t k = top_key(z[v], static_cast<uint32_t>(v));
      if (k != 0 && k >= bound) {
        const int at = atomicAdd(&s_n, 1);
        if (at < kMergeCand) cand[at] = k;
      }
    }
  }
  __syncthreads();
  const int n = s_n;
  if (n <= kMergeCand) {
    for (int i = tid; i < n; i += kMergeThreads) {
      const uint64_t k = cand[i];
      int r = 0;
      for (int j = 0; j < n; ++j) r += cand[j] > k ? 1 : 0;
      if (r < K) best[r] = k;
    }
    __syncthreads();
  } else {
    // Over kMergeCand keys reach the bound (the largest logits all in a few
    // threads' groups): K scans, each for the largest key below the last.
    uint64_t below = ~uint64_t(0);
    for (int i = 0; i < K; ++i) {
      uint64_t k = 0;
      for (uint32_t v = tid; v < static_cast<uint32_t>(V); v += kMergeThreads) {
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
      for (int w = 1; w < kMergeThreads / 32; ++w) below = skey[w] > below ? skey[w] : below;
      if (tid == 0) best[i] = below;
    }
    __syncthreads();
  }
  if (tid < K) write_top(best[tid], t * K + tid, scale, l, top_ids, top_logp);
}

struct DecLayout {
  int n_cta, groups, gpc;
  size_t part, ztgt, gmax, Z, total;
};
DecLayout dec_layout(const vce_problem& p, int K) {
  DecLayout L{};
  L.groups = static_cast<int>(ceil_div(p.V_real, 16));
  const int sms = current_device_info().num_sms;
  L.n_cta = L.groups < sms ? L.groups : sms;
  // a range holds at most ceil(groups / n_cta) groups, in tiles of 8 of them
  L.gpc = static_cast<int>(ceil_div(ceil_div(L.groups, L.n_cta), 8)) * 4;
  size_t off = kWsAlign;   // status word
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, kWsAlign);
    return o;
  };
  const size_t T = static_cast<size_t>(p.T);
  L.part = take(T * 4 * L.n_cta * sizeof(float4));
  L.ztgt = take(T * sizeof(float));
  L.gmax = take(K ? T * L.n_cta * L.gpc * sizeof(uint32_t) : 0);
  L.Z = take(K ? T * static_cast<size_t>(p.Vp) * sizeof(float) : 0);
  L.total = off;
  return L;
}

template <int N>
cudaError_t launch_n(const vce_problem& p, const void* h, const void* W, const DecLayout& L, const DecArgs& a,
                     cudaStream_t st) {
  using D = Dec<N>;
  static std::atomic<uint64_t> configured{0};
  if (device_pending(configured)) {
    const cudaError_t e = cudaFuncSetAttribute(score_decode_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(D::smem));
    if (e != cudaSuccess) return e;
    mark_device_done(configured);
  }
  CUtensorMap mw, mw16, mh;
  const auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!make_tmap_2d(&mw, W, BF, 2, p.H, p.V_real, p.H, kBlockK, kRows, true) ||
      !make_tmap_2d(&mw16, W, BF, 2, p.H, p.V_real, p.H, kBlockK, 16, true) ||
      !make_tmap_2d(&mh, h, BF, 2, p.H, p.T, p.H, kBlockK, N, true))
    return cudaErrorInvalidValue;
  const cudaError_t e = launch_dependent(score_decode_kernel<N>, dim3(static_cast<unsigned>(L.n_cta)),
                                         dim3(D::threads), D::smem, st, mw, mw16, mh, a);
  note_launch(VCE_K_SCORE_DECODE, st);
  return e;
}

}  // namespace

size_t score_decode_ws_bytes(const vce_problem& p, int K) { return dec_layout(p, K).total; }

cudaError_t launch_score_decode(const vce_problem& p, const void* h, const void* W, const int64_t* targets,
                                float scale, int K, float* logp, float* entropy, float* lse, int64_t* top_ids,
                                float* top_logp, void* ws, int32_t* status, cudaStream_t st) {
  const DecLayout L = dec_layout(p, K);
  char* b = static_cast<char*>(ws);
  DecArgs a{};
  a.T = static_cast<int>(p.T);
  a.V = static_cast<int>(p.V_real);
  a.num_kb = static_cast<int>(ceil_div(p.H, kBlockK));
  a.groups = L.groups;
  a.scale = scale;
  a.targets = targets;
  a.Z = K ? reinterpret_cast<float*>(b + L.Z) : nullptr;
  a.ldz = p.Vp;
  a.gmax = K ? reinterpret_cast<uint32_t*>(b + L.gmax) : nullptr;
  a.gpc = L.gpc;
  a.part = reinterpret_cast<float4*>(b + L.part);
  a.ztgt = reinterpret_cast<float*>(b + L.ztgt);
  a.status = status;
  a.limit_ns = wait_limit_ns();
  cudaError_t e = p.T <= 16   ? launch_n<16>(p, h, W, L, a, st)
                  : p.T <= 32 ? launch_n<32>(p, h, W, L, a, st)
                  : p.T <= 64 ? launch_n<64>(p, h, W, L, a, st)
                              : launch_n<128>(p, h, W, L, a, st);
  if (e != cudaSuccess) return e;
  e = launch_dependent(score_merge_kernel, dim3(static_cast<unsigned>(p.T)), dim3(kMergeThreads), 0, st, a.V, L.groups,
                       L.n_cta, L.gpc, static_cast<const float4*>(a.part), static_cast<const uint32_t*>(a.gmax),
                       static_cast<const float*>(a.Z), a.ldz, static_cast<const float*>(a.ztgt), targets,
                       p.ignore_index, scale, K, logp, entropy, lse, top_ids, top_logp, status);
  note_launch(VCE_K_SCORE_MERGE, st);
  return e;
}

}  // namespace vce
