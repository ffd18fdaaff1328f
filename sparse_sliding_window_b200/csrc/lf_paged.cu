// lf_paged.cu -- the decode step over the paged cache.
//
// o = softmax(scale q K^T) V over the newest token's window of its own rows
// and, when there is one, the prefix that every sequence of the batch shares:
//   * the prefix kernels take the queries of the whole batch as the rows of
//     one small attention per key/value head, so each prefix row is read once
//     for the batch; a chunk of the prefix leaves (sum of p v, max, sum of p)
//     of every row in the workspace;
//   * the decode kernel reads a sequence's own rows, adds the prefix partials
//     and writes o and lse.
// Scores are kept in base 2 (scale * log2 e), sums and maxima in float32.
#include <cooperative_groups.h>
#include <math.h>

#include "lf_paged.cuh"

namespace cg = cooperative_groups;

__device__ __forceinline__ float lf_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^(m - M), 0 for an empty part (m = -inf), also when everything is empty
__device__ __forceinline__ float lf_part_scale(float m, float M) {
  return m == -INFINITY ? 0.f : lf_exp2(m - M);
}

// ============================================================ decode kernel

#define LF_PD_WARPS 4
#define LF_PD_LOADS 8  // rows a lane loads per batch

// One cluster of CTAs of 4 warps per (sequence, key/value head, group of GT
// query heads); warps take batches of keys in turn.  A row is read by 64/N
// lanes, 16 bytes each, so a warp has BATCH = 8 * 32 / (64/N) rows of K and V
// in flight.  Every sub-warp of 64/N lanes keeps its own running maximum, sum
// and output for the rows it reads; they are merged once, at the end, through
// registers, shared memory and distributed shared memory.
template <typename T, int GT>
__global__ void __launch_bounds__(LF_PD_WARPS * 32)
    lf_paged_decode_kernel(const __grid_constant__ LfPagedDev P, const T *__restrict__ q,
                           const T *__restrict__ kp, const T *__restrict__ vp, T *__restrict__ o,
                           float *__restrict__ lse, int ngroups, int cl) {
  constexpr int N = LfVec<T>::N;
  constexpr int LPR = LF_HD / N;        // lanes per row
  constexpr int SUB = 32 / LPR;         // rows per warp load
  constexpr int BATCH = SUB * LF_PD_LOADS;
  __shared__ float s_m[LF_PD_WARPS][GT], s_l[LF_PD_WARPS][GT], s_acc[LF_PD_WARPS][GT][LF_HD];
  extern __shared__ float s_cl[];  // CTA 0 of a cluster: [cl][GT] m, l and [cl][GT][64]
  const bool prefix = P.prefix_len > 0;
  // Behind a prefix kernel the call's inputs are already complete: every block
  // of that kernel waited for its own predecessors before it let this one start.
  if (!prefix) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  cg::cluster_group cluster = cg::this_cluster();
  const int crank = cl > 1 ? (int)cluster.block_rank() : 0;
  if (cl > 1) cluster.barrier_arrive();
  const int unit = (int)blockIdx.x / cl;
  const int gc = unit % ngroups, hk = unit / ngroups % P.Hkv, b = unit / ngroups / P.Hkv;
  const int g0 = gc * GT, gn = min(GT, P.G - g0);  // query heads of this unit
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / LPR, lr = lane % LPR;
  const int len = P.lengths[b];
  const bool ok = lf_len_ok(len, P.max_pages, P.shift);
  if (!ok && threadIdx.x == 0 && crank == 0) lf_set_status(P.status, LF_ERR_DEVICE_INPUT, LF_DET_LENGTH + b);
  const int d = P.dil[hk];
  const int nk = ok ? lf_window_keys(len, P.window, d) : 0;
  const int32_t *table = P.table + (size_t)b * P.max_pages;

  float qf[GT][N], acc[GT][N], m[GT], l[GT];
#pragma unroll
  for (int g = 0; g < GT; g++) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int j = 0; j < N; j++) qf[g][j] = acc[g][j] = 0.f;
    if (g < gn && nk > 0) {
      LfVec<T>::ld(q + b * P.qs[0] + (hk * P.G + g0 + g) * P.qs[1] + lr * N, qf[g]);
#pragma unroll
      for (int j = 0; j < N; j++) qf[g][j] *= P.scale_log2;
    }
  }

  const int step = cl * LF_PD_WARPS * BATCH;
  int k0 = (crank * LF_PD_WARPS + warp) * BATCH;
  // lane i holds the pool row of key k0 + i of the batch (the next batch's is
  // fetched while this one is worked on)
  int mine = LF_ROW_NONE;
  if (lane < BATCH && k0 + lane < nk)
    mine = lf_pool_row(table, P.max_pages, P.num_pages, P.shift, P.Hkv, hk, len - 1 - (k0 + lane) * d);
  for (; k0 < nk; k0 += step) {
    if (mine == LF_ROW_BAD) lf_set_status(P.status, LF_ERR_DEVICE_INPUT, LF_DET_PAGE + b);
    uint4 kr[LF_PD_LOADS], vr[LF_PD_LOADS];
    uint32_t have = 0;
#pragma unroll
    for (int i = 0; i < LF_PD_LOADS; i++) {
      const int row = __shfl_sync(0xffffffffu, mine, i * SUB + sub);
      if (row >= 0) have |= 1u << i;
      kr[i] = row >= 0 ? *reinterpret_cast<const uint4 *>(kp + (size_t)row * LF_HD + lr * N) : uint4{0, 0, 0, 0};
      vr[i] = row >= 0 ? *reinterpret_cast<const uint4 *>(vp + (size_t)row * LF_HD + lr * N) : uint4{0, 0, 0, 0};
    }
    const int kn = k0 + step + lane;
    mine = LF_ROW_NONE;
    if (lane < BATCH && kn < nk)
      mine = lf_pool_row(table, P.max_pages, P.num_pages, P.shift, P.Hkv, hk, len - 1 - kn * d);
    float s[GT][LF_PD_LOADS];
#pragma unroll
    for (int i = 0; i < LF_PD_LOADS; i++) {
      float x[N];
      LfVec<T>::ld(reinterpret_cast<const T *>(&kr[i]), x);
#pragma unroll
      for (int g = 0; g < GT; g++) {
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < N; j++) a = fmaf(qf[g][j], x[j], a);
#pragma unroll
        for (int w = LPR / 2; w > 0; w >>= 1) a += __shfl_xor_sync(0xffffffffu, a, w);
        s[g][i] = (have >> i & 1) ? a : -INFINITY;
      }
    }
#pragma unroll
    for (int g = 0; g < GT; g++) {
      float M = m[g];
#pragma unroll
      for (int i = 0; i < LF_PD_LOADS; i++) M = fmaxf(M, s[g][i]);
      const float f = lf_part_scale(m[g], M);
      m[g] = M;
      l[g] *= f;
#pragma unroll
      for (int j = 0; j < N; j++) acc[g][j] *= f;
#pragma unroll
      for (int i = 0; i < LF_PD_LOADS; i++) {
        s[g][i] = (have >> i & 1) ? lf_exp2(s[g][i] - M) : 0.f;
        l[g] += s[g][i];
      }
    }
#pragma unroll
    for (int i = 0; i < LF_PD_LOADS; i++) {
      float x[N];
      LfVec<T>::ld(reinterpret_cast<const T *>(&vr[i]), x);
#pragma unroll
      for (int g = 0; g < GT; g++)
#pragma unroll
        for (int j = 0; j < N; j++) acc[g][j] = fmaf(s[g][i], x[j], acc[g][j]);
    }
  }

  if (prefix) {
    // the prefix partials, one chunk per sub-warp at a time
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (ok) {
      const size_t rows = (size_t)hk * P.B * P.G + (size_t)b * P.G + g0;
      for (int c = (crank * LF_PD_WARPS + warp) * SUB + sub; c < P.nch; c += cl * LF_PD_WARPS * SUB) {
#pragma unroll
        for (int g = 0; g < GT; g++) {
          if (g >= gn) continue;
          const size_t at = (rows + g) * P.nch + c;
          const float2 ml = P.part_ml[at];
          float a[N];
#pragma unroll
          for (int j = 0; j < N; j += 4)
            *reinterpret_cast<float4 *>(a + j) = *reinterpret_cast<const float4 *>(P.part_acc + at * LF_HD + lr * N + j);
          if (ml.x == -INFINITY) continue;
          const float M = fmaxf(m[g], ml.x);
          const float f = lf_part_scale(m[g], M), e = lf_exp2(ml.x - M);
          m[g] = M;
          l[g] = l[g] * f + ml.y * e;
#pragma unroll
          for (int j = 0; j < N; j++) acc[g][j] = acc[g][j] * f + a[j] * e;
        }
      }
    }
  }

  // merge: sub-warps, warps, CTAs
#pragma unroll
  for (int g = 0; g < GT; g++) {
#pragma unroll
    for (int w = LPR; w < 32; w <<= 1) {
      const float om = __shfl_xor_sync(0xffffffffu, m[g], w), ol = __shfl_xor_sync(0xffffffffu, l[g], w);
      const float M = fmaxf(m[g], om);
      const float f = lf_part_scale(m[g], M), e = lf_part_scale(om, M);
      m[g] = M;
      l[g] = l[g] * f + ol * e;
#pragma unroll
      for (int j = 0; j < N; j++) {
        const float oa = __shfl_xor_sync(0xffffffffu, acc[g][j], w);
        acc[g][j] = acc[g][j] * f + oa * e;
      }
    }
    if (lane == 0) {
      s_m[warp][g] = m[g];
      s_l[warp][g] = l[g];
    }
    if (sub == 0)
#pragma unroll
      for (int j = 0; j < N; j++) s_acc[warp][g][lr * N + j] = acc[g][j];
  }
  __syncthreads();
  if (cl > 1) cluster.barrier_wait();  // every CTA of the cluster runs
  float *c_m = s_cl, *c_l = s_cl + cl * GT, *c_acc = s_cl + 2 * cl * GT;
  float *r_m = nullptr, *r_l = nullptr, *r_acc = nullptr;
  if (cl > 1) {
    r_m = cluster.map_shared_rank(c_m, 0);
    r_l = cluster.map_shared_rank(c_l, 0);
    r_acc = cluster.map_shared_rank(c_acc, 0);
  }
  const size_t obase = ((size_t)b * P.H + hk * P.G + g0) * LF_HD;
  const size_t lbase = (size_t)b * P.H + hk * P.G + g0;
  for (int e = threadIdx.x; e < GT * LF_HD; e += LF_PD_WARPS * 32) {
    const int g = e / LF_HD, c = e % LF_HD;
    float M = -INFINITY, L = 0.f, a = 0.f;
#pragma unroll
    for (int w = 0; w < LF_PD_WARPS; w++) M = fmaxf(M, s_m[w][g]);
#pragma unroll
    for (int w = 0; w < LF_PD_WARPS; w++) {
      const float f = lf_part_scale(s_m[w][g], M);
      L += s_l[w][g] * f;
      a += s_acc[w][g][c] * f;
    }
    if (cl > 1) {
      r_acc[(crank * GT + g) * LF_HD + c] = a;
      if (c == 0) {
        r_m[crank * GT + g] = M;
        r_l[crank * GT + g] = L;
      }
    } else if (g < gn) {
      const bool none = M == -INFINITY;
      LfIo1<T>::st(o + obase + e, none ? 0.f : a / L);
      if (lse && c == 0) lse[lbase + g] = none ? -INFINITY : (M + log2f(L)) * LF_LN2;
    }
  }
  if (cl == 1) return;
  cluster.sync();  // the partials are in CTA 0
  if (crank != 0) return;
  for (int e = threadIdx.x; e < gn * LF_HD; e += LF_PD_WARPS * 32) {
    const int g = e / LF_HD, c = e % LF_HD;
    float M = -INFINITY, L = 0.f, a = 0.f;
    for (int r = 0; r < cl; r++) M = fmaxf(M, c_m[r * GT + g]);
    for (int r = 0; r < cl; r++) {
      const float f = lf_part_scale(c_m[r * GT + g], M);
      L += c_l[r * GT + g] * f;
      a += c_acc[(r * GT + g) * LF_HD + c] * f;
    }
    const bool none = M == -INFINITY;
    LfIo1<T>::st(o + obase + e, none ? 0.f : a / L);
    if (lse && c == 0) lse[lbase + g] = none ? -INFINITY : (M + log2f(L)) * LF_LN2;
  }
}

static cudaLaunchAttribute lf_pdl_attr() {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

template <typename T, int GT>
static cudaError_t lf_launch_pd_g(const LfPagedLaunch &L, const void *q, const void *kp,
                                  const void *vp, void *o, float *lse) {
  const LfPagedDev &P = L.dev;
  constexpr int BATCH = 32 / (LF_HD / LfVec<T>::N) * LF_PD_LOADS;
  const int ngroups = (P.G + GT - 1) / GT;
  const int64_t units = (int64_t)P.B * P.Hkv * ngroups;
  // CTAs per unit: enough for four per SM, at most as many as the longest
  // possible window has work for, and 8 (the portable cluster size)
  const int64_t cap = (int64_t)P.max_pages << P.shift;
  const int64_t keys = P.window < 0 || P.window >= cap ? cap : P.window + 1;
  const int64_t work = (keys + BATCH * LF_PD_WARPS - 1) / (BATCH * LF_PD_WARPS);
  int cl = 1;
  while (cl < 8 && units * cl < 4 * lf_sm_count() && cl < work) cl *= 2;
  if (units * cl > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * cl));
  cfg.blockDim = dim3(LF_PD_WARPS * 32);
  cfg.dynamicSmemBytes = cl > 1 ? (size_t)cl * GT * (LF_HD + 2) * 4 : 0;
  cfg.stream = L.stream;
  cudaLaunchAttribute attr[2];
  attr[0] = lf_pdl_attr();
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cl;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cl > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, lf_paged_decode_kernel<T, GT>, P, (const T *)q, (const T *)kp,
                            (const T *)vp, (T *)o, lse, ngroups, cl);
}

template <typename T>
static cudaError_t lf_launch_pd_t(const LfPagedLaunch &L, const void *q, const void *kp,
                                  const void *vp, void *o, float *lse) {
  switch (L.dev.G) {
    case 1: return lf_launch_pd_g<T, 1>(L, q, kp, vp, o, lse);
    case 2: return lf_launch_pd_g<T, 2>(L, q, kp, vp, o, lse);
    default: return lf_launch_pd_g<T, 4>(L, q, kp, vp, o, lse);
  }
}

cudaError_t lf_launch_paged_decode(const LfPagedLaunch &L, const void *q, const void *kp,
                                   const void *vp, void *o, float *lse) {
  cudaError_t e;
  switch (L.dtype) {
    case LF_F32: e = lf_launch_pd_t<float>(L, q, kp, vp, o, lse); break;
    case LF_BF16: e = lf_launch_pd_t<__nv_bfloat16>(L, q, kp, vp, o, lse); break;
    default: e = lf_launch_pd_t<__half>(L, q, kp, vp, o, lse);
  }
  if (e == cudaSuccess) lf_launches_add(1);
  return e;
}
