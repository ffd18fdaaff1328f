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

#include "lf_paged_mma.cuh"

namespace cg = cooperative_groups;

// one element, rounded to nearest even
template <typename T> struct LfIo1;
template <> struct LfIo1<float> {
  static __device__ __forceinline__ void st(float *p, float a) { *p = a; }
};
template <> struct LfIo1<__nv_bfloat16> {
  static __device__ __forceinline__ void st(__nv_bfloat16 *p, float a) { *p = __float2bfloat16_rn(a); }
};
template <> struct LfIo1<__half> {
  static __device__ __forceinline__ void st(__half *p, float a) { *p = __float2half_rn(a); }
};

// Element (row g, channel c) of the newest token's output from its merged
// state: o = a / L, lse = log of the sum, 0 and -inf where nothing was attended.
template <typename T>
__device__ __forceinline__ void lf_pd_write(T *o, float *lse, size_t row, int c, float M, float L, float a) {
  const bool none = M == -INFINITY && L == 0.f;  // (a NaN query has L = NaN)
  LfIo1<T>::st(o + row * LF_HD + c, none ? 0.f : a / L);
  if (lse && c == 0) lse[row] = none ? -INFINITY : (M + log2f(L)) * LF_LN2;
}

// Before a decode kernel reads the call's inputs.  Behind a prefix kernel they
// are already complete: every block of that kernel waited for its own
// predecessors before it let this one start.  What those wrote is in L2, but the
// wait that would make it visible here comes only with the prefix's parts; the
// fence keeps loads behind it from hitting lines that L1 held before (and the
// inputs are not read through the read-only path).  Measured, nothing / fence /
// reads past L1 / waiting for the prefix kernel, in us: 64 x 12 heads on 4096
// rows 27.5 / 27.9 / 29.4 / 29.4, 128 x 16/4 heads on 16384 rows 43.0 / 43.4 /
// 45.1 / 46.4, f32 40 x 8 heads on 1000 rows 22.9 / 23.4 / 23.0 / 29.0.
__device__ __forceinline__ void lf_pd_begin(bool prefix) {
  if (prefix)
    asm volatile("fence.acq_rel.gpu;" ::: "memory");
  else
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ===================================================== decode kernel (f32)

#define LF_PD_WARPS 4
#define LF_PD_LOADS 8  // rows a lane loads per batch

// One cluster of CTAs of 4 warps per (sequence, key/value head, group of GT
// query heads); warps take batches of keys in turn.  A row is read by 64/N
// lanes, 16 bytes each, so a warp has BATCH = 8 * 32 / (64/N) rows of K and V
// in flight.  Every sub-warp of 64/N lanes keeps its own running maximum, sum
// and output for the rows it reads; they are merged once, at the end, through
// registers, shared memory and distributed shared memory.
template <int GT>
__global__ void __launch_bounds__(LF_PD_WARPS * 32)
    lf_paged_decode_kernel(const __grid_constant__ LfPagedDev P, const float *q, const float *kp, const float *vp,
                           float *o, float *lse, int ngroups, int cl) {
  constexpr int N = LfVec<float>::N;
  constexpr int LPR = LF_HD / N;        // lanes per row
  constexpr int SUB = 32 / LPR;         // rows per warp load
  constexpr int BATCH = SUB * LF_PD_LOADS;
  __shared__ float s_m[LF_PD_WARPS][GT], s_l[LF_PD_WARPS][GT], s_acc[LF_PD_WARPS][GT][LF_HD];
  extern __shared__ float s_cl[];  // CTA 0 of a cluster: [cl][GT] m, l and [cl][GT][64]
  const bool prefix = P.nch > 0;  // parts of a prefix kernel to add
  lf_pd_begin(prefix);
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
  const int own = ok ? lf_window_keys(len, P.window, d) : 0;
  const int nk = own + (ok && P.direct ? P.prefix_len : 0);
  const int32_t *table = P.table + (size_t)b * P.max_pages;
  const int pcols = (P.prefix_len + (1 << P.shift) - 1) >> P.shift;
  auto row_of = [&](int k) {  // pool row of key k: the window, then the prefix
    return k < own ? lf_pool_row(table, P.max_pages, P.num_pages, P.shift, P.Hkv, hk, len - 1 - k * d)
                   : lf_pool_row(P.prefix_table, pcols, P.num_pages, P.shift, P.Hkv, hk, k - own);
  };

  float qf[GT][N], acc[GT][N], m[GT], l[GT];
#pragma unroll
  for (int g = 0; g < GT; g++) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int j = 0; j < N; j++) qf[g][j] = acc[g][j] = 0.f;
    if (g < gn && nk > 0) {
      LfVec<float>::ld(q + b * P.qs[0] + (hk * P.G + g0 + g) * P.qs[1] + lr * N, qf[g]);
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
    mine = row_of(k0 + lane);
  for (; k0 < nk; k0 += step) {
    if (mine == LF_ROW_BAD) lf_set_status(P.status, LF_ERR_DEVICE_INPUT, k0 + lane < own ? LF_DET_PAGE + b : LF_DET_PREFIX);
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
      mine = row_of(kn);
    float s[GT][LF_PD_LOADS];
#pragma unroll
    for (int i = 0; i < LF_PD_LOADS; i++) {
      float x[N];
      LfVec<float>::ld(reinterpret_cast<const float *>(&kr[i]), x);
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
      const float e = M == -INFINITY ? 0.f : M;  // no key yet, or scores of -inf alone: p = 0
      m[g] = M;
      l[g] *= f;
#pragma unroll
      for (int j = 0; j < N; j++) acc[g][j] *= f;
#pragma unroll
      for (int i = 0; i < LF_PD_LOADS; i++) {
        s[g][i] = (have >> i & 1) ? lf_ex2(s[g][i] - e) : 0.f;
        l[g] += s[g][i];
      }
    }
#pragma unroll
    for (int i = 0; i < LF_PD_LOADS; i++) {
      float x[N];
      LfVec<float>::ld(reinterpret_cast<const float *>(&vr[i]), x);
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
          const float2 ml = __ldcg(P.part_ml + at);
          float a[N];
#pragma unroll
          for (int j = 0; j < N; j += 4)
            *reinterpret_cast<float4 *>(a + j) = __ldcg(reinterpret_cast<const float4 *>(P.part_acc + at * LF_HD + lr * N + j));
          const float M = fmaxf(m[g], ml.x);
          const float f = lf_part_scale(m[g], M), e = lf_part_scale(ml.x, M);
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
  const size_t orow = (size_t)b * P.H + hk * P.G + g0;
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
      lf_pd_write(o, lse, orow + g, c, M, L, a);
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
    lf_pd_write(o, lse, orow + g, c, M, L, a);
  }
}

// Keys of a sequence's own rows that a query can attend.
static int64_t lf_most_keys(const LfPagedDev &P) {
  const int64_t cap = (int64_t)P.max_pages << P.shift;
  return P.window < 0 || P.window >= cap ? cap : P.window + 1;
}

// Few units (sequence, key/value head): the decode kernel reads the prefix for
// every sequence itself, which saves a kernel and the merging of its parts.
// With up to 37 units (8 CTAs each, two per SM) the repeated reads come from L2
// and keep up to about here.  Measured, prefix kernel / direct, in us, on 300,
// 1000, 4096 and 8192 rows with a window of 64: bf16 1 x 8 heads 5.1 / 4.2, 5.1 /
// 5.0, 8.6 / 7.6, 13.4 / 10.7; 36 x 1 heads 7.1 / 4.9, 8.0 / 6.6, 12.5 / 11.3,
// 12.9 / 16.6; 2 x 32/4 heads 9.8 / 5.9, 9.2 / 6.9, 19.0 / 9.4, 32.5 / 12.6;
// f32 1 x 8 heads 7.9 / 4.0, 8.0 / 5.8, 20.0 / 11.6, 33.8 / 29.2; 36 x 1 heads
// 9.7 / 4.6, 9.8 / 6.6, 11.4 / 14.5, 15.5 / 24.8; 2 x 32/4 heads (four at a time,
// though counted by sixteen) 10.4 / 5.8, 10.5 / 8.9, 18.7 / 20.5, 25.4 / 36.0.
// The rule goes by the units and the prefix alone, and is off by up to a quarter
// where a few sequences of one query head per key/value head leave the prefix
// kernel many heads: bf16 4 x 8 heads 5.2 / 4.6, 5.1 / 6.6, 9.3 / 11.3, 14.0 / 16.6.
bool lf_prefix_direct(const LfPagedDev &P, int dtype) {
  const int64_t units = (int64_t)P.B * P.Hkv * ((P.G + 15) / 16);
  return units * 8 <= 2 * 148 && P.prefix_len <= (dtype == LF_F32 ? 4096 : 8192);
}

// CTAs per unit (sequence, key/value head, query-head group): enough for four
// per SM, at most as many as the longest possible window has steps of `step`
// keys, and `most` (a power of two, up to 8, the portable cluster size).
static int lf_pd_cluster(const LfPagedDev &P, int64_t units, int step, int most) {
  const int64_t keys = lf_most_keys(P) + (P.direct ? P.prefix_len : 0);
  const int64_t work = (keys + step - 1) / step;
  int cl = 1;
  while (cl < most && units * cl < 4 * lf_sm_count() && cl < work) cl *= 2;
  return cl;
}

static cudaError_t lf_pd_launch(const void *fn, const LfPagedLaunch &L, int64_t units, int cl, int smem,
                                const void *q, const void *kp, const void *vp, void *o, float *lse,
                                int ngroups) {
  if (units * cl > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * cl));
  cfg.blockDim = dim3(LF_PD_WARPS * 32);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = L.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cl;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cl > 1 ? 2 : 1;
  void *args[] = {const_cast<LfPagedDev *>(&L.dev), &q, &kp, &vp, &o, &lse, &ngroups, &cl};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

template <int GT>
static cudaError_t lf_launch_pd_f32(const LfPagedLaunch &L, const void *q, const void *kp,
                                    const void *vp, void *o, float *lse) {
  const LfPagedDev &P = L.dev;
  constexpr int BATCH = 32 / (LF_HD / LfVec<float>::N) * LF_PD_LOADS;
  const int ngroups = (P.G + GT - 1) / GT;
  const int64_t units = (int64_t)P.B * P.Hkv * ngroups;
  const int cl = lf_pd_cluster(P, units, BATCH * LF_PD_WARPS, 8);
  return lf_pd_launch((const void *)lf_paged_decode_kernel<GT>, L, units, cl,
                      cl > 1 ? cl * GT * (LF_HD + 2) * 4 : 0, q, kp, vp, o, lse, ngroups);
}

// Another part (its max, sum and output) into (M, L, a).
__device__ __forceinline__ void lf_pd_add(float m, float l, float v, float &M, float &L, float &a) {
  const float N = fmaxf(M, m);
  const float f = lf_part_scale(M, N), h = lf_part_scale(m, N);
  M = N;
  L = L * f + l * h;
  a = a * f + v * h;
}

// A fragments of the queries g0 .. g0 + gn - 1 of a key/value head's group;
// rows behind them repeat the last one and are not written.
template <typename T, int MT>
__device__ __forceinline__ void lf_pd_queries(const LfPagedDev &P, const T *q, int b, int hk, int g0, int gn,
                                              LfPmQ<MT> &qa) {
  const T *qb = q + b * P.qs[0] + (int64_t)(hk * P.G + g0) * P.qs[1];
  const int g = threadIdx.x % 32 / 4;
#pragma unroll
  for (int mt = 0; mt < MT; mt++)
    lf_pm_qfrag<T>(qb + min(16 * mt + g, gn - 1) * P.qs[1], qb + min(16 * mt + g + 8, gn - 1) * P.qs[1], qa[mt]);
}

// Parts first, first + step, ... that the prefix kernel left of a row.  The
// parts are read past L1 (here and below): an earlier call's may still be there.
__device__ __forceinline__ void lf_pd_prefix(const LfPagedDev &P, size_t row, int c, int first, int step,
                                             float &M, float &L, float &a) {
  const float2 *ml = P.part_ml + row * P.nch;
  const float *acc = P.part_acc + row * P.nch * LF_HD + c;
#pragma unroll 4
  for (int k = first; k < P.nch; k += step) {
    const float2 x = __ldcg(ml + k);
    lf_pd_add(x.x, x.y, __ldcg(acc + (size_t)k * LF_HD), M, L, a);
  }
}

// All parts of up to 16 rows, by a block of 128 threads: the weights of a
// row's parts first (8 lanes a row), then their weighted sum with 16 bytes a
// load and every load independent of the others; rows few enough leave
// several threads to an element, whose sums lf_pd_folded adds.  (One thread
// per element that added part after part took 8 us of the 26 us that the
// decode kernel needs behind a prefix with 22 parts for 64 sequences x 12
// heads.)
struct LfPdFold {
  float *w;    // [rows][nch]
  float2 *ml;  // [16]
  float *sum;  // [threads per element][rows][64]
};
__host__ __device__ __forceinline__ int lf_pd_fold_ways(int rows) { return rows == 1 ? 8 : rows == 2 ? 4 : rows <= 4 ? 2 : 1; }
__host__ __device__ __forceinline__ int lf_pd_fold_bytes(int rows, int nch) {  // multiple of 16
  return 16 * 8 + (rows * nch + 3) / 4 * 16 + (rows < 8 ? 8 : rows) * LF_HD * 4;
}
__device__ __forceinline__ LfPdFold lf_pd_fold_at(char *smem, int rows, int nch) {
  LfPdFold F;
  F.ml = reinterpret_cast<float2 *>(smem);
  F.w = reinterpret_cast<float *>(smem + 16 * 8);
  F.sum = F.w + (rows * nch + 3) / 4 * 4;
  return F;
}
__device__ __forceinline__ void lf_pd_fold(const LfPagedDev &P, size_t row0, int rows, const LfPdFold &F) {
  const int tid = threadIdx.x, nch = P.nch;
  {
    const int x = tid / 8, s = tid % 8;
    float2 v[LF_PART_MAX / 8];
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int i = 0; i < LF_PART_MAX / 8; i++) {
      const int k = s + 8 * i;
      v[i] = x < rows && k < nch ? __ldcg(P.part_ml + (row0 + x) * nch + k) : make_float2(-INFINITY, 0.f);
      M = fmaxf(M, v[i].x);
    }
#pragma unroll
    for (int w = 1; w < 8; w <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
#pragma unroll
    for (int i = 0; i < LF_PART_MAX / 8; i++) {
      const int k = s + 8 * i;
      const float f = lf_part_scale(v[i].x, M);
      L += v[i].y * f;
      if (x < rows && k < nch) F.w[x * nch + k] = f;
    }
#pragma unroll
    for (int w = 1; w < 8; w <<= 1) L += __shfl_xor_sync(0xffffffffu, L, w);
    if (s == 0 && x < rows) F.ml[x] = make_float2(M, L);
  }
  __syncthreads();
  const int ways = lf_pd_fold_ways(rows), c = tid % 16 * 4;
  for (int item = tid / 16; item < rows * ways; item += 8) {
    const int x = item % rows, sub = item / rows;
    const float *acc = P.part_acc + (row0 + x) * nch * LF_HD + c, *w = F.w + x * nch;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = sub; k < nch; k += ways) {
      const float4 v = __ldcg(reinterpret_cast<const float4 *>(acc + (size_t)k * LF_HD));
      a.x = fmaf(w[k], v.x, a.x);
      a.y = fmaf(w[k], v.y, a.y);
      a.z = fmaf(w[k], v.z, a.z);
      a.w = fmaf(w[k], v.w, a.w);
    }
    *reinterpret_cast<float4 *>(F.sum + (sub * rows + x) * LF_HD + c) = a;
  }
  __syncthreads();
}
// Channel c of row x of the fold, added to (M, L, a).
__device__ __forceinline__ void lf_pd_folded(const LfPdFold &F, int rows, int x, int c, float &M, float &L, float &a) {
  float v = 0.f;
  for (int sub = 0; sub < lf_pd_fold_ways(rows); sub++) v += F.sum[(sub * rows + x) * LF_HD + c];
  lf_pd_add(F.ml[x].x, F.ml[x].y, v, M, L, a);
}

// ============================= decode kernel (bf16, f16), few sequences

// One cluster of CTAs per (sequence, key/value head, group of 16 MT query
// heads); its CTAs take the window's tiles of 128 keys in turn, add a share of
// the prefix partials each, and merge through CTA 0's shared memory.
template <typename T, int MT>
__global__ void __launch_bounds__(128, 2)
    lf_paged_mma_kernel(const __grid_constant__ LfPagedDev P, const T *q, const T *kp, const T *vp, T *o,
                        float *lse, int ngroups, int cl) {
  constexpr int RB = 16 * MT;
  extern __shared__ __align__(16) char smem_raw[];
  __shared__ float s_m[4][16], s_l[4][16];
  const bool prefix = P.nch > 0;  // parts of a prefix kernel to add
  lf_pd_begin(prefix);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  cg::cluster_group cluster = cg::this_cluster();
  const int crank = cl > 1 ? (int)cluster.block_rank() : 0;
  const int unit = (int)blockIdx.x / cl;
  const int gc = unit % ngroups, hk = unit / ngroups % P.Hkv, b = unit / ngroups / P.Hkv;
  const int g0 = gc * RB, gn = min(RB, P.G - g0);  // query heads of this unit
  const int len = P.lengths[b];
  LfPmQ<MT> qa;  // on their way with the length
  lf_pd_queries<T, MT>(P, q, b, hk, g0, gn, qa);
  const bool ok = lf_len_ok(len, P.max_pages, P.shift);
  if (!ok && threadIdx.x == 0 && crank == 0) lf_set_status(P.status, LF_ERR_DEVICE_INPUT, LF_DET_LENGTH + b);
  const int d = P.dil[hk];
  const int own = ok ? lf_window_keys(len, P.window, d) : 0;
  const LfPmKeys keys{P.table + (size_t)b * P.max_pages, P.max_pages, own, len - 1, -d, LF_DET_PAGE + b,
                      ok && P.direct ? P.prefix_len : 0};
  LfPmState<MT> S;
  lf_pm_attend<T, MT>(P, keys, hk, kp, vp, crank, cl, qa, (uint32_t)__cvta_generic_to_shared(smem_raw), S);

  // Behind the warps' spilled states [4][16][64], shared memory of CTA 0 holds
  // the cluster's: acc [cl][gmax][64], m, l [cl][gmax].  The cluster barrier
  // says that CTA 0 is done with its rings.
  const int gmax = min(RB, P.G);
  float *s_acc = reinterpret_cast<float *>(smem_raw);
  float *c_acc = s_acc + 4 * 16 * LF_HD, *c_m = c_acc + cl * gmax * LF_HD, *c_l = c_m + cl * gmax;
  __syncthreads();
  if (cl > 1) cluster.barrier_arrive();
  if (prefix) asm volatile("griddepcontrol.wait;" ::: "memory");  // the prefix partials
  float *r_acc = cl > 1 ? cluster.map_shared_rank(c_acc, 0) : nullptr;
  float *r_m = cl > 1 ? cluster.map_shared_rank(c_m, 0) : nullptr;
  float *r_l = cl > 1 ? cluster.map_shared_rank(c_l, 0) : nullptr;
  const size_t orow = (size_t)b * P.H + hk * P.G + g0, prow = ((size_t)hk * P.B + b) * P.G + g0;
#pragma unroll
  for (int mt = 0; mt < MT; mt++) {
    if (mt > 0) __syncthreads();
    lf_pm_spill<MT>(S, mt, 16, s_acc, s_m, s_l);
    __syncthreads();
    if (mt == 0 && cl > 1) cluster.barrier_wait();
    for (int e = threadIdx.x; e < min(16, gn - 16 * mt) * LF_HD; e += 128) {
      const int r = e / LF_HD, c = e % LF_HD, x = 16 * mt + r;
      float M, L, a;
      lf_pm_merge(16, s_acc, s_m, s_l, r, c, M, L, a);
      if (prefix && ok) lf_pd_prefix(P, prow + x, c, crank, cl, M, L, a);
      if (cl > 1) {
        r_acc[(crank * gmax + x) * LF_HD + c] = a;
        if (c == 0) {
          r_m[crank * gmax + x] = M;
          r_l[crank * gmax + x] = L;
        }
      } else {
        lf_pd_write(o, lse, orow + x, c, M, L, a);
      }
    }
  }
  if (cl == 1) return;
  cluster.sync();  // the partials are in CTA 0
  if (crank != 0) return;
  for (int e = threadIdx.x; e < gn * LF_HD; e += 128) {
    const int x = e / LF_HD, c = e % LF_HD;
    float M = -INFINITY, L = 0.f, a = 0.f;
    for (int r = 0; r < cl; r++) M = fmaxf(M, c_m[r * gmax + x]);
    for (int r = 0; r < cl; r++) {
      const float f = lf_part_scale(c_m[r * gmax + x], M);
      L += c_l[r * gmax + x] * f;
      a += c_acc[(r * gmax + x) * LF_HD + c] * f;
    }
    lf_pd_write(o, lse, orow + x, c, M, L, a);
  }
}

template <typename T, int MT>
static cudaError_t lf_launch_pd_mma(const LfPagedLaunch &L, const void *q, const void *kp,
                                    const void *vp, void *o, float *lse) {
  const LfPagedDev &P = L.dev;
  constexpr int RB = 16 * MT;
  const int ngroups = (P.G + RB - 1) / RB, gmax = P.G < RB ? P.G : RB;
  const int64_t units = (int64_t)P.B * P.Hkv * ngroups;
  const int cl = lf_pd_cluster(P, units, LF_PM_KEYS, 8);
  const int merge = 4 * 16 * LF_HD * 4 + cl * gmax * (LF_HD + 2) * 4;
  const int smem = merge > LF_PM_RING ? merge : LF_PM_RING;
  const void *fn = (const void *)lf_paged_mma_kernel<T, MT>;
  const cudaError_t e = lf_kernel_smem(fn, smem);
  if (e != cudaSuccess) return e;
  return lf_pd_launch(fn, L, units, cl, smem, q, kp, vp, o, lse, ngroups);
}

// ============================ decode kernel (bf16, f16), many sequences

// All units' tiles in one list, cut into equal runs, one per CTA: CTAs stay
// busy to the end whatever the lengths are, and the loads of a CTA's next unit
// are in flight while it finishes one.  A unit that lies inside a run is
// written at once; of a unit that is cut, every CTA leaves its part in the
// workspace and the one that arrives last adds the parts, in the list's order
// (so the result does not depend on who that is).
struct LfPdRun {
  int b, hk, gc;          // unit
  int tile, nt;           // tile of the unit, its tiles
  int len, nk, d;
};

__device__ __forceinline__ int lf_pd_tiles(int nk) {
  return max(1, (nk + LF_PM_KEYS - 1) / LF_PM_KEYS);  // without keys one empty tile: the output is written all the same
}

__device__ __forceinline__ void lf_pd_unit(const LfPagedDev &P, const int *s_len, LfPdRun &R) {
  R.len = s_len[R.b];
  R.d = P.dil[R.hk];
  R.nk = lf_window_keys(R.len, P.window, R.d);
  R.nt = lf_pd_tiles(R.nk);
}

__device__ __forceinline__ void lf_pd_next(const LfPagedDev &P, const int *s_len, int ngroups, LfPdRun &R) {
  if (++R.tile < R.nt) return;
  R.tile = 0;
  if (++R.gc < ngroups) return;
  R.gc = 0;
  if (++R.hk < P.Hkv) {
    if (P.same_dil) return;
  } else {
    R.hk = 0;
    if (++R.b == P.B) R.b = 0;  // behind the list: not used
  }
  lf_pd_unit(P, s_len, R);
}

// The unit that holds the at-th tile of sequence b, and the tile of it.
__device__ __forceinline__ void lf_pd_find(const LfPagedDev &P, const int *s_len, int ngroups, int b, int at,
                                           LfPdRun &R) {
  R.b = b;
  R.hk = 0;
  for (;;) {
    lf_pd_unit(P, s_len, R);
    const int head = R.nt * ngroups;
    if (P.same_dil && P.Hkv > 1) {
      R.hk = at / head;
      at -= R.hk * head;
    }
    if (at < head) break;
    at -= head;
    R.hk++;
  }
  R.gc = ngroups > 1 ? at / R.nt : 0;
  R.tile = at - R.gc * R.nt;
}

// The list of `total` tiles is cut for n CTAs: per or per + 1 tiles each.
struct LfPdCuts {
  int n, per, more;  // the first `more` CTAs have one tile more
  __device__ __forceinline__ int at(int k) const { return k * per + min(k, more); }
  __device__ __forceinline__ int cta_of(int t) const {
    const int longer = more * (per + 1);
    return t < longer ? t / (per + 1) : more + (t - longer) / per;
  }
};

template <typename T, int MT>
__global__ void __launch_bounds__(128, MT == 1 ? 3 : 2)
    lf_paged_run_kernel(const __grid_constant__ LfPagedDev P, const T *q, const T *kp, const T *vp, T *o,
                        float *lse, int ngroups, int) {
  constexpr int RB = 16 * MT;
  extern __shared__ __align__(16) char smem_raw[];
  __shared__ float s_m[4][16], s_l[4][16];
  __shared__ int s_warp[4], s_last, s_at[2];
  __shared__ LfPdRun s_cut[2];
  const bool prefix = P.nch > 0;  // parts of a prefix kernel to add
  lf_pd_begin(prefix);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int gmax = min(RB, P.G), wrows = min(16, P.G);
  float *s_acc = reinterpret_cast<float *>(smem_raw + LF_PM_RING);  // [4][wrows][64]
  const LfPdFold fold = lf_pd_fold_at(smem_raw + LF_PM_RING + 4 * wrows * LF_HD * 4, wrows, P.nch);
  int *s_len = reinterpret_cast<int *>(s_acc + 4 * wrows * LF_HD);
  if (prefix) s_len += lf_pd_fold_bytes(wrows, P.nch) / 4;
  int *s_end = s_len + P.B;

  // tiles up to the end of each sequence
  int total = 0;
  for (int b0 = 0; b0 < P.B; b0 += 128) {
    const int b = b0 + tid;
    int n = 0;
    if (b < P.B) {
      int len = P.lengths[b];
      if (!lf_len_ok(len, P.max_pages, P.shift)) {
        if (blockIdx.x == 0) lf_set_status(P.status, LF_ERR_DEVICE_INPUT, LF_DET_LENGTH + b);
        len = -1;  // attends nothing, not even the prefix
      }
      s_len[b] = len;
      if (P.same_dil) {
        n = lf_pd_tiles(lf_window_keys(len, P.window, P.dil[0])) * P.Hkv;
      } else {
        for (int h = 0; h < P.Hkv; h++) n += lf_pd_tiles(lf_window_keys(len, P.window, P.dil[h]));
      }
      n *= ngroups;
    }
    int inc = n;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, w);
      if (lane >= w) inc += x;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int before = total;
    for (int w = 0; w < 4; w++) {
      if (w < warp) before += s_warp[w];
      total += s_warp[w];
    }
    if (b < P.B) s_end[b] = before + inc;
    __syncthreads();
  }

  // This CTA's run [begin, end): a cut that falls into a short unit moves to
  // the nearer of its ends (handing the parts of a unit over costs as much as
  // some tiles).  Lanes 0 and 1 of warp 0 find the two cuts' units.
  LfPdCuts cuts;
  cuts.n = min((int)gridDim.x, max(1, total));
  cuts.per = total / cuts.n;
  cuts.more = total - cuts.per * cuts.n;
  const int me = blockIdx.x;
  if (me < cuts.n) {
    for (int b = tid; b < P.B; b += 128) {
      const int b0 = b > 0 ? s_end[b - 1] : 0, b1 = s_end[b];
#pragma unroll
      for (int k = 0; k < 2; k++) {
        const int t = cuts.at(me + k);
        if (t >= b0 && t < b1) {
          s_cut[k].b = b;
          s_cut[k].tile = t - b0;
        }
      }
    }
    __syncthreads();
    LfPdRun C;
    if (tid < 2) {
      int t = cuts.at(me + tid);
      if (t < total) {
        lf_pd_find(P, s_len, ngroups, s_cut[tid].b, s_cut[tid].tile, C);
        if (C.nt <= LF_PDR_WHOLE) {
          t -= C.tile;
          if (2 * C.tile < C.nt) {
            C.tile = 0;
          } else {
            t += C.nt;
            C.tile = C.nt - 1;
            lf_pd_next(P, s_len, ngroups, C);
          }
        }
        s_cut[tid] = C;
      }
      s_at[tid] = t;
    }
    __syncthreads();
    C = s_cut[0];
    const int begin = s_at[0], end = s_at[1];

    LfPdRun F = C;  // the loader, LF_PM_STAGES - 1 tiles ahead
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem_raw) + warp * LF_PM_STAGES * LF_PM_STAGE;
    uint32_t have[LF_PM_STAGES] = {};
    int fill = begin, slot = 0, st = 0;
    LfPmAhead A;
    auto lookup = [&]() {
      lf_pm_lookup(P, LfPmKeys{P.table + (size_t)F.b * P.max_pages, P.max_pages, F.nk, F.len - 1, -F.d,
                               LF_DET_PAGE + F.b, 0}, F.tile, fill < end, A);
    };
    lookup();
    auto load = [&]() {
      uint32_t h = 0;
      if (fill < end) {
        h = lf_pm_load<T>(P, A, F.hk, kp, vp, ring + slot * LF_PM_STAGE);
        lf_pd_next(P, s_len, ngroups, F);
        fill++;
        lookup();
      }
      lf_cp_commit();
      slot = slot + 1 == LF_PM_STAGES ? 0 : slot + 1;
      return h;
    };
#pragma unroll
    for (int i = 0; i < LF_PM_STAGES - 1; i++) have[i] = load();

    LfPmQ<MT> qa;
    LfPmState<MT> S;
    int first = C.tile;  // first tile of the current unit in this run
    for (int i = begin; i < end; i++) {
      const int g0 = C.gc * RB, gn = min(RB, P.G - g0);
      if (i == begin || C.tile == 0) {
        lf_pd_queries<T, MT>(P, q, C.b, C.hk, g0, gn, qa);
        lf_pm_clear<MT>(S);
        first = C.tile;
      }
      lf_cp_wait<LF_PM_STAGES - 2>();
      __syncwarp();  // the tile is in for every lane, and the stage to fill next has been read
      have[LF_PM_STAGES - 1] = load();
      if (have[0]) lf_pm_tile<T, MT>(qa, ring + st * LF_PM_STAGE, have[0], P.scale_log2, S);
#pragma unroll
      for (int k = 0; k + 1 < LF_PM_STAGES; k++) have[k] = have[k + 1];
      st = st + 1 == LF_PM_STAGES ? 0 : st + 1;
      if (C.tile + 1 == C.nt || i + 1 == end) {
        const int ustart = i - C.tile, uend = ustart + C.nt;  // the unit in the list
        const bool whole = first == 0 && C.tile + 1 == C.nt;
        lf_pm_sum<T, MT>(S);
        if (prefix && whole) asm volatile("griddepcontrol.wait;" ::: "memory");  // the prefix partials
        const size_t orow = (size_t)C.b * P.H + C.hk * P.G + g0;
        const size_t prow = ((size_t)C.hk * P.B + C.b) * P.G + g0;
        const size_t mine = (size_t)(2 * me + (first == 0 ? 1 : 0)) * gmax;  // the run's last or first unit
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
          const int nr = min(16, gn - 16 * mt);
          const bool folds = prefix && whole && C.len >= 0 && nr > 0;
          lf_pm_spill<MT>(S, mt, wrows, s_acc, s_m, s_l);
          if (folds) lf_pd_fold(P, prow + 16 * mt, nr, fold);
          __syncthreads();
          for (int e = tid; e < nr * LF_HD; e += 128) {
            const int r = e / LF_HD, c = e % LF_HD, x = 16 * mt + r;
            float M, L, a;
            lf_pm_merge(wrows, s_acc, s_m, s_l, r, c, M, L, a);
            if (whole) {
              if (folds) lf_pd_folded(fold, nr, r, c, M, L, a);
              lf_pd_write(o, lse, orow + x, c, M, L, a);
            } else {
              P.run_acc[(mine + x) * LF_HD + c] = a;
              if (c == 0) P.run_ml[mine + x] = make_float2(M, L);
            }
          }
          if (whole || mt + 1 < MT) __syncthreads();  // s_acc, s_m, s_l are free again
        }
        if (!whole) {
          const int unit = (C.b * P.Hkv + C.hk) * ngroups + C.gc;
          __threadfence();
          __syncthreads();
          if (tid == 0) {
            const int part = C.tile + 1 - first;
            s_last = atomicAdd(P.run_count + unit, part) + part == C.nt;
            if (s_last) P.run_count[unit] = 0;  // for the next call
          }
          __syncthreads();
          if (s_last) {
            __threadfence();
            if (prefix) asm volatile("griddepcontrol.wait;" ::: "memory");
            const int c0 = cuts.cta_of(ustart), c1 = cuts.cta_of(uend - 1);
            for (int x0 = 0; x0 < gn; x0 += 16) {
              const int nr = min(16, gn - x0);
              const bool folds = prefix && C.len >= 0;
              if (folds) lf_pd_fold(P, prow + x0, nr, fold);
              for (int e = tid; e < nr * LF_HD; e += 128) {
                const int r = e / LF_HD, c = e % LF_HD, x = x0 + r;
                float M = -INFINITY, L = 0.f, a = 0.f;
#pragma unroll 4
                for (int k = c0; k <= c1; k++) {
                  const size_t from = (size_t)(2 * k + (cuts.at(k) <= ustart ? 1 : 0)) * gmax + x;
                  const float2 ml = __ldcg(P.run_ml + from);
                  lf_pd_add(ml.x, ml.y, __ldcg(P.run_acc + from * LF_HD + c), M, L, a);
                }
                if (folds) lf_pd_folded(fold, nr, r, c, M, L, a);
                lf_pd_write(o, lse, orow + x, c, M, L, a);
              }
              __syncthreads();
            }
          }
        }
      }
      lf_pd_next(P, s_len, ngroups, C);
    }
    lf_cp_wait<0>();
  }
  if (prefix) asm volatile("griddepcontrol.wait;" ::: "memory");  // no block ends before the prefix kernel
}

static int lf_pdm_rows(const LfPagedDev &P) { return P.G <= 16 ? 16 : 32; }

// Shared memory of the run kernel: rings, spilled states, prefix fold, lengths and ends.
static int lf_pdr_smem(const LfPagedDev &P) {
  const int wrows = P.G < 16 ? P.G : 16;
  return LF_PM_RING + 4 * wrows * LF_HD * 4 + (P.nch > 0 ? lf_pd_fold_bytes(wrows, P.nch) : 0) + 2 * P.B * 4;
}

// CTAs of the run kernel: as many as fit a full B200 at once: three per SM (two
// for groups of more than 16 query heads, whose states take 255 registers), fewer
// where the rings and the lengths leave no room for them.
void lf_paged_plan(LfPagedDev &P, int dtype) {
  P.run_ctas = 0;
  P.same_dil = 1;
  for (int h = 1; h < P.Hkv; h++) P.same_dil &= P.dil[h] == P.dil[0];
  if (dtype == LF_F32 || P.direct || P.B > LF_PDR_MAX_B) return;
  const int rb = lf_pdm_rows(P);
  const int64_t units = (int64_t)P.B * P.Hkv * ((P.G + rb - 1) / rb), keys = lf_most_keys(P);
  const int64_t tiles = units * ((keys + LF_PM_KEYS - 1) / LF_PM_KEYS);
  // Few units stay with a cluster each: its CTAs fit the GPU at once and need
  // no list.  Measured, clusters / runs, bf16, in us: 16 units of 8 heads with a
  // window of 257 keys 4.3 / 6.5, 64 units 5.5 / 6.6, 144 units 9.7 / 8.1; every
  // row up to 4000: 32 units 9.0 / 11.0, 64 units 16.4 / 15.5, 128 units 29.0 /
  // 25.1; up to 16000: 16 units 19.4 / 25.6, 64 units 36.6 / 34.6.  One sequence
  // of 1, 4, 16 and 32 heads: 8000 rows 9.5 / 12.3, 9.8 / 13.2, 12.3 / 14.3, 16.6 /
  // 20.0; 24000 rows 21.6 / 22.8, 22.2 / 24.1, 28.1 / 26.3, 38.1 / 39.8; 128000
  // rows 104 / 57, 105 / 39, 128 / 91, 183 / 169, but with 8 query heads to each
  // of 1 and 4 key/value heads 25.5 / 85.0 and 24.4 / 76.7 for 24000 rows, 106 /
  // 198 and 107 / 79 for 128000, as one CTA adds all parts of a unit.  Rows are
  // known here only as the table's capacity, which most sequences do not fill, so
  // the rule goes by the units.
  // Larger batches than the list's limits, clusters / runs: 1100 x 4 heads, 300
  // rows 60.5 / 59.7, the same behind 2000 rows of prefix 35.5 / 48.5, 2000 x 2
  // heads 72.7 / 96.6 (every CTA reads all lengths), but 1100 x 12 heads 114 / 87;
  // 40000 units 316 / 215, for which the counters would take four times the
  // workspace.
  const int few = P.nch == 0 && keys <= 512 ? 4 * 148 : 2 * 148;
  if (units * 8 <= few || units > LF_PDR_MAX_UNITS || tiles >= 1ll << 31) return;
  const int per = 228 * 1024 / (lf_pdr_smem(P) + 1024 + 640);  // 1 KB of the system's, 640 static
  const int most = rb == 16 ? 3 : 2;
  const int64_t ctas = 148 * (per < most ? per : most);
  P.run_ctas = (int)(tiles < ctas ? tiles : ctas);
}

template <typename T, int MT>
static cudaError_t lf_launch_pd_run(const LfPagedLaunch &L, const void *q, const void *kp,
                                    const void *vp, void *o, float *lse) {
  const LfPagedDev &P = L.dev;
  constexpr int RB = 16 * MT;
  const int smem = lf_pdr_smem(P);
  const void *fn = (const void *)lf_paged_run_kernel<T, MT>;
  const cudaError_t e = lf_kernel_smem(fn, smem);
  if (e != cudaSuccess) return e;
  return lf_pd_launch(fn, L, P.run_ctas, 1, smem, q, kp, vp, o, lse, (P.G + RB - 1) / RB);
}

template <typename T>
static cudaError_t lf_launch_pd_16(const LfPagedLaunch &L, const void *q, const void *kp,
                                   const void *vp, void *o, float *lse) {
  const bool run = L.dev.run_ctas > 0, small = lf_pdm_rows(L.dev) == 16;
  if (run) return small ? lf_launch_pd_run<T, 1>(L, q, kp, vp, o, lse) : lf_launch_pd_run<T, 2>(L, q, kp, vp, o, lse);
  return small ? lf_launch_pd_mma<T, 1>(L, q, kp, vp, o, lse) : lf_launch_pd_mma<T, 2>(L, q, kp, vp, o, lse);
}

cudaError_t lf_launch_paged_decode(const LfPagedLaunch &L, const void *q, const void *kp,
                                   const void *vp, void *o, float *lse) {
  cudaError_t e;
  if (L.dtype == LF_BF16)
    e = lf_launch_pd_16<__nv_bfloat16>(L, q, kp, vp, o, lse);
  else if (L.dtype == LF_F16)
    e = lf_launch_pd_16<__half>(L, q, kp, vp, o, lse);
  else if (L.dev.G == 1)
    e = lf_launch_pd_f32<1>(L, q, kp, vp, o, lse);
  else if (L.dev.G == 2)
    e = lf_launch_pd_f32<2>(L, q, kp, vp, o, lse);
  else
    e = lf_launch_pd_f32<4>(L, q, kp, vp, o, lse);
  if (e == cudaSuccess) lf_launches_add(1);
  return e;
}
