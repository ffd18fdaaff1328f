// lf_prefix.cu -- the shared prefix of the paged decode: the queries of the
// whole batch (B * G rows per key/value head) against the prefix rows.
//
// A CTA takes a block of rows and one chunk of the prefix of one key/value
// head, runs an online softmax over tiles of 64 keys and leaves every row's
// (sum of p v, max, sum of p) of its chunk in the workspace, from where the
// decode kernel adds it to the row's own window.
#include "lf_paged_mma.cuh"

#define LF_PX_KEYS 64  // keys per tile

// Query row x (0 .. B*G-1) of key/value head hk: sequence x / G, head hk*G + x % G.
template <typename T>
__device__ __forceinline__ const T *lf_px_row(const LfPagedDev &P, const T *q, int hk, int x) {
  return q + (int64_t)(x / P.G) * P.qs[0] + (int64_t)(hk * P.G + x % P.G) * P.qs[1];
}

// ------------------------------------------------------------- f32 (CUDA cores)

// 256 threads, 32 rows.  Thread (r, c) = (tid / 16, tid % 16) has rows r and
// r + 16: scores of keys c, c+16, c+32, c+48, then channels 4c .. 4c+3 of the
// output.  The 16 threads of a row are lanes of one warp, so the row's
// statistics and probabilities stay inside the warp.  float32 throughout (no
// TF32: its 10-bit mantissa cannot hold float32 scores).
#define LF_PXS_ROWS 32
#define LF_PXS_KP 68  // padded row of Q and K tiles, in floats (bank spread)
struct LfPxsSmem {
  float q[LF_PXS_ROWS][LF_PXS_KP];
  float p[LF_PXS_ROWS][LF_PX_KEYS];
  float k[2][LF_PX_KEYS][LF_PXS_KP];
  float v[2][LF_PX_KEYS][LF_HD];
  int ok[2][LF_PX_KEYS];
};

__global__ void __launch_bounds__(256) lf_prefix_simt_kernel(const __grid_constant__ LfPagedDev P,
                                                             const float *q, const float *kp,
                                                             const float *vp) {
  extern __shared__ __align__(16) char smem_raw[];
  LfPxsSmem &S = *reinterpret_cast<LfPxsSmem *>(smem_raw);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int chunk = blockIdx.x, x0 = blockIdx.y * LF_PXS_ROWS, hk = blockIdx.z;
  const int rows = P.B * P.G, tid = threadIdx.x, r = tid / 16, c = tid % 16;
  const int j0 = chunk * P.chunk, j1 = min(P.prefix_len, j0 + P.chunk);
  const int columns = (P.prefix_len + (1 << P.shift) - 1) >> P.shift;

  auto load = [&](int j, int buf) {
    // 4 threads per key row, 16 channels each
    const int kr = tid / 4, part = (tid % 4) * 16;
    const int row = j + kr < j1 ? lf_pool_row(P.prefix_table, columns, P.num_pages, P.shift, P.Hkv, hk, j + kr)
                                : LF_ROW_NONE;
    if (row == LF_ROW_BAD) lf_set_status(P.status, LF_ERR_DEVICE_INPUT, LF_DET_PREFIX);
    if (tid % 4 == 0) S.ok[buf][kr] = row >= 0;
    const int64_t at = (int64_t)max(row, 0) * LF_HD + part;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      lf_cp16((uint32_t)__cvta_generic_to_shared(&S.k[buf][kr][part + i]), kp + at + i, row >= 0);
      lf_cp16((uint32_t)__cvta_generic_to_shared(&S.v[buf][kr][part + i]), vp + at + i, row >= 0);
    }
    lf_cp_commit();
  };

  load(j0, 0);
  for (int i = tid; i < LF_PXS_ROWS * LF_HD; i += 256) {
    const int x = i / LF_HD, ch = i % LF_HD;
    S.q[x][ch] = x0 + x < rows ? lf_px_row(P, q, hk, x0 + x)[ch] * P.scale_log2 : 0.f;
  }
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, acc[2][4] = {};
  int buf = 0;
  for (int j = j0; j < j1; j += LF_PX_KEYS, buf ^= 1) {
    lf_cp_wait<0>();
    __syncthreads();  // the tile is in, and the other buffer is free
    if (j + LF_PX_KEYS < j1) load(j + LF_PX_KEYS, buf ^ 1);
    float s[2][4] = {};
#pragma unroll 4
    for (int ch = 0; ch < LF_HD; ch += 4) {
      float4 a[2];
#pragma unroll
      for (int u = 0; u < 2; u++) a[u] = *reinterpret_cast<const float4 *>(&S.q[r + 16 * u][ch]);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float4 k4 = *reinterpret_cast<const float4 *>(&S.k[buf][c + 16 * i][ch]);
#pragma unroll
        for (int u = 0; u < 2; u++)
          s[u][i] += a[u].x * k4.x + a[u].y * k4.y + a[u].z * k4.z + a[u].w * k4.w;
      }
    }
    bool ok[4];
#pragma unroll
    for (int i = 0; i < 4; i++) ok[i] = S.ok[buf][c + 16 * i] != 0;
#pragma unroll
    for (int u = 0; u < 2; u++) {
      float M = m[u];
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (ok[i]) M = fmaxf(M, s[u][i]);
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
      const float f = lf_part_scale(m[u], M), e = M == -INFINITY ? 0.f : M;
      m[u] = M;
      l[u] *= f;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        acc[u][i] *= f;
        const float p = ok[i] ? lf_ex2(s[u][i] - e) : 0.f;
        l[u] += p;
        S.p[r + 16 * u][c + 16 * i] = p;
      }
    }
    __syncwarp();
#pragma unroll 4
    for (int k = 0; k < LF_PX_KEYS; k++) {
      const float4 v4 = *reinterpret_cast<const float4 *>(&S.v[buf][k][4 * c]);
#pragma unroll
      for (int u = 0; u < 2; u++) {
        const float p = S.p[r + 16 * u][k];
        acc[u][0] += p * v4.x;
        acc[u][1] += p * v4.y;
        acc[u][2] += p * v4.z;
        acc[u][3] += p * v4.w;
      }
    }
    __syncwarp();
  }
#pragma unroll
  for (int u = 0; u < 2; u++) {
    float L = l[u];
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) L += __shfl_xor_sync(0xffffffffu, L, w);
    const int x = x0 + r + 16 * u;
    if (x >= rows) continue;
    const size_t at = ((size_t)hk * rows + x) * P.nch + chunk;
    *reinterpret_cast<float4 *>(P.part_acc + at * LF_HD + 4 * c) =
        make_float4(acc[u][0], acc[u][1], acc[u][2], acc[u][3]);
    if (c == 0) P.part_ml[at] = make_float2(m[u], L);
  }
}

// ---------------------------------------- bf16 / f16, 16 MT rows a block

template <typename T, int MT>
__global__ void __launch_bounds__(128, 2) lf_prefix_mma_kernel(const __grid_constant__ LfPagedDev P,
                                                               const T *q, const T *kp, const T *vp) {
  extern __shared__ __align__(16) char smem_raw[];
  __shared__ float s_m[4][16], s_l[4][16];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int chunk = blockIdx.x, x0 = blockIdx.y * 16 * MT, hk = blockIdx.z;
  const int rows = P.B * P.G, g = threadIdx.x % 32 / 4;
  const int j0 = chunk * P.chunk, nkeys = min(P.prefix_len - j0, P.chunk);
  const int columns = (P.prefix_len + (1 << P.shift) - 1) >> P.shift;
  LfPmQ<MT> qa;
#pragma unroll
  for (int mt = 0; mt < MT; mt++) {
    const int xa = x0 + 16 * mt + g;
    lf_pm_qfrag<T>(lf_px_row(P, q, hk, min(xa, rows - 1)), lf_px_row(P, q, hk, min(xa + 8, rows - 1)), qa[mt]);
  }
  LfPmState<MT> S;
  lf_pm_attend<T, MT>(P, LfPmKeys{P.prefix_table, columns, nkeys, j0, 1, LF_DET_PREFIX, 0}, hk, kp, vp, 0, 1, qa,
                      (uint32_t)__cvta_generic_to_shared(smem_raw), S);
  float *s_acc = reinterpret_cast<float *>(smem_raw);
#pragma unroll
  for (int mt = 0; mt < MT; mt++) {
    __syncthreads();  // the rings (and the last rows) have been read
    lf_pm_spill<MT>(S, mt, 16, s_acc, s_m, s_l);
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * LF_HD; e += 128) {
      const int r = e / LF_HD, ch = e % LF_HD, x = x0 + 16 * mt + r;
      if (x >= rows) break;
      float M, L, a;
      lf_pm_merge(16, s_acc, s_m, s_l, r, ch, M, L, a);
      const size_t at = ((size_t)hk * rows + x) * P.nch + chunk;
      P.part_acc[at * LF_HD + ch] = a;
      if (ch == 0) P.part_ml[at] = make_float2(M, L);
    }
  }
}

// ----------------------------------------------------------------- launches

// The tensor-core kernel's tile has 128 rows: it takes over where the rows no
// longer fit one block of the warp-level kernel (which would read the prefix
// once per 32 rows).  Measured, warp-level / tensor-core, bf16, whole calls with a
// window of 64, in us, on 500, 1000, 2000 and 4096 rows: 40 x 12 heads 13.7 /
// 14.6, 13.8 / 14.8, 18.0 / 14.0, 21.3 / 16.2; 64 x 12 heads 15.5 / 16.1, 17.5 /
// 16.5, 22.6 / 17.8, 26.5 / 20.3; 128 x 12 heads 24.4 / 24.9, 28.5 / 25.7, 31.3 /
// 28.1, 38.3 / 30.1; 64 x 16/4 heads 12.3 / 12.1, 14.3 / 13.4, 19.6 / 13.9, 22.7 /
// 15.4.  By the rows alone it is up to a fifth off on prefixes of 1000 and 2000
// rows for few of them: 20 x 16/4 heads 8.6 / 8.5, 8.5 / 9.6, 10.9 / 13.0, 16.1 /
// 13.5.
static bool lf_prefix_is_tc(const LfPagedDev &d, int dtype) { return dtype != LF_F32 && (int64_t)d.B * d.G > 32; }

static int lf_prefix_rows(const LfPagedDev &d, int dtype) {
  if (dtype == LF_F32) return LF_PXS_ROWS;
  return d.B * d.G <= 16 ? 16 : 32;
}

// Chunks: about four CTAs per SM of a full B200 (148 SMs; a fixed count keeps
// the workspace size a function of the params alone), whole tiles each, and
// at most 64 of them, so that merging stays short.
void lf_prefix_plan(LfPagedDev &d, int dtype) {
  d.nch = 0;
  d.chunk = 0;
  d.direct = d.prefix_len > 0 && lf_prefix_direct(d, dtype);
  if (d.prefix_len <= 0 || d.direct) return;
  if (lf_prefix_is_tc(d, dtype)) return lf_prefix_tc_plan(d);
  const int rb = lf_prefix_rows(d, dtype);
  const int64_t blocks = (int64_t)d.Hkv * ((d.B * d.G + rb - 1) / rb);
  const int keys = dtype == LF_F32 ? LF_PX_KEYS : LF_PM_KEYS;  // of a tile
  const int tiles = (d.prefix_len + keys - 1) / keys;
  int64_t want = (4 * 148 + blocks - 1) / blocks;
  if (want > LF_PART_MAX) want = LF_PART_MAX;
  if (want > tiles) want = tiles;
  const int per = (int)((tiles + want - 1) / want);
  d.chunk = per * keys;
  d.nch = (tiles + per - 1) / per;
}

static cudaError_t lf_px_launch(const void *fn, const LfPagedLaunch &L, int rb, int threads, int smem,
                                const void *q, const void *kp, const void *vp) {
  const LfPagedDev &P = L.dev;
  cudaError_t e = lf_kernel_smem(fn, smem);
  if (e != cudaSuccess) return e;
  const int rblocks = (P.B * P.G + rb - 1) / rb;
  if (rblocks > 65535) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)P.nch, (unsigned)rblocks, (unsigned)P.Hkv);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = L.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void *args[] = {const_cast<LfPagedDev *>(&P), &q, &kp, &vp};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

template <typename T>
static cudaError_t lf_launch_prefix_t(const LfPagedLaunch &L, const void *q, const void *kp, const void *vp) {
  const int rb = lf_prefix_rows(L.dev, L.dtype);
  const void *fn = rb == 16 ? (const void *)lf_prefix_mma_kernel<T, 1> : (const void *)lf_prefix_mma_kernel<T, 2>;
  return lf_px_launch(fn, L, rb, 128, LF_PM_RING, q, kp, vp);
}

cudaError_t lf_launch_prefix(const LfPagedLaunch &L, const void *q, const void *kp, const void *vp) {
  cudaError_t e;
  if (L.dtype == LF_F32)
    e = lf_px_launch((const void *)lf_prefix_simt_kernel, L, LF_PXS_ROWS, 256, (int)sizeof(LfPxsSmem), q, kp, vp);
  else if (lf_prefix_is_tc(L.dev, L.dtype))
    e = lf_launch_prefix_tc(L, q, kp, vp);
  else if (L.dtype == LF_BF16)
    e = lf_launch_prefix_t<__nv_bfloat16>(L, q, kp, vp);
  else
    e = lf_launch_prefix_t<__half>(L, q, kp, vp);
  if (e == cudaSuccess) lf_launches_add(1);
  return e;
}
