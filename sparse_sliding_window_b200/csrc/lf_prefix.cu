// lf_prefix.cu -- the shared prefix of the paged decode: the queries of the
// whole batch (B * G rows per key/value head) against the prefix rows.
//
// A CTA takes a block of rows and one chunk of the prefix of one key/value
// head, runs an online softmax over tiles of 64 keys and leaves every row's
// (sum of p v, max, sum of p) of its chunk in the workspace, from where the
// decode kernel adds it to the row's own window.
#include <type_traits>

#include "lf_paged.cuh"

#define LF_PX_KEYS 64  // keys per tile

__device__ __forceinline__ float lf_px_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void lf_cp16(void *dst, const void *src, bool take) {
  const uint32_t s = (uint32_t)__cvta_generic_to_shared(dst);
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(s), "l"(src), "r"(take ? 16 : 0)
               : "memory");
}

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
      lf_cp16(&S.k[buf][kr][part + i], kp + at + i, row >= 0);
      lf_cp16(&S.v[buf][kr][part + i], vp + at + i, row >= 0);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  load(j0, 0);
  for (int i = tid; i < LF_PXS_ROWS * LF_HD; i += 256) {
    const int x = i / LF_HD, ch = i % LF_HD;
    S.q[x][ch] = x0 + x < rows ? lf_px_row(P, q, hk, x0 + x)[ch] * P.scale_log2 : 0.f;
  }
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, acc[2][4] = {};
  int buf = 0;
  for (int j = j0; j < j1; j += LF_PX_KEYS, buf ^= 1) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
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
      const float f = m[u] == -INFINITY ? 0.f : lf_px_exp2(m[u] - M);
      m[u] = M;
      l[u] *= f;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        acc[u][i] *= f;
        const float p = ok[i] ? lf_px_exp2(s[u][i] - M) : 0.f;
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

// ------------------------------------------- bf16 / f16 (warp-level matrix)

// 128 threads; WR warps along the rows (16 each), 4 / WR along the keys of a
// tile.  K and V tiles in a ring of LF_PXM_STAGES shared-memory stages filled
// by 16-byte asynchronous copies (rows that do not count are zero-filled, so
// no stray value of the pool enters a product); S, the probabilities and the
// output stay in registers.
#define LF_PXM_STAGES 4
#define LF_PXM_TILE (LF_PX_KEYS * LF_HD * 2)  // bytes of a K or V tile
#define LF_PXM_SMEM (LF_PXM_STAGES * 2 * LF_PXM_TILE)

__device__ __forceinline__ void lf_ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void lf_ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void lf_mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T>
__device__ __forceinline__ uint32_t lf_px_pack(float a, float b) {
  uint32_t w;
  LfIo<T>::st2(reinterpret_cast<T *>(&w), a, b);
  return w;
}

// 16-byte unit u of row r of a tile of 128-byte rows (units swizzled by row)
__device__ __forceinline__ uint32_t lf_px_at(int r, int u) { return r * 128 + ((u ^ (r & 7)) << 4); }

template <typename T, int WR>
__global__ void __launch_bounds__(128) lf_prefix_mma_kernel(const __grid_constant__ LfPagedDev P,
                                                            const T *q, const T *kp, const T *vp) {
  constexpr int WK = 4 / WR, KW = LF_PX_KEYS / WK;  // warps along the keys, keys per warp
  extern __shared__ __align__(16) char smem_raw[];
  __shared__ uint32_t s_ok[LF_PXM_STAGES][4];  // 16 keys each
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int chunk = blockIdx.x, x0 = blockIdx.y * 16 * WR, hk = blockIdx.z;
  const int rows = P.B * P.G, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int wr = warp / WK, wk = warp % WK, g = lane / 4, t = lane % 4;
  const int j0 = chunk * P.chunk, j1 = min(P.prefix_len, j0 + P.chunk);
  const int ntiles = (j1 - j0 + LF_PX_KEYS - 1) / LF_PX_KEYS;
  const int columns = (P.prefix_len + (1 << P.shift) - 1) >> P.shift;
  const uint32_t sbase = (uint32_t)__cvta_generic_to_shared(smem_raw);

  auto load = [&](int tile) {
    // 2 threads per key row, 4 units each of K and V
    const int st = tile % LF_PXM_STAGES, kr = tid / 2, u0 = (tid % 2) * 4;
    const int j = j0 + tile * LF_PX_KEYS + kr;
    int row = LF_ROW_NONE;
    if (tile < ntiles && j < j1)
      row = lf_pool_row(P.prefix_table, columns, P.num_pages, P.shift, P.Hkv, hk, j);
    if (row == LF_ROW_BAD) lf_set_status(P.status, LF_ERR_DEVICE_INPUT, LF_DET_PREFIX);
    if (tile < ntiles) {
      const uint32_t two = __ballot_sync(0xffffffffu, row >= 0);  // two bits per key
      uint32_t bits = 0;
#pragma unroll
      for (int i = 0; i < 16; i++) bits |= (two >> (2 * i) & 1u) << i;
      if (lane == 0) s_ok[st][warp] = bits;
      char *kd = smem_raw + st * 2 * LF_PXM_TILE, *vd = kd + LF_PXM_TILE;
      const int64_t at = (int64_t)max(row, 0) * LF_HD;
#pragma unroll
      for (int u = 0; u < 4; u++) {
        lf_cp16(kd + lf_px_at(kr, u0 + u), kp + at + (u0 + u) * 8, row >= 0);
        lf_cp16(vd + lf_px_at(kr, u0 + u), vp + at + (u0 + u) * 8, row >= 0);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < LF_PXM_STAGES - 1; i++) load(i);

  // the warp's 16 query rows as A fragments, four steps of 16 channels
  uint32_t qa[4][4];
  {
    const int xa = x0 + wr * 16 + g, xb = xa + 8;
    const T *ra = lf_px_row(P, q, hk, min(xa, rows - 1)), *rb = lf_px_row(P, q, hk, min(xb, rows - 1));
#pragma unroll
    for (int s = 0; s < 4; s++) {
      qa[s][0] = *reinterpret_cast<const uint32_t *>(ra + s * 16 + 2 * t);
      qa[s][1] = *reinterpret_cast<const uint32_t *>(rb + s * 16 + 2 * t);
      qa[s][2] = *reinterpret_cast<const uint32_t *>(ra + s * 16 + 8 + 2 * t);
      qa[s][3] = *reinterpret_cast<const uint32_t *>(rb + s * 16 + 8 + 2 * t);
    }
  }
  float acc[8][4] = {};
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // rows g and g + 8
  for (int tile = 0; tile < ntiles; tile++) {
    asm volatile("cp.async.wait_group %0;" ::"n"(LF_PXM_STAGES - 2) : "memory");
    __syncthreads();
    load(tile + LF_PXM_STAGES - 1);
    const int st = tile % LF_PXM_STAGES;
    const uint32_t sk = sbase + st * 2 * LF_PXM_TILE, sv = sk + LF_PXM_TILE;
    float s[KW / 8][4];
#pragma unroll
    for (int n = 0; n < KW / 8; n++) {
      s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
      for (int hf = 0; hf < 2; hf++) {
        uint32_t b[4];  // 8 keys x 32 channels
        lf_ldsm4(sk + lf_px_at(wk * KW + n * 8 + lane % 8, hf * 4 + lane / 8), b);
        lf_mma16<T>(s[n], qa[2 * hf], b[0], b[1]);
        lf_mma16<T>(s[n], qa[2 * hf + 1], b[2], b[3]);
      }
    }
    uint32_t ok = 0xffffffffu;
    bool all = true;
    float M0 = m[0], M1 = m[1];
#pragma unroll
    for (int n = 0; n < KW / 8; n++) {
      if (n % 2 == 0) {
        ok = s_ok[st][(wk * KW + n * 8) / 16];
        all = ok == 0xffffu;
      }
#pragma unroll
      for (int i = 0; i < 4; i++) {
        s[n][i] *= P.scale_log2;
        if (!all && !(ok >> ((n % 2) * 8 + 2 * t + (i & 1)) & 1u)) s[n][i] = -INFINITY;
      }
      M0 = fmaxf(M0, fmaxf(s[n][0], s[n][1]));
      M1 = fmaxf(M1, fmaxf(s[n][2], s[n][3]));
    }
#pragma unroll
    for (int w = 1; w < 4; w <<= 1) {
      M0 = fmaxf(M0, __shfl_xor_sync(0xffffffffu, M0, w));
      M1 = fmaxf(M1, __shfl_xor_sync(0xffffffffu, M1, w));
    }
    // an all-masked part keeps m = -inf; its exponents then use 0
    const float f0 = m[0] == -INFINITY ? 0.f : lf_px_exp2(m[0] - M0);
    const float f1 = m[1] == -INFINITY ? 0.f : lf_px_exp2(m[1] - M1);
    const float e0 = M0 == -INFINITY ? 0.f : M0, e1 = M1 == -INFINITY ? 0.f : M1;
    m[0] = M0;
    m[1] = M1;
    l[0] *= f0;
    l[1] *= f1;
#pragma unroll
    for (int n = 0; n < 8; n++) {
      acc[n][0] *= f0;
      acc[n][1] *= f0;
      acc[n][2] *= f1;
      acc[n][3] *= f1;
    }
    // P is rounded to the 16-bit type for the product with V (p <= 1, half a
    // step relative each; the row sum keeps the unrounded values)
#pragma unroll
    for (int n = 0; n < KW / 8; n++) {
      s[n][0] = lf_px_exp2(s[n][0] - e0);
      s[n][1] = lf_px_exp2(s[n][1] - e0);
      s[n][2] = lf_px_exp2(s[n][2] - e1);
      s[n][3] = lf_px_exp2(s[n][3] - e1);
      l[0] += s[n][0] + s[n][1];
      l[1] += s[n][2] + s[n][3];
    }
#pragma unroll
    for (int k = 0; k < KW / 16; k++) {
      const uint32_t pa[4] = {lf_px_pack<T>(s[2 * k][0], s[2 * k][1]), lf_px_pack<T>(s[2 * k][2], s[2 * k][3]),
                              lf_px_pack<T>(s[2 * k + 1][0], s[2 * k + 1][1]),
                              lf_px_pack<T>(s[2 * k + 1][2], s[2 * k + 1][3])};
#pragma unroll
      for (int n = 0; n < 8; n += 2) {
        uint32_t b[4];  // 16 keys x 16 channels, transposed
        lf_ldsm4t(sv + lf_px_at(wk * KW + k * 16 + lane % 16, n + lane / 16), b);
        lf_mma16<T>(acc[n], pa, b[0], b[1]);
        lf_mma16<T>(acc[n + 1], pa, b[2], b[3]);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < 2; u++)
#pragma unroll
    for (int w = 1; w < 4; w <<= 1) l[u] += __shfl_xor_sync(0xffffffffu, l[u], w);

  asm volatile("cp.async.wait_group 0;" ::: "memory");
  // warps of the same rows merge through the stage buffers
  float *s_acc = reinterpret_cast<float *>(smem_raw);           // [4 warps][16][64]
  __shared__ float s_m[4][16], s_l[4][16];
  if (WK > 1) {
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; u++) {
      if (t == 0) {
        s_m[warp][g + 8 * u] = m[u];
        s_l[warp][g + 8 * u] = l[u];
      }
#pragma unroll
      for (int n = 0; n < 8; n++)
        *reinterpret_cast<float2 *>(s_acc + (warp * 16 + g + 8 * u) * LF_HD + n * 8 + 2 * t) =
            make_float2(acc[n][2 * u], acc[n][2 * u + 1]);
    }
    __syncthreads();
    for (int e = tid; e < WR * 16 * LF_HD; e += 128) {
      const int w0 = e / (16 * LF_HD) * WK, x = e / LF_HD % 16, ch = e % LF_HD;
      const int xr = x0 + w0 / WK * 16 + x;
      if (xr >= rows) continue;
      float M = -INFINITY, L = 0.f, a = 0.f;
#pragma unroll
      for (int w = 0; w < WK; w++) M = fmaxf(M, s_m[w0 + w][x]);
#pragma unroll
      for (int w = 0; w < WK; w++) {
        const float mw = s_m[w0 + w][x], f = mw == -INFINITY ? 0.f : lf_px_exp2(mw - M);
        L += s_l[w0 + w][x] * f;
        a += s_acc[((w0 + w) * 16 + x) * LF_HD + ch] * f;
      }
      const size_t at = ((size_t)hk * rows + xr) * P.nch + chunk;
      P.part_acc[at * LF_HD + ch] = a;
      if (ch == 0) P.part_ml[at] = make_float2(M, L);
    }
  } else {
#pragma unroll
    for (int u = 0; u < 2; u++) {
      const int xr = x0 + wr * 16 + g + 8 * u;
      if (xr >= rows) continue;
      const size_t at = ((size_t)hk * rows + xr) * P.nch + chunk;
#pragma unroll
      for (int n = 0; n < 8; n++)
        *reinterpret_cast<float2 *>(P.part_acc + at * LF_HD + n * 8 + 2 * t) =
            make_float2(acc[n][2 * u], acc[n][2 * u + 1]);
      if (t == 0) P.part_ml[at] = make_float2(m[u], l[u]);
    }
  }
}

// ----------------------------------------------------------------- launches

static int lf_prefix_rows(const LfPagedDev &d, int dtype) {
  if (dtype == LF_F32) return LF_PXS_ROWS;
  const int rows = d.B * d.G;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

// Chunks: about four CTAs per SM of a full B200 (148 SMs; a fixed count keeps
// the workspace size a function of the params alone), whole tiles each, and
// at most 64 of them, so that merging stays short.
void lf_prefix_plan(LfPagedDev &d, int dtype) {
  d.nch = 0;
  d.chunk = LF_PX_KEYS;
  if (d.prefix_len <= 0) return;
  const int rb = lf_prefix_rows(d, dtype);
  const int64_t blocks = (int64_t)d.Hkv * ((d.B * d.G + rb - 1) / rb);
  const int tiles = (d.prefix_len + LF_PX_KEYS - 1) / LF_PX_KEYS;
  int64_t want = (4 * 148 + blocks - 1) / blocks;
  if (want > 64) want = 64;
  if (want > tiles) want = tiles;
  const int per = (int)((tiles + want - 1) / want);
  d.chunk = per * LF_PX_KEYS;
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
  const void *fn = rb == 16   ? (const void *)lf_prefix_mma_kernel<T, 1>
                   : rb == 32 ? (const void *)lf_prefix_mma_kernel<T, 2>
                              : (const void *)lf_prefix_mma_kernel<T, 4>;
  return lf_px_launch(fn, L, rb, 128, LF_PXM_SMEM, q, kp, vp);
}

cudaError_t lf_launch_prefix(const LfPagedLaunch &L, const void *q, const void *kp, const void *vp) {
  cudaError_t e;
  if (L.dtype == LF_F32)
    e = lf_px_launch((const void *)lf_prefix_simt_kernel, L, LF_PXS_ROWS, 256, (int)sizeof(LfPxsSmem), q, kp, vp);
  else if (L.dtype == LF_BF16)
    e = lf_launch_prefix_t<__nv_bfloat16>(L, q, kp, vp);
  else
    e = lf_launch_prefix_t<__half>(L, q, kp, vp);
  if (e == cudaSuccess) lf_launches_add(1);
  return e;
}
