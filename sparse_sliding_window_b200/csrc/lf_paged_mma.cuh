// lf_paged_mma.cuh -- the attention loop shared by the 16-bit decode kernels
// and the 16-bit prefix kernel: a few query rows (16 MT <= 32) against keys
// that are scattered over the pages of the cache.
//
// The loop is bound by the K/V bytes, so what counts is that copies are
// always in flight and that a byte costs few instructions.  Four warps take
// 32 keys each of a tile of 128, against all rows.  Every warp has a ring of
// shared-memory stages of its own, filled by 16-byte asynchronous copies with
// one page lookup per lane and key: no barrier between warps until a
// sequence's end.  Rows that do not count are zero-filled, so no stray value
// of the pool enters a product.  Scores, probabilities and output stay in
// registers (m16n8k16 fragments).
#pragma once

#include <type_traits>

#include "lf_paged.cuh"
#include "lf_ptx.cuh"

#define LF_PM_KEYS 128                   // keys per tile, 32 per warp
#define LF_PM_HALF (32 * LF_HD * 2)      // bytes of a warp's K (or V) rows of a tile
#define LF_PM_STAGE (2 * LF_PM_HALF)
#define LF_PM_STAGES 2
#define LF_PM_RING (4 * LF_PM_STAGES * LF_PM_STAGE)  // bytes of the four warps' rings

// 2^(m - M), 0 for an empty part (m = -inf), also when everything is empty
__device__ __forceinline__ float lf_part_scale(float m, float M) {
  return m == -INFINITY ? 0.f : lf_ex2(m - M);
}

// 16 bytes to shared memory, zeros when !take (src is then not read)
__device__ __forceinline__ void lf_cp16(uint32_t dst, const void *src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void lf_cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void lf_cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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

// byte of 16-byte unit u of row r in a tile of 128-byte rows (units swizzled by row)
__device__ __forceinline__ uint32_t lf_pm_at(int r, int u) { return r * 128 + ((u ^ (r & 7)) << 4); }

// A warp's state: rows 16 mt + g and + 8 (g = lane / 4), output channels
// 8n + 2t, + 1 (t = lane % 4) in acc[mt][n] (f16: LF_P_SCALE times as large
// until lf_pm_sum).
template <int MT> struct LfPmState {
  float acc[MT][8][4], m[MT][2], l[MT][2];  // l: this thread's keys only, until lf_pm_sum
};
template <int MT> using LfPmQ = uint32_t[MT][4][4];  // A fragments: 16 rows x 64 channels each

// Where the keys are: key k < nkeys is cache row first + k * step of the table
// (detail: of the status when that has no page); the next nprefix keys are the
// rows of the shared prefix.
struct LfPmKeys {
  const int32_t *table;
  int columns, nkeys, first, step, detail, nprefix;
};

// The page of key 32 warp + lane of a tile is fetched one tile early
// (lf_pm_lookup) and only looked at when the tile is loaded (lf_pm_load): the
// table's latency stays off the loop.
struct LfPmAhead {
  int page, row, detail;
};
__device__ __forceinline__ void lf_pm_lookup(const LfPagedDev &P, const LfPmKeys &K, int tile, bool take,
                                             LfPmAhead &A) {
  const int k = tile * LF_PM_KEYS + (int)threadIdx.x;
  const bool own = k < K.nkeys;
  A.row = !take || k >= K.nkeys + K.nprefix ? LF_ROW_NONE : own ? K.first + k * K.step : k - K.nkeys;
  A.detail = own ? K.detail : LF_DET_PREFIX;
  if (lf_row_ok(own ? K.columns : (P.prefix_len + (1 << P.shift) - 1) >> P.shift, P.shift, A.row))
    A.page = (own ? K.table : P.prefix_table)[A.row >> P.shift];
  else
    A.row = LF_ROW_NONE;
}

// Starts the copies of the warp's 32 K and V rows into its stage `to` (eight
// lanes a row: a copy instruction moves whole 128-byte rows); returns the mask
// of the keys that count.
template <typename T>
__device__ __forceinline__ uint32_t lf_pm_load(const LfPagedDev &P, const LfPmAhead &A, int hk, const T *kp,
                                               const T *vp, uint32_t to) {
  const int lane = threadIdx.x % 32;
  int row = A.row;
  if (row >= 0) {
    row = lf_row_in_page(A.page, P.num_pages, P.shift, P.Hkv, hk, row);
    if (row == LF_ROW_BAD) lf_set_status(P.status, LF_ERR_DEVICE_INPUT, A.detail);
  }
  const uint32_t have = __ballot_sync(0xffffffffu, row >= 0);
  if (have == 0) return 0;  // nothing will be read of the stage
  const uint32_t dst = to + lf_pm_at(lane / 8, lane % 8), dst4 = to + lf_pm_at(lane / 8 + 4, lane % 8);
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int r = __shfl_sync(0xffffffffu, row, i * 4 + lane / 8);
    const int64_t at = (int64_t)max(r, 0) * LF_HD + lane % 8 * 8;
    const uint32_t d = (i % 2 ? dst4 : dst) + i / 2 * 1024;
    lf_cp16(d, kp + at, r >= 0);
    lf_cp16(d + LF_PM_HALF, vp + at, r >= 0);
  }
  return have;
}

template <int MT> __device__ __forceinline__ void lf_pm_clear(LfPmState<MT> &S) {
#pragma unroll
  for (int mt = 0; mt < MT; mt++) {
#pragma unroll
    for (int n = 0; n < 8; n++) S.acc[mt][n][0] = S.acc[mt][n][1] = S.acc[mt][n][2] = S.acc[mt][n][3] = 0.f;
    S.m[mt][0] = S.m[mt][1] = -INFINITY;
    S.l[mt][0] = S.l[mt][1] = 0.f;
  }
}

// The warp's 32 keys of a tile (K at sk, V behind it, mask ok of those that
// count, not 0) against its rows.
template <typename T, int MT>
__device__ __forceinline__ void lf_pm_tile(const LfPmQ<MT> &qa, uint32_t sk, uint32_t ok, float scale_log2,
                                           LfPmState<MT> &S) {
  const int lane = threadIdx.x % 32, t = lane % 4;
  const uint32_t sv = sk + LF_PM_HALF;
  float s[MT][4][4];
#pragma unroll
  for (int n = 0; n < 4; n++) {
#pragma unroll
    for (int mt = 0; mt < MT; mt++) s[mt][n][0] = s[mt][n][1] = s[mt][n][2] = s[mt][n][3] = 0.f;
#pragma unroll
    for (int hf = 0; hf < 2; hf++) {
      uint32_t b[4];  // 8 keys x 32 channels
      lf_ldsm4(sk + lf_pm_at(n * 8 + lane % 8, hf * 4 + lane / 8), b);
#pragma unroll
      for (int mt = 0; mt < MT; mt++) {
        lf_mma16<T>(s[mt][n], qa[mt][2 * hf], b[0], b[1]);
        lf_mma16<T>(s[mt][n], qa[mt][2 * hf + 1], b[2], b[3]);
      }
    }
  }
  // The scaled scores are rounded before the maximum is taken from them, and not
  // inside one operation with that subtraction: the largest exponent is 0 then,
  // however large the scores are (beyond 2^24 the difference to the rounded
  // maximum would be whole powers of two, and p infinite or 0 in every key).
#pragma unroll
  for (int mt = 0; mt < MT; mt++)
#pragma unroll
    for (int n = 0; n < 4; n++)
#pragma unroll
      for (int i = 0; i < 4; i++) s[mt][n][i] = __fmul_rn(s[mt][n][i], scale_log2);
  if (ok != 0xffffffffu) {
#pragma unroll
    for (int n = 0; n < 4; n++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (!(ok >> (n * 8 + 2 * t + (i & 1)) & 1u))
#pragma unroll
          for (int mt = 0; mt < MT; mt++) s[mt][n][i] = -INFINITY;
  }
#pragma unroll
  for (int mt = 0; mt < MT; mt++) {
    float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
    for (int n = 0; n < 4; n++) {
      M0 = fmaxf(M0, fmaxf(s[mt][n][0], s[mt][n][1]));
      M1 = fmaxf(M1, fmaxf(s[mt][n][2], s[mt][n][3]));
    }
#pragma unroll
    for (int w = 1; w < 4; w <<= 1) {
      M0 = fmaxf(M0, __shfl_xor_sync(0xffffffffu, M0, w));
      M1 = fmaxf(M1, __shfl_xor_sync(0xffffffffu, M1, w));
    }
    M0 = fmaxf(S.m[mt][0], M0);
    M1 = fmaxf(S.m[mt][1], M1);
    if (__any_sync(0xffffffffu, M0 > S.m[mt][0] || M1 > S.m[mt][1])) {
      const float f0 = lf_part_scale(S.m[mt][0], M0), f1 = lf_part_scale(S.m[mt][1], M1);
      S.m[mt][0] = M0;
      S.m[mt][1] = M1;
      S.l[mt][0] *= f0;
      S.l[mt][1] *= f1;
#pragma unroll
      for (int n = 0; n < 8; n++) {
        S.acc[mt][n][0] *= f0;
        S.acc[mt][n][1] *= f0;
        S.acc[mt][n][2] *= f1;
        S.acc[mt][n][3] *= f1;
      }
    }
    // a row whose scores are all -inf keeps m = -inf; its exponents then use 0
    const float e0 = M0 == -INFINITY ? 0.f : M0, e1 = M1 == -INFINITY ? 0.f : M1;
#pragma unroll
    for (int n = 0; n < 4; n++) {
      s[mt][n][0] = lf_ex2(s[mt][n][0] - e0);
      s[mt][n][1] = lf_ex2(s[mt][n][1] - e0);
      s[mt][n][2] = lf_ex2(s[mt][n][2] - e1);
      s[mt][n][3] = lf_ex2(s[mt][n][3] - e1);
      S.l[mt][0] += s[mt][n][0] + s[mt][n][1];
      S.l[mt][1] += s[mt][n][2] + s[mt][n][3];
    }
  }
  // P enters the product with V as two 16-bit numbers; the second product costs
  // 1 to 5% of a decode step.
#pragma unroll
  for (int k = 0; k < 2; k++) {
    uint32_t pa[MT][4], pb[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        lf_p_split<std::is_same<T, __half>::value, false>(
            s[mt][2 * k + i / 2][2 * (i % 2)], s[mt][2 * k + i / 2][2 * (i % 2) + 1], pa[mt][i], pb[mt][i]);
#pragma unroll
    for (int n = 0; n < 8; n += 2) {
      uint32_t b[4];  // 16 keys x 16 channels, transposed
      lf_ldsm4t(sv + lf_pm_at(k * 16 + lane % 16, n + lane / 16), b);
#pragma unroll
      for (int mt = 0; mt < MT; mt++) {
        lf_mma16<T>(S.acc[mt][n], pa[mt], b[0], b[1]);
        lf_mma16<T>(S.acc[mt][n + 1], pa[mt], b[2], b[3]);
        lf_mma16<T>(S.acc[mt][n], pb[mt], b[0], b[1]);
        lf_mma16<T>(S.acc[mt][n + 1], pb[mt], b[2], b[3]);
      }
    }
  }
}

// The row sums over the row's four threads; f16's factor out of the outputs.
template <typename T, int MT> __device__ __forceinline__ void lf_pm_sum(LfPmState<MT> &S) {
#pragma unroll
  for (int mt = 0; mt < MT; mt++) {
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
      for (int w = 1; w < 4; w <<= 1) S.l[mt][u] += __shfl_xor_sync(0xffffffffu, S.l[mt][u], w);
    if (std::is_same<T, __half>::value)
#pragma unroll
      for (int n = 0; n < 8; n++)
#pragma unroll
        for (int i = 0; i < 4; i++) S.acc[mt][n][i] *= 1.f / LF_P_SCALE;
  }
}

// Tiles tile0, tile0 + tstep, ... of the keys; ring: the four warps' stages.
// On return every copy of the warp has landed and been read.
template <typename T, int MT>
__device__ __forceinline__ void lf_pm_attend(const LfPagedDev &P, const LfPmKeys &K, int hk, const T *kp,
                                             const T *vp, int tile0, int tstep, const LfPmQ<MT> &qa,
                                             uint32_t ring, LfPmState<MT> &S) {
  const int ntiles = (K.nkeys + K.nprefix + LF_PM_KEYS - 1) / LF_PM_KEYS;
  ring += threadIdx.x / 32 * LF_PM_STAGES * LF_PM_STAGE;
  uint32_t ok[LF_PM_STAGES] = {};  // of the tiles in flight, oldest first
  int next = tile0, slot = 0, st = 0;
  LfPmAhead A;
  lf_pm_lookup(P, K, next, next < ntiles, A);
  auto load = [&]() {
    uint32_t have = 0;
    if (next < ntiles) have = lf_pm_load<T>(P, A, hk, kp, vp, ring + slot * LF_PM_STAGE);
    lf_cp_commit();
    next += tstep;
    slot = slot + 1 == LF_PM_STAGES ? 0 : slot + 1;
    lf_pm_lookup(P, K, next, next < ntiles, A);
    return have;
  };
#pragma unroll
  for (int i = 0; i < LF_PM_STAGES - 1; i++) ok[i] = load();
  lf_pm_clear<MT>(S);
  for (int tile = tile0; tile < ntiles; tile += tstep) {
    lf_cp_wait<LF_PM_STAGES - 2>();
    __syncwarp();  // the tile is in for every lane, and the stage to fill next has been read
    ok[LF_PM_STAGES - 1] = load();
    if (ok[0]) lf_pm_tile<T, MT>(qa, ring + st * LF_PM_STAGE, ok[0], P.scale_log2, S);
#pragma unroll
    for (int i = 0; i + 1 < LF_PM_STAGES; i++) ok[i] = ok[i + 1];
    st = st + 1 == LF_PM_STAGES ? 0 : st + 1;
  }
  lf_pm_sum<T, MT>(S);
  lf_cp_wait<0>();
  __syncwarp();
}

// 16 rows (mt) of the warps' states to shared memory, the first `rows` of
// them: acc [4 warps][rows][64], m and l [4][16].  The caller synchronises.
template <int MT>
__device__ __forceinline__ void lf_pm_spill(const LfPmState<MT> &S, int mt, int rows, float *s_acc,
                                            float (*s_m)[16], float (*s_l)[16]) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
#pragma unroll
  for (int k = 0; k < MT; k++) {  // constant indexes keep the state in registers
    if (k != mt) continue;
#pragma unroll
    for (int u = 0; u < 2; u++) {
      if (g + 8 * u >= rows) continue;
      if (t == 0) {
        s_m[warp][g + 8 * u] = S.m[k][u];
        s_l[warp][g + 8 * u] = S.l[k][u];
      }
#pragma unroll
      for (int n = 0; n < 8; n++)
        *reinterpret_cast<float2 *>(s_acc + (warp * rows + g + 8 * u) * LF_HD + n * 8 + 2 * t) =
            make_float2(S.acc[k][n][2 * u], S.acc[k][n][2 * u + 1]);
    }
  }
}

// Row r < rows, channel ch of the four warps' spilled states, merged.
__device__ __forceinline__ void lf_pm_merge(int rows, const float *s_acc, const float (*s_m)[16],
                                            const float (*s_l)[16], int r, int ch, float &M, float &L, float &a) {
  M = -INFINITY;
  L = a = 0.f;
#pragma unroll
  for (int w = 0; w < 4; w++) M = fmaxf(M, s_m[w][r]);
#pragma unroll
  for (int w = 0; w < 4; w++) {
    const float f = lf_part_scale(s_m[w][r], M);
    L += s_l[w][r] * f;
    a += s_acc[(w * rows + r) * LF_HD + ch] * f;
  }
}

// A fragments of rows ra = g and rb = g + 8.
template <typename T>
__device__ __forceinline__ void lf_pm_qfrag(const T *ra, const T *rb, uint32_t (&qa)[4][4]) {
  const int t = threadIdx.x % 4;
#pragma unroll
  for (int s = 0; s < 4; s++) {
    qa[s][0] = *reinterpret_cast<const uint32_t *>(ra + s * 16 + 2 * t);
    qa[s][1] = *reinterpret_cast<const uint32_t *>(rb + s * 16 + 2 * t);
    qa[s][2] = *reinterpret_cast<const uint32_t *>(ra + s * 16 + 8 + 2 * t);
    qa[s][3] = *reinterpret_cast<const uint32_t *>(rb + s * 16 + 8 + 2 * t);
  }
}
