// lf_prefix_tc.cu -- the shared prefix for many query rows (bf16, f16): the
// tensor-core (tcgen05) form of the prefix kernel.
//
// A CTA takes 128 query rows (of the B * G of a key/value head) and one chunk
// of the prefix.  Its 128-key tiles go to two streams in turn; per stream four
// softmax warps, one row per thread, with S, O and P in TMEM:
//   warp 8   loads K and V tiles by TMA, a box per page, into a ring
//   warp 9   issues S = Q K^T (128 x 128 x 64) and O += P V (128 x 64 x 128)
//   warps 0-3, 4-7  softmax of stream 0, 1
// S is read into registers whole and handed back at once, so the next S of
// the stream is computed while this one's exponentials are; with two streams
// the exponentials (128 per row and tile, 16 a cycle and SM) never wait for a
// matrix product.  Every stream leaves (sum of p v, max, sum of p) per row.
#include <cuda.h>

#include "lf_paged.cuh"
#include "lf_ptx.cuh"
#include "lf_tc.cuh"

#define LF_PT_ROWS 128
#define LF_PT_KEYS 128
#define LF_PT_THREADS 384  // warps 10 and 11 fill the loader's warpgroup and do nothing
// Registers: the launch gives 168 a thread (384 * 168 = 64512); the loader's
// warpgroup keeps 88, so that the softmax warps can hold a whole row of S.
#define LF_PT_REGS_FEW 88
#define LF_PT_REGS_MANY 208
static_assert(256 * LF_PT_REGS_MANY + 128 * LF_PT_REGS_FEW <= 384 * 168, "register split");
#define LF_PT_NS 6  // K/V tiles in the ring (32 KB each)

#define LF_PT_Q 0
#define LF_PT_K(s) (16384 + (s)*32768)
#define LF_PT_V(s) (16384 + (s)*32768 + 16384)
#define LF_PT_MISC (16384 + LF_PT_NS * 32768)
#define LF_PT_SMEM (LF_PT_MISC + 512)
// barriers, from LF_PT_MISC
#define LF_PT_KV_FULL(s) (8 * (s))
#define LF_PT_KV_EMPTY(s) (8 * (LF_PT_NS + (s)))
#define LF_PT_LAND (16 * LF_PT_NS)
#define LF_PT_Q_FULL (LF_PT_LAND + 8)
#define LF_PT_S_FULL(g) (LF_PT_LAND + 16 + 8 * (g))
#define LF_PT_S_FREE(g) (LF_PT_LAND + 32 + 8 * (g))
#define LF_PT_P_FULL(g) (LF_PT_LAND + 48 + 8 * (g))
#define LF_PT_PV_DONE(g) (LF_PT_LAND + 64 + 8 * (g))
#define LF_PT_END (LF_PT_LAND + 80)
#define LF_PT_TMEM (LF_PT_LAND + 88)   // TMEM address
#define LF_PT_ABORT (LF_PT_LAND + 96)  // abort flag
#define LF_PT_MASK (LF_PT_LAND + 112)  // uint4 per ring slot: keys that count
static_assert(LF_PT_MASK % 16 == 0 && LF_PT_MASK + 16 * LF_PT_NS <= 512, "small shared data");
static_assert(LF_PT_SMEM <= 232448, "shared memory per CTA");

// TMEM columns of stream g
#define LF_PT_TS(g) (256 * (g))
#define LF_PT_TO(g) (256 * (g) + 128)
#define LF_PT_TP(g) (256 * (g) + 192)

// A row's reference may lag its running maximum by this much (log2): p stays
// below 2^8 and O is rescaled only when a score is far above everything before.
#define LF_PT_LAG 8.f
// One pair of exponentials in so many goes to the FMA pipe: the special
// function unit takes 8 cycles for a warp's 32, the rest of the work leaves
// the FMA pipe half idle.
#define LF_PT_FMA_EXP 0

// Warp-uniform bounded wait, inlined: the softmax warps hold a row of S in
// registers across it, which a call would push to local memory.
__device__ __forceinline__ bool lf_pt_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                           int32_t *status, int site) {
  bool ok = true;
  uint64_t t0 = 0;
  for (uint32_t it = 1; !lf_mbar_try(bar, parity); it++) {
    if (it & 255) continue;
    if (*abort_flag) {
      ok = false;
      break;
    }
    const uint64_t now = lf_globaltimer();
    if (t0 == 0) {
      t0 = now;
    } else if (now - t0 > LF_WAIT_NS) {
      *abort_flag = 1;
      lf_set_status(status, LF_ERR_DEVICE_TIMEOUT, site);
      ok = false;
      break;
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// The same for copies and products already issued, also after an abort.
__device__ __forceinline__ void lf_pt_drain(uint32_t bar, uint32_t parity, int32_t *status, int site) {
  const uint64_t t0 = lf_globaltimer();
  while (!lf_mbar_try(bar, parity)) {
    if (lf_globaltimer() - t0 > LF_WAIT_NS) {
      lf_set_status(status, LF_ERR_DEVICE_TIMEOUT, site);
      break;
    }
  }
}

// ---- pairs of float32 in one 64-bit register (sm_100 packed arithmetic)
typedef unsigned long long LfPair;
__device__ __forceinline__ LfPair lf_pair(float a, float b) {
  LfPair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ LfPair lf_pair_u(uint32_t a, uint32_t b) {
  LfPair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void lf_unpair(LfPair p, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ LfPair lf_fma2(LfPair a, LfPair b, LfPair c) {
  LfPair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ LfPair lf_add2(LfPair a, LfPair b) {
  LfPair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ LfPair lf_mul2(LfPair a, LfPair b) {
  LfPair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float lf_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float lf_max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 2^x of a pair on the FMA pipe, x <= 2^8 or NaN: x = n + f with n the nearest
// integer (adding 1.5 * 2^23 leaves n in the low bits), 2^f on [-1/2, 1/2] by
// the polynomial of degree 5 of least largest relative error (fitted by
// iterated reweighted least squares: 7.5e-8, 2.2e-7 with float32 roundings;
// ex2.approx: 2 units in the last place), times 2^n made from its bits.
// Results below 2^-126 come out as about 2^-126; NaN stays NaN.
__device__ __forceinline__ LfPair lf_exp2_fma(LfPair x) {
  float a, b;
  lf_unpair(x, a, b);
  x = lf_pair(lf_max_nan(a, -126.f), lf_max_nan(b, -126.f));
  const LfPair t = lf_add2(x, lf_pair(12582912.f, 12582912.f));
  const LfPair n = lf_add2(t, lf_pair(-12582912.f, -12582912.f));
  const LfPair f = lf_fma2(n, lf_pair(-1.f, -1.f), x);
  LfPair r = lf_fma2(lf_pair(1.3276461e-3f, 1.3276461e-3f), f, lf_pair(9.675541e-3f, 9.675541e-3f));
  r = lf_fma2(r, f, lf_pair(5.5507135e-2f, 5.5507135e-2f));
  r = lf_fma2(r, f, lf_pair(0.2402212f, 0.2402212f));
  r = lf_fma2(r, f, lf_pair(0.69314694f, 0.69314694f));
  r = lf_fma2(r, f, lf_pair(1.0000001f, 1.0000001f));
  float ta, tb;
  lf_unpair(t, ta, tb);
  return lf_mul2(r, lf_pair_u((__float_as_uint(ta) << 23) + 0x3f800000u, (__float_as_uint(tb) << 23) + 0x3f800000u));
}

struct LfPtParams {
  CUtensorMap k, v;  // the pools as rows of 64, boxes of box_rows rows
  LfPagedDev dev;
  const void *q;
  int box_rows;
};

template <typename T, int kF16>
__global__ void __launch_bounds__(LF_PT_THREADS, 1) lf_prefix_tc_kernel(const __grid_constant__ LfPtParams A) {
  extern __shared__ __align__(1024) uint8_t lf_smem_raw[];
  const LfPagedDev &P = A.dev;
  const uint32_t sbase = lf_smem(lf_smem_raw), bar = sbase + LF_PT_MISC;
  uint8_t *misc = lf_smem_raw + LF_PT_MISC;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + LF_PT_ABORT);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc + LF_PT_TMEM);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (sbase & 1023u) {  // 128-byte swizzled tiles need it
    if (tid == 0) lf_set_status(P.status, LF_ERR_UNSUPPORTED, 9000);
    return;
  }
  if (tid == 0) {
    for (int s = 0; s < LF_PT_NS; s++) {
      lf_mbar_init(bar + LF_PT_KV_FULL(s), 1);
      lf_mbar_init(bar + LF_PT_KV_EMPTY(s), 1);
    }
    lf_mbar_init(bar + LF_PT_LAND, 1);
    lf_mbar_init(bar + LF_PT_Q_FULL, 8);
    for (int g = 0; g < 2; g++) {
      lf_mbar_init(bar + LF_PT_S_FULL(g), 1);
      lf_mbar_init(bar + LF_PT_S_FREE(g), 4);
      lf_mbar_init(bar + LF_PT_P_FULL(g), 4);
      lf_mbar_init(bar + LF_PT_PV_DONE(g), 1);
    }
    lf_mbar_init(bar + LF_PT_END, 1);
    abort_flag[0] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(lf_smem(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  lf_tc_fence_before();
  __syncthreads();
  lf_tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int chunk = blockIdx.x, x0 = blockIdx.y * LF_PT_ROWS, hk = blockIdx.z;
  const int rows = P.B * P.G;
  const int j0 = chunk * P.chunk, j1 = min(P.prefix_len, j0 + P.chunk);
  const int n = (j1 - j0 + LF_PT_KEYS - 1) / LF_PT_KEYS;  // tiles, >= 1

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(LF_PT_REGS_FEW));
    if (warp == 8) {
      // ================================================== loader
      const int nbox = LF_PT_KEYS / A.box_rows, columns = (P.prefix_len + (1 << P.shift) - 1) >> P.shift;
      auto page_of = [&](int i) {  // this lane's box of tile i: a page of the table, -1 behind the prefix
        const int j = j0 + i * LF_PT_KEYS + lane * A.box_rows;
        return lane < nbox && j < j1 && lf_row_ok(columns, P.shift, j) ? P.prefix_table[j >> P.shift] : -1;
      };
      int page = page_of(0), lands = 0, issued = 0;
      bool ok = true, landing = false;
      for (int i = 0; i < n; i++) {
        const int s = i % LF_PT_NS, jt = j0 + i * LF_PT_KEYS, j = jt + lane * A.box_rows;
        if (i >= LF_PT_NS &&
            !lf_pt_wait(bar + LF_PT_KV_EMPTY(s), (i / LF_PT_NS - 1) & 1, abort_flag, P.status, 40)) {
          ok = false;
          break;
        }
        const bool want = lane < nbox && j < j1;
        const int row = want ? lf_row_in_page(page, P.num_pages, P.shift, P.Hkv, hk, j) : LF_ROW_NONE;
        if (row == LF_ROW_BAD) lf_set_status(P.status, LF_ERR_DEVICE_INPUT, LF_DET_PREFIX);
        if (i + 1 < n) page = page_of(i + 1);
        const uint32_t boxes = __ballot_sync(0xffffffffu, row >= 0);
        // keys that count: their box is there and they lie before the chunk's end
        uint32_t word = 0;
        if (lane < 4) {
          for (int k = 0; k < 32; k += 16)
            if (boxes >> ((32 * lane + k) / A.box_rows) & 1u) word |= 0xffffu << k;
          word &= lf_range_bits(0, j1 - 1 - jt, 32 * lane);
          reinterpret_cast<uint32_t *>(misc + LF_PT_MASK)[4 * s + lane] = word;
        }
        const bool full = __all_sync(0xffffffffu, lane >= 4 || word == 0xffffffffu);
        const uint32_t on = bar + (full ? LF_PT_KV_FULL(s) : LF_PT_LAND);
        __syncwarp();
        if (lane == 0 && boxes) lf_mbar_expect_tx(on, 2 * __popc(boxes) * A.box_rows * 128);
        __syncwarp();
        if (row >= 0) {
          const uint32_t to = sbase + LF_PT_K(s) + lane * A.box_rows * 128;
          lf_tma_load4(to, &A.k, on, 0, row, 0, 0);
          lf_tma_load4(to + 16384, &A.v, on, 0, row, 0, 0);
        }
        if (full) {
          issued = i + 1;
          continue;
        }
        // A tile with keys that do not count: their value rows become zeros (a
        // probability of 0 times a stray NaN would not), then the tile is full.
        if (boxes) {
          landing = true;
          if (!lf_pt_wait(bar + LF_PT_LAND, lands & 1, abort_flag, P.status, 41)) {
            ok = false;
            break;
          }
          landing = false;
          lands++;
        }
        for (int r0 = 0; r0 < LF_PT_KEYS; r0 += 4) {
          const int r = r0 + lane / 8;
          const uint32_t w = __shfl_sync(0xffffffffu, word, r / 32);
          if (!(w >> (r % 32) & 1u))
            *reinterpret_cast<uint4 *>(lf_smem_raw + LF_PT_V(s) + r * 128 + lane % 8 * 16) = uint4{0, 0, 0, 0};
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) lf_mbar_arrive(bar + LF_PT_KV_FULL(s));
        issued = i + 1;
      }
      if (!ok) {  // let the copies already issued land before the CTA exits
        for (int i = max(0, issued - LF_PT_NS); i < issued; i++)
          lf_pt_drain(bar + LF_PT_KV_FULL(i % LF_PT_NS), (i / LF_PT_NS) & 1, P.status, 42);
        if (landing) lf_pt_drain(bar + LF_PT_LAND, lands & 1, P.status, 43);
      }
    } else if (warp == 9) {
      // ================================================== MMA issuer
      const uint64_t dq = lf_sdesc(sbase + LF_PT_Q, 16, 1024);
      const uint64_t dk = lf_sdesc(sbase + LF_PT_K(0), 16, 1024);
      const uint64_t dv = lf_sdesc(sbase + LF_PT_V(0), 0, 1024);
      const uint32_t id_s = lf_idesc(kF16, LF_PT_KEYS, 0), id_pv = lf_idesc(kF16, LF_HD, 1);
      auto issue_s = [&](int i) {
        const int s = i % LF_PT_NS;
        if (!lf_pt_wait(bar + LF_PT_KV_FULL(s), (i / LF_PT_NS) & 1, abort_flag, P.status, 44)) return false;
        lf_tc_fence_after();
        lf_mma_s_phase(tmem + LF_PT_TS(i & 1), dq, dk + (uint64_t)(s * (32768 >> 4)), id_s, bar + LF_PT_S_FULL(i & 1));
        return true;
      };
      bool ok = lf_pt_wait(bar + LF_PT_Q_FULL, 0, abort_flag, P.status, 45);
      ok = ok && issue_s(0) && (n < 2 || issue_s(1));
      for (int i = 0; i < n && ok; i++) {
        const int g = i & 1, c = i >> 1, s = i % LF_PT_NS;
        if (i + 2 < n) {  // S of the stream's next tile, once this one is in registers
          ok = lf_pt_wait(bar + LF_PT_S_FREE(g), c & 1, abort_flag, P.status, 46);
          if (!ok) break;
          lf_tc_fence_after();
          ok = issue_s(i + 2);
          if (!ok) break;
        }
        ok = lf_pt_wait(bar + LF_PT_P_FULL(g), c & 1, abort_flag, P.status, 47);
        if (!ok) break;
        lf_tc_fence_after();
        lf_mma_ts_phase(tmem + LF_PT_TO(g), tmem + LF_PT_TP(g), dv + (uint64_t)(s * (32768 >> 4)), 2048 >> 4, id_pv,
                        0xffu, c > 0 ? 1u : 0u, bar + LF_PT_KV_EMPTY(s), bar + LF_PT_PV_DONE(g), 0u);
      }
      // every MMA of this warp has completed once the barrier flips (TMEM is
      // freed after this, also after an abort)
      lf_commit_w(bar + LF_PT_END);
      lf_pt_drain(bar + LF_PT_END, 0, P.status, 48);
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(LF_PT_REGS_MANY));
    // ================================================== softmax warps
    {  // the block's query rows, two threads a row; rows behind the last are zeros
      const int x = tid >> 1;
      const bool take = x0 + x < rows;
      const T *src = reinterpret_cast<const T *>(A.q);
      if (take) {
        const int m = x0 + x;
        src += (int64_t)(m / P.G) * P.qs[0] + (int64_t)(hk * P.G + m % P.G) * P.qs[1];
      }
#pragma unroll
      for (int k = 0; k < 4; k++) {
        const int u = (tid & 1) * 4 + k;
        const uint4 v = take ? *reinterpret_cast<const uint4 *>(src + u * 8) : uint4{0, 0, 0, 0};
        *reinterpret_cast<uint4 *>(lf_smem_raw + LF_PT_Q + x * 128 + ((u ^ (x & 7)) << 4)) = v;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) lf_mbar_arrive(bar + LF_PT_Q_FULL);
    }
    const int g = warp >> 2, quarter = warp & 3, x = x0 + quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_off + LF_PT_TS(g), tO = tmem + lane_off + LF_PT_TO(g);
    const uint32_t tP = tmem + lane_off + LF_PT_TP(g);
    const bool live = x0 + quarter * 32 < rows;  // the warp has rows: the others only keep step
    const float sl2 = P.scale_log2;
    const int steps = (n + 1 - g) / 2;  // this stream's tiles
    float m_ref = 0.f, l = 0.f;
    bool fresh = true, ok = true;  // fresh: no key has counted yet
    for (int c = 0; c < steps; c++) {
      const int s = (2 * c + g) % LF_PT_NS;
      ok = lf_pt_wait(bar + LF_PT_S_FULL(g), c & 1, abort_flag, P.status, 49);
      if (!ok) break;
      lf_tc_fence_after();
      uint32_t v[4][32];
      if (live) {
#pragma unroll
        for (int k = 0; k < 4; k++) lf_tmem_ld32_nowait(tS + 32 * k, v[k]);
        lf_tmem_wait_ld_regs(v[0]);
#pragma unroll
        for (int k = 1; k < 4; k++) lf_tmem_pin_regs(v[k]);
      }
      lf_tc_fence_before();
      __syncwarp();
      if (lane == 0) lf_mbar_arrive(bar + LF_PT_S_FREE(g));  // S is in registers
      bool waited = c == 0;
      if (live) {
        // the tile's mask, behind the barrier that its writer arrived at
        ok = lf_pt_wait(bar + LF_PT_KV_FULL(s), ((2 * c + g) / LF_PT_NS) & 1, abort_flag, P.status, 50);
        if (!ok) break;
        const uint4 mask = *reinterpret_cast<const uint4 *>(misc + LF_PT_MASK + 16 * s);
        const uint32_t w[4] = {mask.x, mask.y, mask.z, mask.w};
        const bool all = (w[0] & w[1] & w[2] & w[3]) == 0xffffffffu;
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (all) {
#pragma unroll
          for (int e = 0; e < 32; e += 2)
#pragma unroll
            for (int k = 0; k < 4; k++)
              mx[k] = lf_max3(mx[k], __uint_as_float(v[k][e]), __uint_as_float(v[k][e + 1]));
        } else {
#pragma unroll
          for (int k = 0; k < 4; k++)
#pragma unroll
            for (int e = 0; e < 32; e++) mx[k] = fmaxf(mx[k], (w[k] >> e & 1u) ? __uint_as_float(v[k][e]) : -INFINITY);
        }
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
        if (fresh && (w[0] | w[1] | w[2] | w[3]) != 0u) {
          // O holds nothing yet (or products of zeros): the reference moves freely
          m_ref = mt == -INFINITY ? 0.f : mt;
          fresh = false;
        } else if (__any_sync(0xffffffffu, mt > m_ref + LF_PT_LAG)) {
          ok = waited || lf_pt_wait(bar + LF_PT_PV_DONE(g), (c - 1) & 1, abort_flag, P.status, 51);
          if (!ok) break;
          waited = true;
          lf_tc_fence_after();
          const bool up = mt > m_ref + LF_PT_LAG;
          const float f = up ? lf_ex2(m_ref - mt) : 1.f;
          if (up) m_ref = mt;
          l *= f;
#pragma unroll 1
          for (int e = 0; e < LF_HD; e += 16) {
            uint32_t ov[16];
            lf_tmem_ld16(tO + e, ov);
#pragma unroll
            for (int k = 0; k < 16; k++) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * f);
            lf_tmem_st16(tO + e, ov);
          }
        }
        if (!waited) {  // the stream's last product has read P
          ok = lf_pt_wait(bar + LF_PT_PV_DONE(g), (c - 1) & 1, abort_flag, P.status, 52);
          if (!ok) break;
          lf_tc_fence_after();
        }
        // P is rounded to the 16-bit type for the product with V (p < 2^8,
        // half a step relative each); the row sum keeps the unrounded values
        if (all) {
          LfPair sums[2] = {lf_pair(0.f, 0.f), lf_pair(0.f, 0.f)};
          const LfPair sl2p = lf_pair(sl2, sl2), refp = lf_pair(-m_ref, -m_ref);
#pragma unroll
          for (int k = 0; k < 4; k++) {
            uint32_t pw[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              LfPair x2 = lf_fma2(lf_pair_u(v[k][e], v[k][e + 1]), sl2p, refp);
              float p0, p1;
              if (LF_PT_FMA_EXP && e / 2 % LF_PT_FMA_EXP == LF_PT_FMA_EXP - 1) {
                x2 = lf_exp2_fma(x2);
                lf_unpair(x2, p0, p1);
              } else {
                lf_unpair(x2, p0, p1);
                p0 = lf_ex2(p0);
                p1 = lf_ex2(p1);
                x2 = lf_pair(p0, p1);
              }
              sums[e / 2 % 2] = lf_add2(sums[e / 2 % 2], x2);
              pw[e / 2] = lf_pack2<kF16>(p0, p1);
            }
            lf_tmem_st16(tP + 16 * k, pw);
          }
          float s0, s1;
          lf_unpair(lf_add2(sums[0], sums[1]), s0, s1);
          l += s0 + s1;
        } else {
#pragma unroll
          for (int k = 0; k < 4; k++) {
            uint32_t pw[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float p0 = (w[k] >> e & 1u) ? lf_ex2(fmaf(__uint_as_float(v[k][e]), sl2, -m_ref)) : 0.f;
              const float p1 = (w[k] >> e & 2u) ? lf_ex2(fmaf(__uint_as_float(v[k][e + 1]), sl2, -m_ref)) : 0.f;
              l += p0 + p1;
              pw[e / 2] = lf_pack2<kF16>(p0, p1);
            }
            lf_tmem_st16(tP + 16 * k, pw);
          }
        }
        lf_tmem_wait_st();
      }
      lf_tc_fence_before();
      __syncwarp();
      if (lane == 0) lf_mbar_arrive(bar + LF_PT_P_FULL(g));
    }
    if (ok && live) {
      const size_t at = ((size_t)hk * rows + x) * P.nch + 2 * chunk + g;
      if (steps > 0) {
        ok = lf_pt_wait(bar + LF_PT_PV_DONE(g), (steps - 1) & 1, abort_flag, P.status, 53);
        lf_tc_fence_after();
      }
      if (ok) {
        uint32_t ra[32], rb[32];
        if (steps > 0) {
          lf_tmem_ld32_nowait(tO, ra);
          lf_tmem_ld32_nowait(tO + 32, rb);
          lf_tmem_wait_ld_regs(ra);
          lf_tmem_pin_regs(rb);
        }
        if (x < rows) {
          float4 *dst = reinterpret_cast<float4 *>(P.part_acc + at * LF_HD);
#pragma unroll
          for (int k = 0; k < 8; k++) {
            const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
            const float4 a = make_float4(__uint_as_float(ra[4 * k]), __uint_as_float(ra[4 * k + 1]),
                                         __uint_as_float(ra[4 * k + 2]), __uint_as_float(ra[4 * k + 3]));
            const float4 b = make_float4(__uint_as_float(rb[4 * k]), __uint_as_float(rb[4 * k + 1]),
                                         __uint_as_float(rb[4 * k + 2]), __uint_as_float(rb[4 * k + 3]));
            dst[k] = fresh ? z : a;
            dst[8 + k] = fresh ? z : b;
          }
          P.part_ml[at] = make_float2(fresh ? -INFINITY : m_ref, l);
        }
      }
    }
    lf_tmem_wait_st();  // (an abort may leave stores in flight)
  }
  lf_tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    lf_tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// ----------------------------------------------------------------- host side

// Chunks: one CTA per SM of a full B200 (148, fixed: the workspace size is a
// function of the params alone) if the rows and heads leave that many, whole
// tiles each; two streams, so two parts per chunk.
void lf_prefix_tc_plan(LfPagedDev &d) {
  const int tiles = (d.prefix_len + LF_PT_KEYS - 1) / LF_PT_KEYS;
  const int64_t blocks = (int64_t)d.Hkv * (((int64_t)d.B * d.G + LF_PT_ROWS - 1) / LF_PT_ROWS);
  int64_t want = 148 / blocks;
  if (want < 1) want = 1;
  if (want > LF_PART_MAX / 2) want = LF_PART_MAX / 2;
  if (want > tiles) want = tiles;
  const int per = (int)((tiles + want - 1) / want);
  d.chunk = per * LF_PT_KEYS;
  d.nch = 2 * ((tiles + per - 1) / per);
}

template <typename T, int kF16>
static cudaError_t lf_launch_prefix_tc_t(const LfPagedLaunch &L, const void *q, const void *kp, const void *vp) {
  LfPtParams A;
  A.dev = L.dev;
  A.q = q;
  const LfPagedDev &P = L.dev;
  A.box_rows = P.shift >= 7 ? LF_PT_KEYS : 1 << P.shift;
  const uint64_t rows = (uint64_t)P.num_pages * P.Hkv << P.shift;
  if (!lf_make_map(&A.k, kF16, kp, rows, 1, 1, 128, rows * 128, rows * 128, A.box_rows) ||
      !lf_make_map(&A.v, kF16, vp, rows, 1, 1, 128, rows * 128, rows * 128, A.box_rows))
    return cudaErrorInvalidValue;
  const void *fn = (const void *)lf_prefix_tc_kernel<T, kF16>;
  const cudaError_t e = lf_kernel_smem(fn, LF_PT_SMEM);
  if (e != cudaSuccess) return e;
  const int64_t rblocks = ((int64_t)P.B * P.G + LF_PT_ROWS - 1) / LF_PT_ROWS;
  if (rblocks > 65535) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(P.nch / 2), (unsigned)rblocks, (unsigned)P.Hkv);
  cfg.blockDim = dim3(LF_PT_THREADS);
  cfg.dynamicSmemBytes = LF_PT_SMEM;
  cfg.stream = L.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void *args[] = {&A};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

cudaError_t lf_launch_prefix_tc(const LfPagedLaunch &L, const void *q, const void *kp, const void *vp) {
  return L.dtype == LF_F16 ? lf_launch_prefix_tc_t<__half, 1>(L, q, kp, vp)
                           : lf_launch_prefix_tc_t<__nv_bfloat16, 0>(L, q, kp, vp);
}
