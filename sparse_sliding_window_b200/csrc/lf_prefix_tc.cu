// lf_prefix_tc.cu -- the shared prefix for many query rows (bf16, f16): the
// tensor-core (tcgen05) form of the prefix kernel.
//
// A CTA takes 128 query rows (of the B * G of a key/value head) and one chunk
// of the prefix.  Its 64-key tiles go to three streams in turn; per stream four
// softmax warps, one row per thread, with S, O and P in TMEM:
//   warps 0-11  softmax of streams 0, 1, 2 (four each)
//   warp 12     loads K and V tiles by TMA, a box per page, into a ring
//   warps 13-15 issue S = Q K^T (128 x 64 x 64) and O += P V (128 x 64 x 64) of
//               their stream, P as two 16-bit numbers (one warp for all three
//               needs about 780 cycles a tile for its waits and issues, more than
//               the softmax)
// What bounds it is the softmax: 128 x 64 exponentials a tile at 16 a cycle
// and SM, and, around them, a chain of barrier and TMEM waits of about 1200
// cycles per step of a stream.  S is read into registers whole and handed back
// at once, so the stream's next S is computed meanwhile; three streams of short
// tiles (three softmax warps per scheduler) cover the chain better than two of
// 128 keys, which is what TMEM would hold instead.  The streams' results are
// merged from TMEM at the end: one (sum of p v, max, sum of p) per row and
// chunk.
#include <cuda.h>

#include "lf_paged.cuh"
#include "lf_ptx.cuh"
#include "lf_tc.cuh"

#define LF_PT_ROWS 128
#define LF_PT_KEYS 64
#define LF_PT_G 3        // streams
#define LF_PT_SOFT (128 * LF_PT_G)
#define LF_PT_THREADS (LF_PT_SOFT + 32 * (1 + LF_PT_G))
#define LF_PT_NS 9       // K/V tiles in the ring (16 KB each; with 8 of them 0.5 of 43 us slower, with 10 the same)
#define LF_PT_TILE (LF_PT_KEYS * 128)

#define LF_PT_Q 0
#define LF_PT_K(s) (16384 + (s)*2 * LF_PT_TILE)
#define LF_PT_V(s) (LF_PT_K(s) + LF_PT_TILE)
#define LF_PT_L(g) (LF_PT_K(LF_PT_NS) + (g)*LF_PT_ROWS * 128)  // P's second numbers, per stream, laid out like Q
#define LF_PT_MISC LF_PT_L(LF_PT_G)
// barriers, from LF_PT_MISC
#define LF_PT_KV_FULL(s) (8 * (s))
#define LF_PT_KV_EMPTY(s) (8 * (LF_PT_NS + (s)))
#define LF_PT_LAND (16 * LF_PT_NS)
#define LF_PT_Q_FULL (LF_PT_LAND + 8)
#define LF_PT_END (LF_PT_LAND + 16)
#define LF_PT_S_FULL(g) (LF_PT_LAND + 24 + 8 * (g))
#define LF_PT_S_FREE(g) (LF_PT_S_FULL(LF_PT_G) + 8 * (g))
#define LF_PT_P_FULL(g) (LF_PT_S_FREE(LF_PT_G) + 8 * (g))
#define LF_PT_PV_DONE(g) (LF_PT_P_FULL(LF_PT_G) + 8 * (g))
#define LF_PT_TMEM LF_PT_PV_DONE(LF_PT_G)   // TMEM address
#define LF_PT_ABORT (LF_PT_TMEM + 8)        // abort flag
#define LF_PT_MASK (LF_PT_ABORT + 8)        // uint2 per ring slot: keys that count
#define LF_PT_ML (LF_PT_MASK + 8 * LF_PT_NS)  // float2 [streams][128]: max and sum of a row
#define LF_PT_SMEM (LF_PT_MISC + LF_PT_ML + LF_PT_G * 128 * 8)
static_assert(LF_PT_SMEM <= 232448, "shared memory per CTA");
// rows of the merged output on their way out, in the ring: [8 warps][32][36]
static_assert(8 * 32 * 36 * 4 <= LF_PT_MISC - LF_PT_K(0), "staging");

// TMEM columns of stream g
#define LF_PT_TS(g) (160 * (g))
#define LF_PT_TO(g) (160 * (g) + 64)
#define LF_PT_TP(g) (160 * (g) + 128)

// A row's reference may lag its running maximum by this much (log2): p stays
// below 2^8 and O is rescaled only when a score is far above everything before.
#define LF_PT_LAG 8.f
#define LF_PT_NEAR 1048576.f

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

__device__ __forceinline__ float lf_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// D (+)= A B with A (128 x 64, laid out like Q) and B (64 keys of V) in shared
// memory: four K = 16 steps, no commit; acc = 0: the first step overwrites D.
__device__ __forceinline__ void lf_pt_mma_low(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred e, pa;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
      "add.s64 b1, %2, 128;\n\tadd.s64 b2, %2, 256;\n\tadd.s64 b3, %2, 384;\n\t"
      "setp.ne.b32 pa, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, pa;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
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
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the decode kernel relies on it
    return;
  }
  if (tid == 0) {
    for (int s = 0; s < LF_PT_NS; s++) {
      lf_mbar_init(bar + LF_PT_KV_FULL(s), 1);
      lf_mbar_init(bar + LF_PT_KV_EMPTY(s), 1);
    }
    lf_mbar_init(bar + LF_PT_LAND, 1);
    lf_mbar_init(bar + LF_PT_Q_FULL, 4 * LF_PT_G);
    lf_mbar_init(bar + LF_PT_END, LF_PT_G);
    for (int g = 0; g < LF_PT_G; g++) {
      lf_mbar_init(bar + LF_PT_S_FULL(g), 1);
      lf_mbar_init(bar + LF_PT_S_FREE(g), 4);
      lf_mbar_init(bar + LF_PT_P_FULL(g), 4);
      lf_mbar_init(bar + LF_PT_PV_DONE(g), 1);
    }
    abort_flag[0] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == LF_PT_SOFT / 32 + 1) {
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

  if (warp >= LF_PT_SOFT / 32) {
    if (warp == LF_PT_SOFT / 32) {
      // ================================================== loader
      const int bshift = 31 - __clz(A.box_rows), nbox = LF_PT_KEYS >> bshift;
      const int columns = (P.prefix_len + (1 << P.shift) - 1) >> P.shift;
      // The pool rows of 32 boxes at a time (lane k: box 32 grp + k of the
      // chunk), their table entries one group ahead: what is left per tile is
      // short, or the loads would not keep up (1000 cycles a tile when it
      // looked each page up by itself, 1.5 times what the softmax takes).
      const int nboxes = (j1 - j0 + A.box_rows - 1) >> bshift;
      auto entries = [&](int grp) {
        const int j = j0 + ((32 * grp + lane) << bshift);
        return 32 * grp + lane < nboxes && lf_row_ok(columns, P.shift, j) ? P.prefix_table[j >> P.shift] : -1;
      };
      int ahead = entries(0), at = 32, grp = -1, rowsv = LF_ROW_NONE, slot = 0, round = 0, lands = 0, issued = 0;
      uint32_t there = 0;  // which of the group's boxes are
      bool ok = true, landing = false;
      for (int i = 0; i < n; i++, at += nbox) {
        if (at == 32) {
          at = 0;
          grp++;
          const int j = j0 + ((32 * grp + lane) << bshift);
          rowsv = 32 * grp + lane < nboxes ? lf_row_in_page(ahead, P.num_pages, P.shift, P.Hkv, hk, j) : LF_ROW_NONE;
          if (rowsv == LF_ROW_BAD) lf_set_status(P.status, LF_ERR_DEVICE_INPUT, LF_DET_PREFIX);
          there = __ballot_sync(0xffffffffu, rowsv >= 0);
          ahead = entries(grp + 1);
        }
        const int s = slot;
        if (round > 0 && !lf_pt_wait(bar + LF_PT_KV_EMPTY(s), (round - 1) & 1, abort_flag, P.status, 40)) {
          ok = false;
          break;
        }
        if (++slot == LF_PT_NS) {
          slot = 0;
          round++;
        }
        const int left = j1 - j0 - i * LF_PT_KEYS;  // keys of the chunk from here on
        const uint32_t every = (1u << nbox) - 1u, boxes = there >> at & every;
        const bool full = boxes == every && left >= LF_PT_KEYS;
        const uint32_t on = bar + (full ? LF_PT_KV_FULL(s) : LF_PT_LAND);
        const int row = __shfl_sync(0xffffffffu, rowsv, at + lane);
        // keys that count: their box is there and they lie before the chunk's end
        uint32_t word = 0xffffffffu;
        if (!full) {
          word = 0;
          for (int k = 0; k < 32; k += 16)
            if (boxes >> ((32 * (lane & 1) + k) >> bshift) & 1u) word |= 0xffffu << k;
          word &= lf_range_bits(0, left - 1, 32 * (lane & 1));
        }
        if (lane < 2) reinterpret_cast<uint32_t *>(misc + LF_PT_MASK)[2 * s + lane] = word;
        __syncwarp();  // the mask before the arrival
        if (lane == 0 && boxes) lf_mbar_expect_tx(on, 2 * __popc(boxes) * A.box_rows * 128);
        if (boxes >> lane & 1u) {
          const uint32_t to = sbase + LF_PT_K(s) + ((lane << bshift) * 128);
          lf_tma_load4(to, &A.k, on, 0, row, 0, 0);
          lf_tma_load4(to + LF_PT_TILE, &A.v, on, 0, row, 0, 0);
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
          const uint32_t w = __shfl_sync(0xffffffffu, word, r / 32);  // lanes 0 and 1 hold the words
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
    } else {
      // ================================================== MMA issuer
      const uint64_t dq = lf_sdesc(sbase + LF_PT_Q, 16, 1024);
      const uint64_t dk = lf_sdesc(sbase + LF_PT_K(0), 16, 1024);
      const uint64_t dv = lf_sdesc(sbase + LF_PT_V(0), 0, 1024);
      const uint32_t id_s = lf_idesc(kF16, LF_PT_KEYS, 0), id_pv = lf_idesc(kF16, LF_HD, 1);
      const uint64_t slot = 2 * LF_PT_TILE >> 4;
      const int g = warp - LF_PT_SOFT / 32 - 1;
      const uint64_t dl = lf_sdesc(sbase + LF_PT_L(g), 16, 1024);
      auto issue_s = [&](int i) {
        const int s = i % LF_PT_NS;
        if (!lf_pt_wait(bar + LF_PT_KV_FULL(s), (i / LF_PT_NS) & 1, abort_flag, P.status, 44)) return false;
        lf_tc_fence_after();
        lf_mma_s_phase(tmem + LF_PT_TS(g), dq, dk + s * slot, id_s, bar + LF_PT_S_FULL(g));
        return true;
      };
      bool ok = lf_pt_wait(bar + LF_PT_Q_FULL, 0, abort_flag, P.status, 45);
      if (ok && g < n) ok = issue_s(g);
      for (int i = g, c = 0; i < n && ok; i += LF_PT_G, c++) {
        const int s = i % LF_PT_NS;
        if (i + LF_PT_G < n) {  // S of the stream's next tile, once this one is in registers
          ok = lf_pt_wait(bar + LF_PT_S_FREE(g), c & 1, abort_flag, P.status, 46);
          if (!ok) break;
          lf_tc_fence_after();
          ok = issue_s(i + LF_PT_G);
          if (!ok) break;
        }
        ok = lf_pt_wait(bar + LF_PT_P_FULL(g), c & 1, abort_flag, P.status, 47);
        if (!ok) break;
        lf_tc_fence_after();
        lf_pt_mma_low(tmem + LF_PT_TO(g), dl, dv + s * slot, id_pv, c > 0 ? 1u : 0u);
        lf_mma_ts_phase(tmem + LF_PT_TO(g), tmem + LF_PT_TP(g), dv + s * slot, 2048 >> 4, id_pv,
                        (1u << (LF_PT_KEYS / 16)) - 1u, 1u, bar + LF_PT_KV_EMPTY(s),
                        bar + LF_PT_PV_DONE(g), 0u);
      }
      // every MMA of the three warps has completed once the barrier flips (TMEM is
      // freed after this, also after an abort)
      lf_commit_w(bar + LF_PT_END);
      lf_pt_drain(bar + LF_PT_END, 0, P.status, 48);
      __syncwarp();
    }
  } else {
    // ================================================== softmax warps
    // the block's query rows, in 16-byte units; rows behind the last are zeros
    for (int e = tid; e < LF_PT_ROWS * 8; e += LF_PT_SOFT) {
      const int x = e / 8, u = e % 8, m = x0 + x;
      uint4 v = {0, 0, 0, 0};
      if (m < rows)
        v = *reinterpret_cast<const uint4 *>(reinterpret_cast<const T *>(A.q) + (int64_t)(m / P.G) * P.qs[0] +
                                             (int64_t)(hk * P.G + m % P.G) * P.qs[1] + u * 8);
      *reinterpret_cast<uint4 *>(lf_smem_raw + LF_PT_Q + x * 128 + ((u ^ (x & 7)) << 4)) = v;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) lf_mbar_arrive(bar + LF_PT_Q_FULL);

    const int g = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t tq = tmem + ((uint32_t)(quarter * 32) << 16);  // this warp's lanes
    const uint32_t tS = tq + LF_PT_TS(g), tO = tq + LF_PT_TO(g), tP = tq + LF_PT_TP(g);
    const bool live = x0 + quarter * 32 < rows;  // the warp has rows: the others only keep step
    const float sl2 = P.scale_log2;
    const LfPair sl2p = lf_pair(sl2, sl2);
    float m_ref = 0.f, l = 0.f;
    bool fresh = true, ok = true;  // fresh: no score above -inf yet
    int c = 0;                     // the stream's tile
    for (int i = g; i < n; i += LF_PT_G, c++) {
      const int s = i % LF_PT_NS;
      ok = lf_pt_wait(bar + LF_PT_S_FULL(g), c & 1, abort_flag, P.status, 49);
      if (!ok) break;
      lf_tc_fence_after();
      uint32_t v[2][32];
      if (live) {
        lf_tmem_ld32_nowait(tS, v[0]);
        lf_tmem_ld32_nowait(tS + 32, v[1]);
        lf_tmem_wait_ld_regs(v[0]);
        lf_tmem_pin_regs(v[1]);
      }
      lf_tc_fence_before();
      __syncwarp();
      if (lane == 0) lf_mbar_arrive(bar + LF_PT_S_FREE(g));  // S is in registers
      if (live) {
        // the tile's mask, behind the barrier that its writer arrived at
        ok = lf_pt_wait(bar + LF_PT_KV_FULL(s), (i / LF_PT_NS) & 1, abort_flag, P.status, 50);
        if (!ok) break;
        const uint2 mask = *reinterpret_cast<const uint2 *>(misc + LF_PT_MASK + 8 * s);
        const uint32_t w[2] = {mask.x, mask.y};
        const bool all = (w[0] & w[1]) == 0xffffffffu;
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (all) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
#pragma unroll
            for (int k = 0; k < 4; k++)
              mx[k] = lf_max3(mx[k], __uint_as_float(v[k & 1][e + (k & 2)]), __uint_as_float(v[k & 1][e + (k & 2) + 1]));
        } else {
#pragma unroll
          for (int k = 0; k < 2; k++)
#pragma unroll
            for (int e = 0; e < 32; e++) mx[k] = fmaxf(mx[k], (w[k] >> e & 1u) ? __uint_as_float(v[k][e]) : -INFINITY);
        }
        const float mt = __fmul_rn(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), sl2);
        if (c > 0) {  // the stream's last product has read P and is in O
          ok = lf_pt_wait(bar + LF_PT_PV_DONE(g), (c - 1) & 1, abort_flag, P.status, 51);
          if (!ok) break;
          lf_tc_fence_after();
        }
        if (fresh && mt > -INFINITY) {
          // O holds nothing yet (or products of zeros): the reference moves freely
          m_ref = mt;
          fresh = false;
        }
        const bool up = !fresh && mt - m_ref > LF_PT_LAG;
        if (__any_sync(0xffffffffu, up)) {
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
        // P enters the product with V as two 16-bit numbers: the first through
        // TMEM, the second, for which TMEM has no room, through shared memory.
        // (One number alone: 128 x 16/4 heads on 16384 rows 38.4 us instead of
        // 43.2, 64 x 12 heads on 4096 rows 25.8 instead of 27.8.)
        uint8_t *low = lf_smem_raw + LF_PT_L(g) + row * 128;
        // The scaling and the subtraction of the reference are one operation where
        // the reference's own rounding is far below 1 (at most 2^-4).  Beyond, the
        // scaled score is rounded first, as the reference was: the difference would
        // else be whole powers of two, and p infinite or 0 in every key.
        if (all && __all_sync(0xffffffffu, fabsf(m_ref) < LF_PT_NEAR)) {
          LfPair sums[2] = {lf_pair(0.f, 0.f), lf_pair(0.f, 0.f)};
          const LfPair refp = lf_pair(-m_ref, -m_ref);
#pragma unroll
          for (int k = 0; k < 2; k++) {
            uint32_t pw[16], pl[4];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float p0, p1;
              lf_unpair(lf_fma2(lf_pair_u(v[k][e], v[k][e + 1]), sl2p, refp), p0, p1);
              p0 = lf_ex2(p0);
              p1 = lf_ex2(p1);
              sums[e / 2 % 2] = lf_add2(sums[e / 2 % 2], lf_pair(p0, p1));
              lf_p_split<kF16, true>(p0, p1, pw[e / 2], pl[e / 2 % 4]);
              if (e % 8 == 6)
                *reinterpret_cast<uint4 *>(low + (((4 * k + e / 8) ^ (row & 7)) << 4)) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
            }
            lf_tmem_st16(tP + 16 * k, pw);
          }
          float s0, s1;
          lf_unpair(lf_add2(sums[0], sums[1]), s0, s1);
          l += s0 + s1;
        } else {
#pragma unroll
          for (int k = 0; k < 2; k++) {
            uint32_t pw[16], pl[4];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float p0 = (w[k] >> e & 1u) ? lf_ex2(__fmul_rn(__uint_as_float(v[k][e]), sl2) - m_ref) : 0.f;
              const float p1 = (w[k] >> e & 2u) ? lf_ex2(__fmul_rn(__uint_as_float(v[k][e + 1]), sl2) - m_ref) : 0.f;
              l += p0 + p1;
              lf_p_split<kF16, true>(p0, p1, pw[e / 2], pl[e / 2 % 4]);
              if (e % 8 == 6)
                *reinterpret_cast<uint4 *>(low + (((4 * k + e / 8) ^ (row & 7)) << 4)) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
            }
            lf_tmem_st16(tP + 16 * k, pw);
          }
        }
        lf_tmem_wait_st();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      } else if (c > 0) {
        // A warp without rows must not arrive for this tile while the others
        // still owe the last one: its arrival would complete their phase.
        ok = lf_pt_wait(bar + LF_PT_PV_DONE(g), (c - 1) & 1, abort_flag, P.status, 54);
        if (!ok) break;
      }
      lf_tc_fence_before();
      __syncwarp();
      if (lane == 0) lf_mbar_arrive(bar + LF_PT_P_FULL(g));
    }
    // ---- the streams' results, merged from TMEM: streams 0 and 1 take 32
    // channels each (a warp reaches the same lanes of every stream)
    if (ok && c > 0) ok = lf_pt_wait(bar + LF_PT_PV_DONE(g), (c - 1) & 1, abort_flag, P.status, 52);
    lf_tmem_wait_st();  // (an abort may leave stores in flight)
    float2 *s_ml = reinterpret_cast<float2 *>(misc + LF_PT_ML);
    s_ml[g * 128 + row] = make_float2(fresh ? -INFINITY : m_ref, l);  // (l of NaN scores stays)
    lf_tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"n"(LF_PT_SOFT) : "memory");  // every softmax warp comes here
    lf_tc_fence_after();
    if (g < 2 && live && *abort_flag == 0) {
      float M = -INFINITY, L = 0.f, acc[32];
#pragma unroll
      for (int k = 0; k < LF_PT_G; k++) M = fmaxf(M, s_ml[k * 128 + row].x);
#pragma unroll
      for (int e = 0; e < 32; e++) acc[e] = 0.f;
#pragma unroll
      for (int k = 0; k < LF_PT_G; k++) {
        const float2 ml = s_ml[k * 128 + row];
        const float f = ml.x == -INFINITY ? 0.f : lf_ex2(ml.x - M);
        L += ml.y * f;
        if (k < n) {  // a stream without tiles has nothing in TMEM
          uint32_t ov[32];
          lf_tmem_ld32_nowait(tq + LF_PT_TO(k) + 32 * g, ov);
          lf_tmem_wait_ld_regs(ov);
          const float fo = kF16 ? f * (1.f / LF_P_SCALE) : f;
#pragma unroll
          for (int e = 0; e < 32; e++) acc[e] = fmaf(__uint_as_float(ov[e]), fo, acc[e]);
        }
      }
      // through shared memory (the ring is done with), so that whole rows leave
      float *stage = reinterpret_cast<float *>(lf_smem_raw + LF_PT_K(0)) + warp * 32 * 36;
#pragma unroll
      for (int e = 0; e < 32; e += 4)
        *reinterpret_cast<float4 *>(stage + lane * 36 + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
      __syncwarp();
      const size_t first = (size_t)hk * rows + x0 + quarter * 32;
#pragma unroll
      for (int r0 = 0; r0 < 32; r0 += 4) {
        const int r = r0 + lane / 8;
        if (x0 + quarter * 32 + r < rows)
          *reinterpret_cast<float4 *>(P.part_acc + ((first + r) * P.nch + chunk) * LF_HD + 32 * g + lane % 8 * 4) =
              *reinterpret_cast<const float4 *>(stage + r * 36 + lane % 8 * 4);
      }
      if (g == 0 && x0 + row < rows) P.part_ml[(first + lane) * P.nch + chunk] = make_float2(M, L);
    }
  }
  lf_tc_fence_before();
  __syncthreads();
  if (warp == LF_PT_SOFT / 32 + 1) {
    lf_tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// ----------------------------------------------------------------- host side

// Chunks: one CTA per SM of a full B200 (148, fixed: the workspace size is a
// function of the params alone) if the rows and heads leave that many, whole
// tiles each.
void lf_prefix_tc_plan(LfPagedDev &d) {
  const int tiles = (d.prefix_len + LF_PT_KEYS - 1) / LF_PT_KEYS;
  const int64_t blocks = (int64_t)d.Hkv * (((int64_t)d.B * d.G + LF_PT_ROWS - 1) / LF_PT_ROWS);
  int64_t want = 148 / blocks;
  if (want < 1) want = 1;
  if (want > LF_PART_MAX) want = LF_PART_MAX;
  if (want > tiles) want = tiles;
  const int per = (int)((tiles + want - 1) / want);
  d.chunk = per * LF_PT_KEYS;
  d.nch = (tiles + per - 1) / per;
}

template <typename T, int kF16>
static cudaError_t lf_launch_prefix_tc_t(const LfPagedLaunch &L, const void *q, const void *kp, const void *vp) {
  cudaError_t e = lf_need_context();
  if (e != cudaSuccess) return e;
  LfPtParams A;
  A.dev = L.dev;
  A.q = q;
  const LfPagedDev &P = L.dev;
  A.box_rows = 1 << P.shift < LF_PT_KEYS ? 1 << P.shift : LF_PT_KEYS;
  const uint64_t rows = (uint64_t)P.num_pages * P.Hkv << P.shift;
  if (!lf_make_map(&A.k, kF16, kp, rows, 1, 1, 128, rows * 128, rows * 128, A.box_rows) ||
      !lf_make_map(&A.v, kF16, vp, rows, 1, 1, 128, rows * 128, rows * 128, A.box_rows))
    return cudaErrorInvalidValue;
  const void *fn = (const void *)lf_prefix_tc_kernel<T, kF16>;
  e = lf_kernel_smem(fn, LF_PT_SMEM);
  if (e != cudaSuccess) return e;
  const int64_t rblocks = ((int64_t)P.B * P.G + LF_PT_ROWS - 1) / LF_PT_ROWS;
  if (rblocks > 65535) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)P.nch, (unsigned)rblocks, (unsigned)P.Hkv);
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
