// lf_paged.cuh -- host/device interface of the rotation, the paged cache
// append and the paged decode (include/lf_paged.h).
#pragma once

#include "lf_common.cuh"
#include "lf_paged.h"
#include "lf_pages.cuh"
#include "lf_status.cuh"

#define LF_ROPE_MAX_PAIRS 32
#define LF_ROPE_MAX_AXES 4
#define LF_ROPE_MAX_JOBS 8

// Turns (angle / 2 pi) per position of each pair, as hi + lo.
struct LfRopeDev {
  int pairs, interleaved, n_axes;
  float sign;  // +1 forward, -1 backward
  double hi[LF_ROPE_MAX_PAIRS], lo[LF_ROPE_MAX_PAIRS];
  uint8_t axis[LF_ROPE_MAX_PAIRS];
};

// One tensor of a rotation or append: out == nullptr with pool != nullptr
// writes head h of a token to its row of that pool.
struct LfRopeJob {
  const void *x;
  void *out;
  void *pool;
  int heads;
  int rotate;
  int64_t xs[3], os[3];  // batch, head, token
};

struct LfRopeArgs {
  LfRopeDev r;
  LfRopeJob job[LF_ROPE_MAX_JOBS];
  int heads_total;
  int heads_per_block;  // heads a thread works through
  int n;                // tokens per sequence (rotation)
  int64_t tokens;       // tokens in all
  const int32_t *positions;
  // append
  int B, Hkv, shift, num_pages, max_pages, pos_offset;
  const int32_t *cu, *lengths, *table;
  int32_t *status;
};

// nch: parts that the prefix kernel leaves per row; chunk: keys a block takes;
// direct: no prefix kernel (nch = 0), the decode kernel reads the prefix itself.
struct LfPagedDev {
  int B, H, Hkv, G;      // G = H / Hkv
  int shift, num_pages, max_pages;
  int window, prefix_len, nch, chunk, direct;
  float scale_log2;
  int64_t qs[2];         // q strides: sequence, head
  const int32_t *table, *lengths, *prefix_table;
  int32_t *status;
  float *part_acc;       // [Hkv * B * G][nch][64]
  float2 *part_ml;       // [Hkv * B * G][nch]
  // decode over many sequences: CTAs (0: not used), their parts and counters
  int run_ctas, same_dil;
  float *run_acc;        // [2 * run_ctas][min(G, 32)][64]
  float2 *run_ml;        // [2 * run_ctas][min(G, 32)]
  int32_t *run_count;    // [units], zero between calls
  int dil[LF_MAX_H];     // per key/value head
};

#define LF_PART_MAX 64          // parts per row at most
#define LF_PDR_MAX_UNITS 32768  // units with a counter
#define LF_PDR_MAX_B 1024  // sequences whose lengths the decode kernel keeps in shared memory
// Units up to so many tiles are not cut.  Measured, whole / cut, in us: three
// tiles (window 256), 64 x 12 heads (f16) 15.8 / 18.1, 12 x 12 (bf16) 8.2 / 8.1,
// 32 x 16/4 8.6 / 9.7; four tiles 19.8 / 21.9, 9.8 / 9.5, 10.1 / 10.5; five tiles
// (window 512) 23.7 / 25.7, 11.3 / 11.5, 11.6 / 13.5; six tiles 27.5 / 29.7, but
// 12.8 / 10.3 and 13.1 / 11.6.
#define LF_PDR_WHOLE 5

cudaError_t lf_launch_rope(const LfRopeArgs &a, int dtype, bool append, cudaStream_t stream);

struct LfPagedLaunch {
  LfPagedDev dev;
  size_t off_acc, off_ml, off_run_acc, off_run_ml, total;  // workspace
  int dtype;
  cudaStream_t stream;
};

cudaError_t lf_launch_paged_decode(const LfPagedLaunch &L, const void *q, const void *kp,
                                   const void *vp, void *o, float *lse);
cudaError_t lf_launch_prefix(const LfPagedLaunch &L, const void *q, const void *kp, const void *vp);
// how the prefix is read: direct, or parts and keys per chunk of its split
void lf_prefix_plan(LfPagedDev &d, int dtype);
// the same of the tensor-core kernel (bf16, f16, more than 32 rows)
cudaError_t lf_launch_prefix_tc(const LfPagedLaunch &L, const void *q, const void *kp, const void *vp);
void lf_prefix_tc_plan(LfPagedDev &d);
bool lf_prefix_direct(const LfPagedDev &d, int dtype);
// run_ctas and same_dil
void lf_paged_plan(LfPagedDev &d, int dtype);

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

#define LF_P_UP 7
#define LF_P_SCALE ((float)(1 << LF_P_UP))

// Two probabilities as two 16-bit numbers each, for the product with V: p cut
// towards zero and, in `low`, what the cut left (together within the square of
// a step of p), so that the output's only rounding to 16 bits is its last.
// With one number the error of a bf16 output against 64 bits is 0.0023 of its
// norm, with two 0.0017, which is the output's own rounding.  kPacked: packed
// subtraction (43.0 us where single ones take 43.4 in the tensor-core prefix
// kernel; the warp-level kernels of 32 rows would spill a register pair).
// f16: p enters 2^LF_P_UP times as large, so that numbers down to 2^-31 of the
// largest one are held (2^-24 is f16's smallest; p <= 2^8 stays below 65504);
// the output's owner takes the factor out again.
template <int kF16, bool kPacked>
__device__ __forceinline__ void lf_p_split(float p0, float p1, uint32_t &high, uint32_t &low) {
  float h0, h1, r0, r1;
  if (kF16) {
    if (kPacked) {
      lf_unpair(lf_mul2(lf_pair(p0, p1), lf_pair(LF_P_SCALE, LF_P_SCALE)), p0, p1);
    } else {
      p0 *= LF_P_SCALE;
      p1 *= LF_P_SCALE;
    }
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(high) : "f"(p1), "f"(p0));
    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&high));
    h0 = h.x;
    h1 = h.y;
  } else {
    high = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
    h0 = __uint_as_float(__float_as_uint(p0) & 0xffff0000u);
    h1 = __uint_as_float(__float_as_uint(p1) & 0xffff0000u);
  }
  if (kPacked) {
    lf_unpair(lf_fma2(lf_pair(h0, h1), lf_pair(-1.f, -1.f), lf_pair(p0, p1)), r0, r1);
  } else {
    r0 = p0 - h0;
    r1 = p1 - h1;
  }
  // Unless p is 0 in the type, `low` is at least the type's smallest positive
  // number (2^-31 of the largest p, or less): 0 times an infinite value would be
  // NaN.  (bf16: the smallest normal one, as a product may flush others to 0.)
  if (kF16)
    asm("{\n\t.reg .b32 r, t;\n\tcvt.rn.f16x2.f32 r, %1, %2;\n\tmin.f16x2 t, %4, %3;\n\tmax.f16x2 %0, r, t;\n\t}"
        : "=r"(low) : "f"(r1), "f"(r0), "r"(0x00010001u), "r"(high));
  else
    asm("{\n\t.reg .b32 r, t;\n\tcvt.rn.bf16x2.f32 r, %1, %2;\n\tmin.bf16x2 t, %4, %3;\n\tmax.bf16x2 %0, r, t;\n\t}"
        : "=r"(low) : "f"(r1), "f"(r0), "r"(0x00800080u), "r"(high));
}
