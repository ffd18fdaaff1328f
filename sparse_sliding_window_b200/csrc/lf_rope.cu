// lf_rope.cu -- rotation of queries and keys by their positions, and the
// append of new tokens to the paged cache with that rotation on the way.
//
// Both move every element once and compute a few operations for it, so they
// are bound by memory: 269 MB in 48.0 us per call (5.6 TB/s, 0.85 of a plain
// copy's rate; 46.5 us in graph replays) for bf16 queries and keys of 2 x 16
// heads x 16384 tokens.  A thread keeps one 16-byte slice (two for pairs
// (p, p + rot/2), so that both halves of its pairs are in its registers) of
// one token and works through heads: the cosines and sines, the same for
// every head of a token, are computed once per thread.
#include "lf_paged.cuh"

#define LF_ROPE_THREADS 256
#define LF_ROPE_BATCH 2  // heads of a group (4: 48.1 us where 2 takes 46.6, 1: 49.7)

#define LF_ROPE_COPY 0    // no rotation: one slice per thread
#define LF_ROPE_INTER 1   // pairs (2p, 2p+1): one slice holds whole pairs
#define LF_ROPE_HALF 2    // pairs (p, p + pairs), pairs a multiple of the slice: two slices
#define LF_ROPE_ANY 3     // pairs (p, p + pairs), any count: partners through shared memory

template <typename T> struct LfSlice { static constexpr int N = 16 / (int)sizeof(T); };

// cos and sin of the angle of pair p at position pos: turns = pos * (hi + lo)
// less the nearest integer (the product's rounding is undone by the fma), so
// the error does not grow with the position.
__device__ __forceinline__ void lf_rope_angle(const LfRopeDev &r, int p, int pos, float &c, float &s) {
  const double x = (double)pos;
  const double n = rint(x * r.hi[p]);
  const double f = fma(x, r.hi[p], -n) + x * r.lo[p];
  sincospif((float)(2.0 * f), &s, &c);
}

template <typename T>
__device__ __forceinline__ void lf_unpack(const uint4 &v, float (&x)[LfSlice<T>::N]) {
  LfVec<T>::ld(reinterpret_cast<const T *>(&v), x);
}
template <typename T>
__device__ __forceinline__ uint4 lf_repack(const float (&x)[LfSlice<T>::N]) {
  uint4 v;
  LfVec<T>::st(reinterpret_cast<T *>(&v), x);
  return v;
}

template <typename T, int KIND, bool APPEND>
__global__ void __launch_bounds__(LF_ROPE_THREADS) lf_rope_kernel(const __grid_constant__ LfRopeArgs A) {
  constexpr int N = LfSlice<T>::N;                      // channels of a slice
  constexpr int NV = KIND == LF_ROPE_HALF ? 2 : 1;      // slices per thread
  constexpr int TPR = LF_HD / (N * NV);                 // threads per token
  constexpr int NA = KIND == LF_ROPE_COPY ? 1 : KIND == LF_ROPE_INTER ? N / 2 : N;  // angles
  __shared__ float s_row[KIND == LF_ROPE_ANY ? LF_ROPE_THREADS * N : 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tok = blockIdx.x * (LF_ROPE_THREADS / TPR) + threadIdx.x / TPR;  // < 2^31 + 64
  const int q = threadIdx.x % TPR;
  bool active = tok < (uint32_t)A.tokens;
  int64_t b = 0, t = tok;
  int row = 0, pool_row = 0;
  if (!APPEND) {
    const uint32_t seq = tok / (uint32_t)A.n;
    b = seq;
    t = tok - seq * (uint32_t)A.n;
  }

  // channels of the thread's slices
  const int pairs = KIND == LF_ROPE_COPY ? 0 : A.r.pairs;
  int ch[NV];
  bool turn = false;  // HALF: the thread's slices are both halves of N pairs
  if (KIND == LF_ROPE_HALF) {
    const int nq = pairs / N;
    turn = q < nq;
    ch[0] = turn ? q * N : 2 * pairs + (q - nq) * 2 * N;
    ch[NV - 1] = turn ? ch[0] + pairs : ch[0] + N;
  } else {
    ch[0] = q * N;
  }

  // Groups of heads: the next group's loads are started before a group is
  // turned and stored, the first one's before the token's row and angles are
  // known (its inputs do not depend on them).
  int h = blockIdx.y * A.heads_per_block, jb = 0, h0 = 0;  // the job that holds head h, and its first head
  const int hend = min(A.heads_total, h + A.heads_per_block);
  uint4 v[LF_ROPE_BATCH][NV];
  auto group = [&](uint4 (&to)[LF_ROPE_BATCH][NV]) {  // loads the group that starts at h; returns its heads
    while (h >= h0 + A.job[jb].heads) {
      h0 += A.job[jb].heads;
      jb++;
    }
    const LfRopeJob &J = A.job[jb];
    const int cnt = min(min(LF_ROPE_BATCH, hend - h), h0 + J.heads - h);
    const T *x = (const T *)J.x + b * J.xs[0] + (int64_t)(h - h0) * J.xs[1] + t * J.xs[2];
#pragma unroll
    for (int u = 0; u < LF_ROPE_BATCH; u++)
#pragma unroll
      for (int w = 0; w < NV; w++)
        if (tok < (uint32_t)A.tokens && u < cnt) to[u][w] = *reinterpret_cast<const uint4 *>(x + u * J.xs[1] + ch[w]);
    return cnt;
  };
  int cnt = group(v);

  if (APPEND && active) {
    // the token's sequence, its cache row and the pool row of head 0
    int seq = (int)tok, cnt = 1, i = 0;
    bool ok = true;
    if (A.cu) {
      seq = lf_token_seq(A.cu, A.B, (int)tok);
      const int c0 = A.cu[seq], c1 = A.cu[seq + 1];
      ok = c0 >= 0 && c0 <= (int)tok && (int)tok < c1;
      cnt = c1 - c0;
      i = (int)tok - c0;
      // tokens behind the last sequence are nobody's
      if (!ok) {
        active = false;
        if ((int)tok < A.cu[A.B] && q == 0) lf_set_status(A.status, LF_ERR_DEVICE_INPUT, LF_DET_TOKENS + seq);
      }
    }
    if (active) {
      const int len = A.lengths[seq];
      row = lf_new_row(len, cnt, i, A.max_pages, A.shift, A.cu != nullptr);
      if (row >= 0)
        pool_row = lf_pool_row(A.table + (size_t)seq * A.max_pages, A.max_pages, A.num_pages,
                               A.shift, A.Hkv, 0, row);
      if (row < 0 || pool_row < 0) {
        active = false;
        if (q == 0) {
          if (row == LF_ROW_BAD)
            lf_set_status(A.status, LF_ERR_DEVICE_INPUT,
                          (lf_len_ok(len, A.max_pages, A.shift) ? LF_DET_TOKENS : LF_DET_LENGTH) + seq);
          else if (row >= 0)
            lf_set_status(A.status, LF_ERR_DEVICE_INPUT, LF_DET_PAGE + seq);
        }
      }
    }
  }
  float co[NA], si[NA];
  uint32_t on = 0;  // INTER / ANY: which of the thread's pairs / channels turn
  if (KIND != LF_ROPE_COPY && active) {
    int pos[LF_ROPE_MAX_AXES];
#pragma unroll
    for (int a = 0; a < LF_ROPE_MAX_AXES; a++)
      pos[a] = a >= A.r.n_axes ? 0
               : A.positions   ? A.positions[a * A.tokens + tok]
               : APPEND        ? A.pos_offset + row
                               : (int)t;
#pragma unroll
    for (int j = 0; j < NA; j++) {
      int p;
      float sg = A.r.sign;
      if (KIND == LF_ROPE_HALF) {
        p = turn ? q * N + j : -1;
      } else if (KIND == LF_ROPE_INTER) {
        p = q * (N / 2) + j;
      } else {
        p = q * N + j;
        if (p < pairs) sg = -sg;  // x'_u = x_u cos - x_v sin
        else p -= pairs;
      }
      co[j] = 1.f;
      si[j] = 0.f;
      if (p >= 0 && p < pairs) {
        const int ax = A.r.axis[p];
        int x = pos[0];
#pragma unroll
        for (int a = 1; a < LF_ROPE_MAX_AXES; a++) x = ax == a ? pos[a] : x;
        lf_rope_angle(A.r, p, x, co[j], si[j]);
        si[j] *= sg;
        on |= 1u << j;
      }
    }
  }

  for (;;) {
    const LfRopeJob &J = A.job[jb];
    T *out;
    int64_t ohead;
    if (APPEND && J.pool) {
      ohead = (int64_t)LF_HD << A.shift;
      out = (T *)J.pool + (int64_t)pool_row * LF_HD + (h - h0) * ohead;
    } else {
      ohead = J.os[1];
      out = (T *)J.out + b * J.os[0] + (h - h0) * ohead + t * J.os[2];
    }
    const bool rot = KIND != LF_ROPE_COPY && J.rotate;
    const int now = cnt;
    uint4 ahead[LF_ROPE_BATCH][NV];
    h += now;
    const bool more = h < hend;
    if (more) cnt = group(ahead);
#pragma unroll
    for (int u = 0; u < LF_ROPE_BATCH; u++) {
      if (u >= now) continue;
      if (rot && KIND == LF_ROPE_HALF && active && turn) {
        float a[N], c[N], y[N], z[N];
        lf_unpack<T>(v[u][0], a);
        lf_unpack<T>(v[u][NV - 1], c);
#pragma unroll
        for (int j = 0; j < N; j++) {
          const int k = j < NA ? j : 0;
          y[j] = a[j] * co[k] - c[j] * si[k];
          z[j] = c[j] * co[k] + a[j] * si[k];
        }
        v[u][0] = lf_repack<T>(y);
        v[u][NV - 1] = lf_repack<T>(z);
      }
      if (rot && KIND == LF_ROPE_INTER && active) {
        float a[N];
        lf_unpack<T>(v[u][0], a);
#pragma unroll
        for (int j = 0; j < N / 2; j++) {
          const int k = j < NA ? j : 0;
          const float y = a[2 * j] * co[k] - a[2 * j + 1] * si[k];
          const float z = a[2 * j + 1] * co[k] + a[2 * j] * si[k];
          if (on >> j & 1) {
            a[2 * j] = y;
            a[2 * j + 1] = z;
          }
        }
        v[u][0] = lf_repack<T>(a);
      }
      if (rot && KIND == LF_ROPE_ANY) {
        // the token's row in shared memory; its threads are lanes of one warp
        float a[N];
        float *r = s_row + (threadIdx.x / TPR) * LF_HD;
        if (active) {
          lf_unpack<T>(v[u][0], a);
#pragma unroll
          for (int j = 0; j < N; j++) r[q * N + j] = a[j];
        }
        __syncwarp();
        if (active) {
#pragma unroll
          for (int j = 0; j < N; j++) {
            const int c = q * N + j, k = j < NA ? j : 0;
            if (on >> j & 1) a[j] = a[j] * co[k] + r[c < pairs ? c + pairs : c - pairs] * si[k];
          }
          v[u][0] = lf_repack<T>(a);
        }
        __syncwarp();
      }
      if (active)
#pragma unroll
        for (int w = 0; w < NV; w++) *reinterpret_cast<uint4 *>(out + u * ohead + ch[w]) = v[u][w];
    }
    if (!more) break;
#pragma unroll
    for (int u = 0; u < LF_ROPE_BATCH; u++)
#pragma unroll
      for (int w = 0; w < NV; w++) v[u][w] = ahead[u][w];
  }

  // cu_new ascends from 0 to at most the tokens there are: all of it is looked
  // at, as the search above reads only a few entries (and finds a sequence in
  // offsets that are none, too).
  if (APPEND && A.cu && blockIdx.y == 0)
    for (int b = blockIdx.x * LF_ROPE_THREADS + threadIdx.x; b < A.B; b += gridDim.x * LF_ROPE_THREADS) {
      const int c0 = A.cu[b], c1 = A.cu[b + 1];
      if (c1 < c0 || (b == 0 && c0 != 0) || (b == A.B - 1 && c1 > A.tokens))
        lf_set_status(A.status, LF_ERR_DEVICE_INPUT, LF_DET_TOKENS + b);
    }
}

template <typename T, int KIND, bool APPEND>
static cudaError_t lf_launch_rope_k(LfRopeArgs a, cudaStream_t stream) {
  constexpr int N = LfSlice<T>::N;
  constexpr int per = LF_ROPE_THREADS * N * (KIND == LF_ROPE_HALF ? 2 : 1) / LF_HD;  // tokens a block
  const int64_t blocks = (a.tokens + per - 1) / per;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  // Heads a thread works through: more share the angles, fewer fill the GPU.
  // As many as leave about eight blocks per SM (measured, bf16 q and k of 2 x 16
  // heads x 16384 and f32 of 3 x 12 x 1369: 4 blocks 47.5 and 11.4 us, 8 blocks
  // 46.5 and 10.9, 16 blocks 48.2 and 12.1), in whole groups, and at least one.
  const int64_t want = (8 * (int64_t)lf_sm_count() + blocks - 1) / blocks;
  const int split = (int)(want < a.heads_total ? want : a.heads_total);
  a.heads_per_block = (a.heads_total + split - 1) / split;
  if (a.heads_per_block > 1) a.heads_per_block = (a.heads_per_block + LF_ROPE_BATCH - 1) / LF_ROPE_BATCH * LF_ROPE_BATCH;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, (unsigned)((a.heads_total + a.heads_per_block - 1) / a.heads_per_block));
  cfg.blockDim = dim3(LF_ROPE_THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lf_rope_kernel<T, KIND, APPEND>, a);
}

template <typename T, bool APPEND>
static cudaError_t lf_launch_rope_t(const LfRopeArgs &a, cudaStream_t stream) {
  if constexpr (APPEND) {  // a rotation always has pairs
    if (a.r.pairs == 0) return lf_launch_rope_k<T, LF_ROPE_COPY, APPEND>(a, stream);
  }
  if (a.r.interleaved) return lf_launch_rope_k<T, LF_ROPE_INTER, APPEND>(a, stream);
  if (a.r.pairs % LfSlice<T>::N == 0) return lf_launch_rope_k<T, LF_ROPE_HALF, APPEND>(a, stream);
  return lf_launch_rope_k<T, LF_ROPE_ANY, APPEND>(a, stream);
}

template <bool APPEND>
static cudaError_t lf_launch_rope_d(const LfRopeArgs &a, int dtype, cudaStream_t stream) {
  if (dtype == LF_F32) return lf_launch_rope_t<float, APPEND>(a, stream);
  if (dtype == LF_BF16) return lf_launch_rope_t<__nv_bfloat16, APPEND>(a, stream);
  return lf_launch_rope_t<__half, APPEND>(a, stream);
}

cudaError_t lf_launch_rope(const LfRopeArgs &a, int dtype, bool append, cudaStream_t stream) {
  const cudaError_t e = append ? lf_launch_rope_d<true>(a, dtype, stream) : lf_launch_rope_d<false>(a, dtype, stream);
  if (e == cudaSuccess) lf_launches_add(1);
  return e;
}
