/*
 * lf_paged.h -- C ABI of the serving side of the causal-window attention, in
 * the same library as lf_attn.h (liblf_attn.so): the rotation of queries and
 * keys by their positions, the append of new tokens to a paged key/value
 * cache with that rotation on the way, and the decode step that reads the
 * paged cache, alone or behind a prefix that every sequence of the batch
 * shares.
 *
 * The attention is the one of lf_attn_decode ("Longformer：处理长文档的
 * Transformer模型", segmentfault, 实现: autoregressive language modelling with
 * dilated sliding windows); a shared prefix plays the part that the global
 * tokens play in the encoder (section 全局注意力: tokens that every other token
 * attends).  The pages have no paged cache and no rotary positions.
 *
 * Conventions are those of lf_attn.h: DEVICE pointers owned by the caller
 * unless marked HOST, every call asynchronous on `stream` (which belongs to
 * the current device), nothing allocated, LF_* return codes with
 * lf_attn_last_error(), device-side problems in the status word at the start
 * of the workspace (lf_attn_status).  Tensors of one call share a dtype
 * (LF_F32, LF_BF16, LF_F16) and are 16-byte aligned; int32 arrays are 4-byte
 * aligned.  Strides count elements; the last dimension (64 channels) is
 * contiguous and every other stride is a multiple of 16 bytes.  An output
 * overlaps no other tensor of its call, except where it is said that it may.
 */
#ifndef LF_PAGED_H
#define LF_PAGED_H

#include <stddef.h>
#include <stdint.h>

#include "lf_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- rotation
 * Channel pair p < rot_dim/2 of a token is turned by the angle
 *   a_p = position[pair_axis[p]] * freqs[p]   (freqs NULL: base^(-2p/rot_dim))
 *   x'_u = x_u cos a_p - x_v sin a_p,   x'_v = x_v cos a_p + x_u sin a_p
 * with (u, v) = (p, p + rot_dim/2), or (2p, 2p+1) when interleaved.  Channels
 * >= rot_dim are copied.  A token has n_axes positions (1: text; time,
 * height, width: images and video).  Angles are reduced in double precision,
 * so positions up to the int32 limits keep full accuracy; the rotation is
 * float32, each result rounded once to the dtype. */
typedef struct lf_rope_params {
  int rot_dim;              /* rotated channels: even, 2..64; 0 => 64 */
  int interleaved;          /* 0: pairs (p, p + rot_dim/2); 1: pairs (2p, 2p+1) */
  int n_axes;               /* positions per token, 1..4 */
  const int32_t *pair_axis; /* HOST [rot_dim/2], each in [0, n_axes); NULL = all 0 */
  const double *freqs;      /* HOST [rot_dim/2], radians per position, of size at most 1e6; NULL: from base */
  double base;              /* > 0, finite, no frequency above 1e6 (64 channels: base >= 6.5e-7); 0 => 10000 */
} lf_rope_params;

/* One tensor of a rotation: x and out are [B, heads, n, 64] with strides
 * {batch, head, token}.  out may be x itself with the same strides;
 * otherwise it must not overlap any x or out of the call. */
typedef struct lf_rope_tensor {
  const void *x;
  void *out;
  int heads; /* 1..128 */
  int64_t x_stride[3];
  int64_t out_stride[3];
} lf_rope_tensor;

/* Rotate ntensors (1..8, HOST array) tensors of B sequences of n tokens, all
 * by the same positions: int32 [n_axes, B, n], or NULL (n_axes = 1 only) for
 * the token index 0..n-1. */
int lf_rope_fwd(const lf_rope_params *r, int B, int n, int dtype, int ntensors,
                const lf_rope_tensor *tensors, const int32_t *positions, void *stream);

/* The backward of lf_rope_fwd: x holds the gradients of the rotated tensors,
 * out receives those of the tensors (the rotation by the negative angles). */
int lf_rope_bwd(const lf_rope_params *r, int B, int n, int dtype, int ntensors,
                const lf_rope_tensor *tensors, const int32_t *positions, void *stream);

/* ------------------------------------------------------------- paged cache
 * k_pages, v_pages  [num_pages, Hkv, page_size, 64] contiguous: the pools
 * block_table       int32 [B, max_pages]: the page of rows
 *                   c*page_size .. (c+1)*page_size - 1 of sequence b
 * lengths           int32 [B]: rows of sequence b in the cache, the new
 *                   tokens included; 0 = the sequence is idle
 * Only the table entries that the lengths reach are read. */
typedef struct lf_paged_params {
  int B;                   /* sequences, 1..999999 */
  int H;                   /* query heads, 1..128 */
  int Hkv;                 /* key/value heads, a divisor of H; query head h reads
                              key/value head h / (H / Hkv) */
  int head_dim;            /* must be 64 */
  int page_size;           /* rows a page: a power of two, 16..1024 */
  int num_pages;           /* pages of the pools; num_pages*Hkv*page_size < 2^31 */
  int max_pages;           /* columns of the block table; max_pages*page_size <= 2^30 */
  int window;              /* r >= 0: keys (L-1) - k*d, k = 0..r; < 0: every row of the sequence */
  const int32_t *dilation; /* HOST [Hkv] of d >= 1 per key/value head, or NULL (all 1); all 1 when window < 0 */
  float scale;             /* score scale, 0..2.3e38; 0 => 1/sqrt(head_dim) */
  int dtype;               /* LF_F32 / LF_BF16 / LF_F16 */
  int prefix_len;          /* rows of the prefix that the batch shares, 0..2^30 (0: none); row 0 of
                              a sequence stands at position prefix_len */
} lf_paged_params;

/* Bytes of device workspace lf_cache_append and lf_paged_decode need (256-byte
 * aligned); 0 on invalid params.  Zero all of it once after allocating; every
 * call leaves its counters at zero for the next, which may have other params.
 * One workspace must not be used by two calls that may run at the same time. */
size_t lf_paged_workspace_size(const lf_paged_params *p);

/* Append T new tokens: K rotated, V as it is, to their rows of the pages, Q
 * rotated to q_out.  Sequence b has the tokens cu_new[b] .. cu_new[b+1] - 1
 * (int32 [B+1], ascending from 0; NULL: one token per sequence, T = B), its
 * last rows: token i of cnt goes to row lengths[b] - cnt + i.
 *   q [T,H,64], k, v [T,Hkv,64]: strides {token, head} of q, k, v in the HOST
 *   array strides[6] (NULL: contiguous).  q and q_out may both be NULL.
 *   rope NULL: nothing is rotated.
 *   positions int32 [n_axes, T]; NULL (n_axes = 1): prefix_len + row
 *   q_out [T,H,64] contiguous; it may be q itself when q is contiguous
 * Left as they were: tokens of idle sequences and those >= cu_new[B] in
 * q_out, and every row of the pages that no token goes to.  A length outside
 * [0, max_pages*page_size], a token whose row would be < 0 and a page outside
 * [0, num_pages) are recorded as LF_ERR_DEVICE_INPUT; their tokens are skipped.
 * So is a cu_new that does not ascend from 0 to at most T: tokens that no
 * sequence holds are skipped then, the others go to rows of one that does.
 * Two tokens that the table sends to one row leave either of them there. */
int lf_cache_append(const lf_paged_params *p, const lf_rope_params *rope, int T, const void *q,
                    const void *k, const void *v, const int64_t *strides, const int32_t *cu_new,
                    const int32_t *lengths, const int32_t *positions, const int32_t *block_table,
                    void *q_out, void *k_pages, void *v_pages, void *workspace, size_t ws_bytes,
                    void *stream);

/* Decode step over the paged cache: the newest token of sequence b (row
 * L-1, L = lengths[b]) attends the rows (L-1) - k*d >= 0, k = 0..window, of
 * its own pages (window < 0: every row), and all prefix_len rows of the
 * shared prefix, whose keys and values are read once for the whole batch.
 *   q [B,H,64] with strides {sequence, head} in the HOST array q_stride[2]
 *   (NULL: contiguous)
 *   prefix_table int32 [ceil(prefix_len / page_size)], pages of the same
 *   pools; NULL when prefix_len = 0
 *   o [B,H,64] contiguous (overwritten); lse float32 [B,H] or NULL
 * A sequence of length 0 attends the prefix alone; a query that attends
 * nothing, or scores of -inf alone, gets o = 0 and lse = -inf, and so does one
 * whose length is outside [0, max_pages*page_size].  Such a length and a page
 * outside [0, num_pages) (its rows are left out) are recorded as
 * LF_ERR_DEVICE_INPUT.  Scores, sums and the softmax are float32, and a 16-bit
 * output is rounded once, whichever kernel runs.  An infinite value of an
 * attended row makes its channel infinite, or NaN where another one's sign
 * differs or the row's probability is 0 in the tensors' type.  Results do not
 * depend on the order in which blocks run. */
int lf_paged_decode(const lf_paged_params *p, const void *q, const int64_t *q_stride,
                    const void *k_pages, const void *v_pages, const int32_t *block_table,
                    const int32_t *lengths, const int32_t *prefix_table, void *o, float *lse,
                    void *workspace, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LF_PAGED_H */
