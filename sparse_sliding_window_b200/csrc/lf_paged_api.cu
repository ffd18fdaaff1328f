// lf_paged_api.cu -- the C ABI of include/lf_paged.h: argument checks, the
// workspace, and the launches of each call on the caller's stream.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include "lf_paged.cuh"

// defined in lf_api.cu: record an error for lf_attn_last_error()
int lf_record_error(int code, const char *msg);

static int lp_fail(int code, const char *fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return lf_record_error(code, msg);
}

static int lp_cuda(cudaError_t e, const char *what) {
  if (e == cudaSuccess) return LF_OK;
  return lp_fail(LF_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

static int lp_ptr(const void *ptr, const char *name, int align) {
  if (!ptr) return lp_fail(LF_ERR_INVALID, "%s is NULL", name);
  if ((uintptr_t)ptr % align) return lp_fail(LF_ERR_INVALID, "%s is not %d-byte aligned", name, align);
  return LF_OK;
}

static int lp_dtype_bytes(int dtype) { return dtype == LF_F32 ? 4 : 2; }

// A stride in elements; that of a dimension of one is nobody's and set to 0.
static int lp_stride(int64_t &s, int64_t dim, int dtype, const char *name) {
  if (dim <= 1) {
    s = 0;
    return LF_OK;
  }
  if (s < 0 || s > (1ll << 40) || s * lp_dtype_bytes(dtype) % 16)
    return lp_fail(LF_ERR_INVALID, "stride %lld of %s: 0..2^40 and a multiple of 16 bytes is wanted", (long long)s, name);
  return LF_OK;
}

// ------------------------------------------------------------------ rotation

static const double LP_TWO_PI_HI = 6.283185307179586, LP_TWO_PI_LO = 2.4492935982947064e-16;

// Radians per position: its product with an int32 position (below 2^31) is
// within 2^48 turns, which double precision reduces to a turn without loss.
static const double LP_MAX_FREQ = 1e6;

static int lp_rope(const lf_rope_params *r, bool backward, LfRopeDev &d) {
  memset(&d, 0, sizeof(d));
  if (!r) return LF_OK;  // pairs = 0: nothing turns
  const int rot = r->rot_dim == 0 ? LF_HD : r->rot_dim;
  if (rot < 2 || rot > LF_HD || rot % 2)
    return lp_fail(LF_ERR_INVALID, "rot_dim must be even, 2..64 (got %d)", r->rot_dim);
  if (r->interleaved != 0 && r->interleaved != 1) return lp_fail(LF_ERR_INVALID, "interleaved must be 0 or 1");
  if (r->n_axes < 1 || r->n_axes > LF_ROPE_MAX_AXES)
    return lp_fail(LF_ERR_INVALID, "n_axes must be 1..%d (got %d)", LF_ROPE_MAX_AXES, r->n_axes);
  const double base = r->base == 0 ? 10000.0 : r->base;
  if (!(base > 0) || isinf(base)) return lp_fail(LF_ERR_INVALID, "base must be finite and > 0");
  d.pairs = rot / 2;
  d.interleaved = r->interleaved;
  d.n_axes = r->n_axes;
  d.sign = backward ? -1.f : 1.f;
  for (int p = 0; p < d.pairs; p++) {
    const int ax = r->pair_axis ? r->pair_axis[p] : 0;
    if (ax < 0 || ax >= r->n_axes) return lp_fail(LF_ERR_INVALID, "pair_axis[%d] = %d is no axis", p, ax);
    d.axis[p] = (uint8_t)ax;
    const double f = r->freqs ? r->freqs[p] : pow(base, -2.0 * p / rot);
    if (!(fabs(f) <= LP_MAX_FREQ)) {
      if (r->freqs) return lp_fail(LF_ERR_INVALID, "freqs[%d] must be finite, of size at most 1e6", p);
      return lp_fail(LF_ERR_INVALID, "base %g is too small: pair %d turns by more than 1e6 radians a position", base, p);
    }
    // f / 2 pi in twice double precision
    d.hi[p] = f / LP_TWO_PI_HI;
    d.lo[p] = (fma(-d.hi[p], LP_TWO_PI_HI, f) - d.hi[p] * LP_TWO_PI_LO) / LP_TWO_PI_HI;
  }
  return LF_OK;
}

// Do two elements of [B, heads, n, 64] with these strides share memory?
static bool lp_overlaps_itself(const int64_t *s, int B, int heads, int n) {
  int64_t dim[3] = {B, heads, n}, st[3] = {s[0], s[1], s[2]};
  int64_t need = LF_HD;  // elements below the next dimension's stride
  for (int k = 0; k < 3; k++) {
    int at = -1;  // the smallest stride left of a dimension of more than one
    for (int i = 0; i < 3; i++)
      if (dim[i] > 1 && (at < 0 || st[i] < st[at])) at = i;
    if (at < 0) return false;
    if (st[at] < need) return true;
    need = st[at] * (dim[at] - 1) + need;
    dim[at] = 1;
  }
  return false;
}

static int lp_rope_run(const lf_rope_params *r, bool backward, int B, int n, int dtype, int ntensors,
                       const lf_rope_tensor *tensors, const int32_t *positions, void *stream) {
  int st;
  lf_record_error(LF_OK, "");
  if (!r) return lp_fail(LF_ERR_INVALID, "rope params is NULL");
  LfRopeArgs a;
  memset(&a, 0, sizeof(a));
  if ((st = lp_rope(r, backward, a.r))) return st;
  if (B < 1 || n < 1) return lp_fail(LF_ERR_INVALID, "B, n must be >= 1 (got %d, %d)", B, n);
  if (dtype < LF_F32 || dtype > LF_F16) return lp_fail(LF_ERR_INVALID, "bad dtype %d", dtype);
  if (ntensors < 1 || ntensors > LF_ROPE_MAX_JOBS || !tensors)
    return lp_fail(LF_ERR_INVALID, "1..%d tensors wanted (got %d)", LF_ROPE_MAX_JOBS, ntensors);
  if (positions) {
    if ((st = lp_ptr(positions, "positions", 4))) return st;
  } else if (a.r.n_axes != 1) {
    return lp_fail(LF_ERR_INVALID, "positions may be NULL for one axis only");
  }
  if ((long long)B * n > (1ll << 31) - 64) return lp_fail(LF_ERR_UNSUPPORTED, "B*n too large");
  for (int i = 0; i < ntensors; i++) {
    const lf_rope_tensor &t = tensors[i];
    if (t.heads < 1 || t.heads > LF_MAX_H)
      return lp_fail(LF_ERR_INVALID, "tensor %d: heads must be 1..%d (got %d)", i, LF_MAX_H, t.heads);
    if ((st = lp_ptr(t.x, "x", 16)) || (st = lp_ptr(t.out, "out", 16))) return st;
    LfRopeJob &J = a.job[i];
    memcpy(J.xs, t.x_stride, sizeof(J.xs));
    memcpy(J.os, t.out_stride, sizeof(J.os));
    const int dim[3] = {B, t.heads, n};
    for (int k = 0; k < 3; k++) {
      if ((st = lp_stride(J.xs[k], dim[k], dtype, "x")) || (st = lp_stride(J.os[k], dim[k], dtype, "out"))) return st;
      if (t.x == t.out && J.xs[k] != J.os[k])
        return lp_fail(LF_ERR_INVALID, "tensor %d: in place, but x and out have other strides", i);
    }
    if (lp_overlaps_itself(J.os, B, t.heads, n)) return lp_fail(LF_ERR_INVALID, "tensor %d: out overlaps itself", i);
    J.x = t.x;
    J.out = t.out;
    J.heads = t.heads;
    J.rotate = 1;
    a.heads_total += t.heads;
  }
  a.n = n;
  a.tokens = (int64_t)B * n;
  a.positions = positions;
  return lp_cuda(lf_launch_rope(a, dtype, false, (cudaStream_t)stream), backward ? "lf_rope_bwd" : "lf_rope_fwd");
}

extern "C" int lf_rope_fwd(const lf_rope_params *r, int B, int n, int dtype, int ntensors,
                           const lf_rope_tensor *tensors, const int32_t *positions, void *stream) {
  return lp_rope_run(r, false, B, n, dtype, ntensors, tensors, positions, stream);
}

extern "C" int lf_rope_bwd(const lf_rope_params *r, int B, int n, int dtype, int ntensors,
                           const lf_rope_tensor *tensors, const int32_t *positions, void *stream) {
  return lp_rope_run(r, true, B, n, dtype, ntensors, tensors, positions, stream);
}

// --------------------------------------------------------------- paged cache

#define LP_OFF_COUNT 256  // counters of the decode kernel, behind the status words

static size_t lp_align(size_t x) { return (x + 255) & ~(size_t)255; }

static int lp_prepare(const lf_paged_params *p, LfPagedLaunch &L) {
  lf_record_error(LF_OK, "");
  if (!p) return lp_fail(LF_ERR_INVALID, "params is NULL");
  if (p->B < 1 || p->H < 1 || p->Hkv < 1)
    return lp_fail(LF_ERR_INVALID, "B, H, Hkv must be >= 1 (got %d, %d, %d)", p->B, p->H, p->Hkv);
  if (p->B > 999999) return lp_fail(LF_ERR_UNSUPPORTED, "B = %d > 999999", p->B);
  if (p->H > LF_MAX_H) return lp_fail(LF_ERR_UNSUPPORTED, "H = %d > %d", p->H, LF_MAX_H);
  if (p->H % p->Hkv) return lp_fail(LF_ERR_INVALID, "H = %d is no multiple of Hkv = %d", p->H, p->Hkv);
  if (p->head_dim != LF_HD) return lp_fail(LF_ERR_UNSUPPORTED, "head_dim must be 64 (got %d)", p->head_dim);
  if (p->page_size < 16 || p->page_size > 1024 || (p->page_size & (p->page_size - 1)))
    return lp_fail(LF_ERR_INVALID, "page_size must be a power of two, 16..1024 (got %d)", p->page_size);
  if (p->num_pages < 1 || p->max_pages < 1)
    return lp_fail(LF_ERR_INVALID, "num_pages, max_pages must be >= 1 (got %d, %d)", p->num_pages, p->max_pages);
  if ((long long)p->num_pages * p->Hkv * p->page_size >= 1ll << 31)
    return lp_fail(LF_ERR_UNSUPPORTED, "num_pages * Hkv * page_size must be below 2^31");
  if ((long long)p->max_pages * p->page_size > 1ll << 30)
    return lp_fail(LF_ERR_UNSUPPORTED, "max_pages * page_size must be at most 2^30");
  if (p->dtype < LF_F32 || p->dtype > LF_F16) return lp_fail(LF_ERR_INVALID, "bad dtype %d", p->dtype);
  if (!(p->scale >= 0.f) || isinf(p->scale * LF_LOG2E))
    return lp_fail(LF_ERR_INVALID, "scale must be 0 .. 2.3e38 (got %g)", p->scale);
  if (p->prefix_len < 0 || p->prefix_len > 1 << 30)
    return lp_fail(LF_ERR_INVALID, "prefix_len must be 0..2^30 (got %d)", p->prefix_len);
  if (p->prefix_len > 0 && (long long)p->B * (p->H / p->Hkv) > 2000000)
    return lp_fail(LF_ERR_UNSUPPORTED, "more than 2000000 queries per key/value head behind a prefix");
  LfPagedDev &d = L.dev;
  memset(&d, 0, sizeof(d));
  for (int h = 0; h < p->Hkv; h++) {
    d.dil[h] = p->dilation ? p->dilation[h] : 1;
    if (d.dil[h] < 1) return lp_fail(LF_ERR_INVALID, "dilation[%d] = %d < 1", h, d.dil[h]);
    if (d.dil[h] > 1 && p->window < 0) return lp_fail(LF_ERR_INVALID, "a dilation above 1 needs a window");
  }
  d.B = p->B;
  d.H = p->H;
  d.Hkv = p->Hkv;
  d.G = p->H / p->Hkv;
  while ((1 << d.shift) < p->page_size) d.shift++;
  d.num_pages = p->num_pages;
  d.max_pages = p->max_pages;
  d.window = p->window < 0 ? -1 : p->window;
  d.prefix_len = p->prefix_len;
  d.scale_log2 = (p->scale > 0.f ? p->scale : 1.f / sqrtf((float)LF_HD)) * LF_LOG2E;
  lf_prefix_plan(d, p->dtype);
  const size_t parts = (size_t)p->B * p->H * d.nch;
  // the counters have the same place whatever the params are, so that one
  // zeroed workspace serves calls with different params
  size_t off = LP_OFF_COUNT + LF_PDR_MAX_UNITS * 4;
  L.off_acc = off;
  off = lp_align(off + parts * LF_HD * 4);
  L.off_ml = off;
  off = lp_align(off + parts * 8);
  lf_paged_plan(d, p->dtype);
  const size_t rows = d.run_ctas ? 2 * (size_t)d.run_ctas * (d.G < 32 ? d.G : 32) : 0;
  L.off_run_acc = off;
  off = lp_align(off + rows * LF_HD * 4);
  L.off_run_ml = off;
  off = lp_align(off + rows * 8);
  L.total = off;
  L.dtype = p->dtype;
  return LF_OK;
}

extern "C" size_t lf_paged_workspace_size(const lf_paged_params *p) {
  LfPagedLaunch L;
  return lp_prepare(p, L) == LF_OK ? L.total : 0;
}

static int lp_bind(const lf_paged_params *p, void *workspace, size_t ws_bytes, void *stream, LfPagedLaunch &L) {
  int st;
  if ((st = lp_prepare(p, L)) || (st = lp_ptr(workspace, "workspace", 256))) return st;
  if (ws_bytes < L.total)
    return lp_fail(LF_ERR_INVALID, "workspace too small: %zu < %zu bytes", ws_bytes, L.total);
  char *ws = (char *)workspace;
  L.dev.status = (int32_t *)ws;
  L.dev.part_acc = (float *)(ws + L.off_acc);
  L.dev.part_ml = (float2 *)(ws + L.off_ml);
  L.dev.run_acc = (float *)(ws + L.off_run_acc);
  L.dev.run_ml = (float2 *)(ws + L.off_run_ml);
  L.dev.run_count = (int32_t *)(ws + LP_OFF_COUNT);
  L.stream = (cudaStream_t)stream;
  return LF_OK;
}

extern "C" int lf_cache_append(const lf_paged_params *p, const lf_rope_params *rope, int T, const void *q,
                               const void *k, const void *v, const int64_t *strides,
                               const int32_t *cu_new, const int32_t *lengths,
                               const int32_t *positions, const int32_t *block_table, void *q_out,
                               void *k_pages, void *v_pages, void *workspace, size_t ws_bytes,
                               void *stream) {
  int st;
  LfPagedLaunch L;
  if ((st = lp_bind(p, workspace, ws_bytes, stream, L))) return st;
  LfRopeArgs a;
  memset(&a, 0, sizeof(a));
  if ((st = lp_rope(rope, false, a.r))) return st;
  if (T < 0) return lp_fail(LF_ERR_INVALID, "T must be >= 0 (got %d)", T);
  if (!cu_new && T != p->B)
    return lp_fail(LF_ERR_INVALID, "without cu_new there is one token per sequence: T = %d, B = %d", T, p->B);
  if (!q != !q_out) return lp_fail(LF_ERR_INVALID, "q and q_out go together");
  if ((st = lp_ptr(lengths, "lengths", 4)) || (st = lp_ptr(block_table, "block_table", 4))) return st;
  if (cu_new && (st = lp_ptr(cu_new, "cu_new", 4))) return st;
  if (positions && (st = lp_ptr(positions, "positions", 4))) return st;
  if (rope && !positions && a.r.n_axes != 1)
    return lp_fail(LF_ERR_INVALID, "positions may be NULL for one axis only");
  if (T == 0) return LF_OK;
  const void *x[3] = {q, k, v};
  static const char *const names[3] = {"q", "k", "v"};
  const int heads[3] = {p->H, p->Hkv, p->Hkv};
  int nj = 0;
  for (int i = 0; i < 3; i++) {
    if (i == 0 && !q) continue;
    if ((st = lp_ptr(x[i], names[i], 16))) return st;
    LfRopeJob &J = a.job[nj++];
    J.x = x[i];
    J.heads = heads[i];
    J.rotate = i < 2 && a.r.pairs > 0;
    J.xs[2] = strides ? strides[2 * i] : (int64_t)heads[i] * LF_HD;
    J.xs[1] = strides ? strides[2 * i + 1] : LF_HD;
    if ((st = lp_stride(J.xs[2], T, p->dtype, names[i])) || (st = lp_stride(J.xs[1], heads[i], p->dtype, names[i])))
      return st;
    a.heads_total += heads[i];
    if (i == 0) {
      if ((st = lp_ptr(q_out, "q_out", 16))) return st;
      if (q == q_out && ((T > 1 && J.xs[2] != (int64_t)p->H * LF_HD) || (p->H > 1 && J.xs[1] != LF_HD)))
        return lp_fail(LF_ERR_INVALID, "q_out is q, but q is not contiguous");
      J.out = q_out;
      J.os[1] = LF_HD;
      J.os[2] = (int64_t)p->H * LF_HD;
    } else {
      J.pool = i == 1 ? k_pages : v_pages;
      if ((st = lp_ptr(J.pool, i == 1 ? "k_pages" : "v_pages", 16))) return st;
    }
  }
  a.tokens = T;
  a.n = T;
  a.positions = positions;
  a.B = p->B;
  a.Hkv = p->Hkv;
  a.shift = L.dev.shift;
  a.num_pages = p->num_pages;
  a.max_pages = p->max_pages;
  a.pos_offset = p->prefix_len;
  a.cu = cu_new;
  a.lengths = lengths;
  a.table = block_table;
  a.status = L.dev.status;
  return lp_cuda(lf_launch_rope(a, p->dtype, true, L.stream), "lf_cache_append");
}

extern "C" int lf_paged_decode(const lf_paged_params *p, const void *q, const int64_t *q_stride,
                               const void *k_pages, const void *v_pages, const int32_t *block_table,
                               const int32_t *lengths, const int32_t *prefix_table, void *o,
                               float *lse, void *workspace, size_t ws_bytes, void *stream) {
  int st;
  LfPagedLaunch L;
  if ((st = lp_bind(p, workspace, ws_bytes, stream, L))) return st;
  if ((st = lp_ptr(q, "q", 16)) || (st = lp_ptr(k_pages, "k_pages", 16)) ||
      (st = lp_ptr(v_pages, "v_pages", 16)) || (st = lp_ptr(block_table, "block_table", 4)) ||
      (st = lp_ptr(lengths, "lengths", 4)) || (st = lp_ptr(o, "o", 16)) ||
      (lse && (st = lp_ptr(lse, "lse", 4))))
    return st;
  if (p->prefix_len > 0 && (st = lp_ptr(prefix_table, "prefix_table", 4))) return st;
  L.dev.qs[0] = q_stride ? q_stride[0] : (int64_t)p->H * LF_HD;
  L.dev.qs[1] = q_stride ? q_stride[1] : LF_HD;
  if ((st = lp_stride(L.dev.qs[0], p->B, p->dtype, "q")) || (st = lp_stride(L.dev.qs[1], p->H, p->dtype, "q"))) return st;
  L.dev.table = block_table;
  L.dev.lengths = lengths;
  L.dev.prefix_table = prefix_table;
  if (L.dev.nch > 0 && (st = lp_cuda(lf_launch_prefix(L, q, k_pages, v_pages), "lf_paged_decode (prefix)")))
    return st;
  return lp_cuda(lf_launch_paged_decode(L, q, k_pages, v_pages, o, lse), "lf_paged_decode");
}
