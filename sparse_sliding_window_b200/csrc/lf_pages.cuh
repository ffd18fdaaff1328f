// lf_pages.cuh -- index arithmetic of the paged key/value cache: which row
// of the pool a cache row is, which rows a decode step attends, where a new
// token goes.  Every kernel takes its addresses from here.  Plain integer
// code, so it also compiles as host C++.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define LF_PAGES_FN __host__ __device__ __forceinline__
#else
#define LF_PAGES_FN static inline
#endif

#define LF_ROW_NONE (-1)  // no such row
#define LF_ROW_BAD (-2)   // the table holds no valid page for it

// A sequence length the table can hold?
LF_PAGES_FN bool lf_len_ok(int len, int columns, int shift) {
  return len >= 0 && len <= (columns << shift);
}

// Is cache row `row` inside its table?
LF_PAGES_FN bool lf_row_ok(int columns, int shift, int row) { return row >= 0 && (row >> shift) < columns; }

// Pool row of cache row `row`, which lies in `page`, for key/value head h: the
// pools are [num_pages, Hkv, page_size] rows of 64.  num_pages * Hkv *
// page_size < 2^31 holds on entry, so nothing overflows.
LF_PAGES_FN int lf_row_in_page(int page, int num_pages, int shift, int Hkv, int h, int row) {
  if (page < 0 || page >= num_pages) return LF_ROW_BAD;
  return ((page * Hkv + h) << shift) + (row & ((1 << shift) - 1));
}

// The two together, through the table (columns * page_size <= 2^30).
LF_PAGES_FN int lf_pool_row(const int32_t *table, int columns, int num_pages, int shift, int Hkv,
                            int h, int row) {
  if (!lf_row_ok(columns, shift, row)) return LF_ROW_NONE;
  return lf_row_in_page(table[row >> shift], num_pages, shift, Hkv, h, row);
}

// Keys that the newest token of a sequence of length len attends among its
// own rows: key k is row (len - 1) - k*d, k < the result.
LF_PAGES_FN int lf_window_keys(int len, int window, int d) {
  if (len <= 0) return 0;
  if (window < 0) return len;
  const int last = d == 1 ? len - 1 : (len - 1) / d;
  return (window < last ? window : last) + 1;
}

// The sequence that packed token t belongs to: the largest b with
// cu[b] <= t.  Ends for any contents of cu[0..B]; the caller checks
// cu[b] <= t < cu[b+1].
LF_PAGES_FN int lf_token_seq(const int32_t *cu, int B, int t) {
  int lo = 0, hi = B;  // cu[lo] <= t is assumed of lo, cu[hi] > t of hi
  while (hi - lo > 1) {
    const int mid = lo + ((hi - lo) >> 1);
    if (cu[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Cache row of the i-th of cnt new tokens of a sequence whose length is len
// with them: LF_ROW_NONE for an idle sequence (len = 0, one token per
// sequence), LF_ROW_BAD where there is no such row.
LF_PAGES_FN int lf_new_row(int len, int cnt, int i, int columns, int shift, bool ragged) {
  if (len == 0 && !ragged) return LF_ROW_NONE;
  if (!lf_len_ok(len, columns, shift) || len - cnt + i < 0) return LF_ROW_BAD;
  return len - cnt + i;
}
