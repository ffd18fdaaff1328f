// lf_status.cuh -- details of LF_ERR_DEVICE_INPUT in the status word outside
// the mask pass, whose own are 1000000 and more without end: negative, plus
// the sequence (below 999999) or, for the projections, less the sequence.
#pragma once

#define LF_DET_ROWS (-5000000)    // more selected rows than max_rows (less the sequence)
#define LF_DET_LENGTH (-4000000)  // length outside [0, capacity]
#define LF_DET_PAGE (-3000000)    // block table entry outside [0, num_pages)
#define LF_DET_PREFIX (-2000000)  // prefix table entry outside [0, num_pages)
#define LF_DET_TOKENS (-1000000)  // new tokens without a row, or cu_new not ascending
