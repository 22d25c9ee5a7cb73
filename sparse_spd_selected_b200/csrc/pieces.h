// Rows of a line cut into pieces of equal length: segments of the scan, chunks of the convolution.
#pragma once

#ifdef __CUDACC__
#define SELINV_PIECES_FN __host__ __device__ inline
#else
#define SELINV_PIECES_FN inline
#endif

namespace selinv {

// The row behind the last of the piece of `step` rows that begins at row r0 <= rows.  r0 + step itself may pass 2^31: a
// line may have all but 65 rows of that, and a piece is longer.
SELINV_PIECES_FN int piece_end(int r0, int step, int rows) { return rows - r0 < step ? rows : r0 + step; }

}  // namespace selinv
