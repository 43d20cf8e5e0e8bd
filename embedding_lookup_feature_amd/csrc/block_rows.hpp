// block_rows.hpp -- which rows and gate rows the block norm's backward deals out to its slots: plain
// integer functions, the same on the host and in the kernels.
#pragma once

#include <hip/hip_runtime.h>

namespace el {

// Rows [first, first + n).
struct RowRange {
  int first, n;
};

// The rows of slot s where M rows are dealt out to `slots` slots in order.
__host__ __device__ inline RowRange rows_of_slot(int s, int slots, int M) {
  const int base = M / slots, rem = M - base * slots;
  return RowRange{s * base + (s < rem ? s : rem), base + (s < rem)};
}
__host__ __device__ inline int slot_of_row(int r, int slots, int M) {
  const int base = M / slots, rem = M - base * slots, wide = rem * (base + 1);
  return r < wide ? r / (base + 1) : rem + (r - wide) / base;
}

// The gate rows that rows [first, first + n) of M lie in (those of them that exist; first < M, n > 0),
// gate_rows rows to each.
__host__ __device__ inline RowRange gates_of_rows(int first, long n, int gate_rows, int M) {
  const long end = first + n;
  const int last = static_cast<int>((end < M ? end : M) - 1), g0 = first / gate_rows;
  return RowRange{g0, last / gate_rows - g0 + 1};
}

}  // namespace el
