// slm_norm_rows.h - which rows the block norm's ring backward takes, and which 16-byte pieces of a
// row it copies whole.  Plain C++, so that a host program can walk every case.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SLM_HOST_DEVICE __host__ __device__
#else
#define SLM_HOST_DEVICE
#endif

namespace slm {

// Rows of `d` channels, pieces of `elems` of them.  A row's pieces start `shift` < elems elements
// before it and end less than a piece behind it.  From d = elems on, those ends lie in the
// neighbouring rows, and only the array's first and last row have pieces that reach outside it;
// narrower rows' pieces may cover several neighbours and reach outside from other rows too.
SLM_HOST_DEVICE inline bool norm_ring_takes(int64_t d, int elems) { return d >= elems; }

// Of the pieces [piece0, piece0 + mine) of row `row` of N, those [lo, hi) that lie inside the array
// (rows at least d apart): the others' elements are loaded one by one.
struct NormWindow {
  int lo, hi;
};
SLM_HOST_DEVICE inline NormWindow norm_window(int64_t row, int64_t N, int64_t d, int shift,
                                              int elems, int piece0, int mine) {
  NormWindow w{piece0, piece0 + mine};
  if (row == 0 && shift > 0 && w.lo < 1) w.lo = 1;
  if (row == N - 1) {
    const int whole = static_cast<int>((d + shift) / elems);
    if (w.hi > whole) w.hi = whole;
  }
  if (w.hi < w.lo) w.hi = w.lo;
  return w;
}

}  // namespace slm
