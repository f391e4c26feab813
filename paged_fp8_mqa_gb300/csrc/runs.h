// runs.h -- a line of `total` items cut into `runs` consecutive runs: run c has items
// [total * c / runs, total * (c + 1) / runs).  Host and device; 0 < runs <= total.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define IDX_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define IDX_HOST_DEVICE inline
#endif

namespace idx {

// The first item of run c (c = runs: the line's end); runs at most 2048.  32-bit divisions are a
// tenth of the 64-bit ones.
IDX_HOST_DEVICE int64_t run_begin(int64_t total, int64_t runs, int64_t c) {
  if (total < (1 << 21))
    return static_cast<uint32_t>(total) * static_cast<uint32_t>(c) / static_cast<uint32_t>(runs);
  return total * c / runs;
}

// The run that item x is in: the last whose first item is at most x.
IDX_HOST_DEVICE int32_t run_of(int64_t total, int64_t runs, int64_t x) {
  const int64_t y = (x + 1) * runs - 1;
  if (y <= INT32_MAX && total <= INT32_MAX)
    return static_cast<int32_t>(y) / static_cast<int32_t>(total);
  return static_cast<int32_t>(y / total);
}

}  // namespace idx
