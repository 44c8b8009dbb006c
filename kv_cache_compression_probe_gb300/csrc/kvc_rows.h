// Row ranges that come from device memory.  Plain C++ as well, so that the arithmetic is tested on the host.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define KVC_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define KVC_HOST_DEVICE inline
#endif

namespace kvc {

// Whether rows off .. off + len - 1 lie in 0 .. rows - 1 (rows >= 0).  off may be anything: off + len is not
// formed, which passes 63 bits for offsets near 2^63 and would then look small.
KVC_HOST_DEVICE bool rows_fit(int64_t off, int64_t len, int64_t rows) {
  return off >= 0 && len >= 0 && len <= rows && off <= rows - len;
}

}  // namespace kvc
