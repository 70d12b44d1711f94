// Equal runs of consecutive units, one a CTA. Plain C++, so that it can be checked without a GPU.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define PMOE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define PMOE_HOST_DEVICE inline
#endif

namespace pmoe {
namespace chunk {

// The first unit of CTA c's run. (A 64-bit division takes some 500 cycles, one of 32 bits a tenth.)
PMOE_HOST_DEVICE int64_t run_start(int64_t units, int ctas, int c) {
  const int64_t x = units * c;
  return x >> 32 ? x / ctas : (int64_t)((uint32_t)x / (uint32_t)ctas);
}

// The CTA that takes unit u: the largest c with run_start(c) <= u.
PMOE_HOST_DEVICE int cta_of(int64_t units, int ctas, int64_t u) {
  const int64_t x = (u + 1) * ctas - 1;
  return (x | units) >> 32 ? (int)(x / units) : (int)((uint32_t)x / (uint32_t)units);
}

}  // namespace chunk
}  // namespace pmoe
