// Host declarations shared by the microscaled operators.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_internal.h"
#include "mxfp4.h"

namespace moe {

// Rows of fp32 or bf16 values into an MX matrix; arguments already checked.
void launch_mx_quantize(int dtype, int64_t rows, int64_t cols, const void* x, int64_t stride, void* codes,
                        void* scales, hipStream_t s);

inline bool mx_overlaps(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return a && b && na > 0 && nb > 0 && pa < pb + static_cast<uintptr_t>(nb) && pb < pa + static_cast<uintptr_t>(na);
}

}  // namespace moe
