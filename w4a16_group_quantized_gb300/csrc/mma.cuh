// Register-operand tensor-core products and the 16-bit pieces around them, shared by the kernels whose rows choose
// their weights.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace w4 {
namespace detail {

// D += A (16 x 16, row-major fragments) . B (16 x 8): fp16 or bf16 operands, fp32 sums. Lane 4 g + t holds of A the
// pairs (row g, k-pair 0), (row g + 8, k-pair 0), (g, 1), (g + 8, 1), of B column g's pairs 0 and 1, and of D rows
// g and g + 8, columns 2 t and 2 t + 1. Which k a lane's pairs stand for is free as long as A and B agree: the
// kernels give lane t consecutive k, so that its loads are wide.
template <int DT>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  if (DT == kDtypeBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int DT>
__device__ __forceinline__ float value_f32(uint32_t bits) {
  if (DT == kDtypeBf16) return __uint_as_float(bits << 16);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}

}  // namespace detail
}  // namespace w4
