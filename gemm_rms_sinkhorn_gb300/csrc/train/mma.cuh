// The tensor product of bf16 values in registers (16 × 8 × 16) that the
// residual update's backward uses, and the transposition that goes with it.
#pragma once

#include <cstdint>

namespace mhc {

// D += A·B.  The lane (g = lane / 4, t = lane % 4) holds, of A [16][16], rows g
// (a0, a2) and g + 8 (a1, a3) at k = 2t, 2t+1 (a0, a1) and 2t+8, 2t+9 (a2, a3);
// of B [16][8] column g at the same k (b0, b1); of D [16][8] row g (d0, d1) and
// g + 8 (d2, d3) at columns 2t, 2t+1.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same without an addend: D = A·B.
__device__ __forceinline__ void mma_16816_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// An 8 × 8 matrix of 16-bit values, row g at lanes 4g .. 4g+3 in column pairs,
// to its transpose in the same layout.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

}  // namespace mhc
