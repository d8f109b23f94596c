// How the reductions over a token's channels lay its streams on a warp: 8 slots
// of 4 lanes, a slot being one stream of one token.  And the 16 × 8 × 16 tensor
// product of bf16 values in registers that they, and the gradient's mixing, use.
#pragma once

#include <cstdint>

namespace mhc {

template <int n>
struct Slots {
    static constexpr int n2 = n <= 1 ? 1 : n <= 2 ? 2 : n <= 4 ? 4 : 8;  // slots of a token
    static constexpr int tokens = 8 / n2;                                // tokens of a warp
};

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

// The same with rows 8 to 15 of A zero (d[2] and d[3] keep their value).  The
// 16 k are the four channels of each of four lanes: the same order in A and B,
// so any assignment of channels to k gives the sum over them.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a2, uint32_t b0,
                                          uint32_t b1)
{
    mma_16816(d, a0, 0u, a2, 0u, b0, b1);
}

}  // namespace mhc
