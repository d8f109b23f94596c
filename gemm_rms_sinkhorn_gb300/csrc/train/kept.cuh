// The 8-bit form in which the training step keeps X [B][n][C] for its backward.
//
//   codes   [B][n][C]              one byte per value, OCP e4m3
//   scales  [B][n][ceil(C / 32)]   one byte E per 32 channels of a stream: the
//                                  block's scale is 2^(E - 127)
//
// A value stands for code · 2^(E - 127).  E is the smallest one in [10, 247]
// with amax <= 448 · 2^(E - 127), 448 being e4m3's largest value, so no value
// saturates.  The lower end keeps every value that can be stood for a normal
// number, in fp32 and in bf16: the smallest step is 2^-9 · 2^-117 = 2^-126;
// with 4 significant bits each is exact in bf16.  At the upper end a magnitude
// over 240·2^120 is kept as that, for the next code would stand for 2^128, which
// is infinite in both.  A block that holds an infinity or a NaN gets E = 255 and NaN
// codes: the whole block reads as NaN.
//
// Off by at most: 2^-4 of a magnitude from 2^-6 times the scale on, below that (e4m3's
// subnormals) 2^-10 times the scale.  With E > 10 amax is over 224 times the scale, so
// the first holds within 2^-13 of amax (2^-6/224 = 2^-13.8), not further.
#pragma once

#include <cstdint>

#include "mix.cuh"
#include "ptx.cuh"

namespace mhc {
namespace kept {

constexpr uint32_t kScaleMin = 10, kScaleMax = 247, kScaleNan = 255;
constexpr uint32_t kCodesNan = 0x7F7F7F7Fu;

// The largest magnitude of 8 bf16 values, as its bit pattern (bf16 magnitudes
// order as their bits do; 0x7F80 and above: an infinity or a NaN among them).
__device__ __forceinline__ uint32_t amax8(const uint4 &v)
{
    constexpr uint32_t m = 0x7FFF7FFFu;
    const uint32_t a = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
    return max(a & 0xFFFFu, a >> 16);
}

// E of a block from its largest magnitude's bits: with amax = 2^e·(1 + f/128),
// amax <= 448·2^k = 1.75·2^(8+k) needs k >= e - 8, and e - 7 when f > 96.
__device__ __forceinline__ uint32_t scale_code(uint32_t amax)
{
    if (amax >= 0x7F80u) return kScaleNan;
    const int e = static_cast<int>((amax + 31u) >> 7) - 8;
    return e < static_cast<int>(kScaleMin) ? kScaleMin : static_cast<uint32_t>(e);
}

// Eight bf16 values to codes (round to nearest even) under the scale E.
__device__ __forceinline__ uint2 encode8(const uint4 &v, uint32_t E)
{
    if (E == kScaleNan) return make_uint2(kCodesNan, kCodesNan);
    const float inv = __uint_as_float((254u - E) << 23);  // 2^(127 - E), exact
    float f[8];
    unpack8(v, f);
    if (E == kScaleMax) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = fminf(fmaxf(f[e], -0x1.ep127f), 0x1.ep127f);
    }
    uint32_t h[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) h[p] = f32x2_to_e4m3(f[2 * p] * inv, f[2 * p + 1] * inv);
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// 2^(E - 127); infinity for E = 255, whose codes are NaN.
__device__ __forceinline__ float scale_value(uint32_t E) { return __uint_as_float(E << 23); }

__device__ __forceinline__ void f16x2_to_f32(uint32_t h2, float &lo, float &hi)
{
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi) : "r"(h2));
}

// Eight codes to the fp32 values they stand for (exact).
__device__ __forceinline__ void decode8(const uint2 &q, float scale, float (&f)[8])
{
    const uint32_t w[4] = {q.x, q.x >> 16, q.y, q.y >> 16};
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        float lo, hi;
        f16x2_to_f32(e4m3x2_to_f16x2(w[p]), lo, hi);
        f[2 * p] = lo * scale;
        f[2 * p + 1] = hi * scale;
    }
}

// Eight codes to the fp32 values of the codes alone, as four channel pairs:
// where sums run over one block, its scale is applied to the sum.
__device__ __forceinline__ void codes8_pairs(const uint2 &q, uint64_t (&t)[4])
{
    const uint32_t w[4] = {q.x, q.x >> 16, q.y, q.y >> 16};
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        float lo, hi;
        f16x2_to_f32(e4m3x2_to_f16x2(w[p]), lo, hi);
        t[p] = f2_pack(lo, hi);
    }
}

// The same as bf16 pairs (exact).
__device__ __forceinline__ uint4 codes8_bf16(const uint2 &q)
{
    const uint32_t w[4] = {q.x, q.x >> 16, q.y, q.y >> 16};
    uint32_t r[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        float lo, hi;
        f16x2_to_f32(e4m3x2_to_f16x2(w[p]), lo, hi);
        r[p] = pack_bf16_rn(lo, hi);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// The values that eight codes stand for under the scale E, as bf16 (exact: the
// scale is a power of two, so it may multiply the packed bf16 pairs).
__device__ __forceinline__ uint4 decode8_bf16(const uint2 &q, uint32_t E)
{
    const uint4 c = codes8_bf16(q);
    const uint32_t s = (E << 7) | (E << 23);  // 2^(E - 127) as a bf16 pair
    uint32_t r[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int p = 0; p < 4; ++p) asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(r[p]) : "r"(s));
    return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ uint2 ld_stream_v2(const void *p)
{
    uint2 v;
    asm volatile("ld.global.cs.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void st_stream_v2(void *p, uint2 v)
{
    asm volatile("st.global.cs.v2.u32 [%0], {%1,%2};" ::"l"(p), "r"(v.x), "r"(v.y) : "memory");
}

// Eight consecutive values as fp32 from bf16 or fp32 storage.
__device__ __forceinline__ void load_f8(const uint16_t *p, float (&f)[8])
{
    unpack8(ptx::ld_stream_v4(p), f);
}
__device__ __forceinline__ void load_f8(const float *p, float (&f)[8])
{
    const uint4 a = ptx::ld_stream_v4(p), b = ptx::ld_stream_v4(p + 4);
    f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y);
    f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
    f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y);
    f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
}

}  // namespace kept
}  // namespace mhc
