// Backward of the residual update X_next = H_res·X + H_post ⊗ F_out, X read as
// it was kept (kept.cuh).  With G = dX_next:
//
//   dF_out[c]    = Σ_i H_post[i]·G[i][c]
//   dH_res[i][j] = Σ_c G[i][c]·X[j][c]
//   dH_post[i]   = Σ_c G[i][c]·F_out[c]
//
// (dX = H_resᵀ·G + … is left to the backward of what precedes, which has more
// to add to it, so G is not mixed and written twice.)
//
// One pass over G, the codes and F_out, bound by their bytes.  A CTA takes one
// group of tokens over all channels.  The lanes of a warp are 8 slots × 4: a
// slot is one stream of one token (n rounded up to a power of two, so 8, 4, 2
// or 1 tokens a group), and its four lanes hold 8 neighbouring channels each.
//   - G·Xᵀ over the slots is an 8 × 8 product per 32 channels: two
//     mma.m16n8k16 on values that are exact in bf16, accumulated in fp32, with
//     the slots of X as the rows (the other 8 rows zero) and those of G as the
//     columns.  What it wastes (rows, pairs of different tokens) costs nothing
//     here: tcgen05's smallest tile is 128 rows, and per-thread FMAs would take
//     n² registers of accumulators and as many cross-lane sums at the end.
//   - dF_out sums over the slots of a token: a butterfly that halves the
//     channels a lane holds at each step, so 7 shuffles for 8 streams.
//   - the warps of the CTA take the channel groups in turn, and their sums are
//     added in warp order at the end: the result does not depend on timing.
#include <cuda_runtime.h>

#include <cstdint>

#include "check.cuh"
#include "kept.cuh"
#include "mix.cuh"
#include "ptx.cuh"
#include "slots.cuh"
#include "train.h"

namespace mhc {
namespace {

// Keeps half of the 2·W values per step, those this lane's slot bit selects,
// with the other lane's halves added: after log2(n2) steps the sum over the
// n2 slots of 8/n2 channels is left in v[0 ..], the channels from `off` on.
template <int n2>
__device__ __forceinline__ int sum_over_slots(float (&v)[8], int slot)
{
    int off = 0;
#pragma unroll
    for (int s = 1, w = 4; s < n2; s *= 2, w /= 2) {
        const bool up = (slot & s) != 0;
#pragma unroll
        for (int e = 0; e < w; ++e) {
            const float give = up ? v[e] : v[w + e];
            const float keep = up ? v[w + e] : v[e];
            v[e] = keep + __shfl_xor_sync(0xffffffffu, give, s * 4);
        }
        off += up ? w : 0;
    }
    return off;
}

template <int cnt>
__device__ __forceinline__ void store_vals(uint16_t *p, const float (&v)[8])
{
    if constexpr (cnt == 8) {
        ptx::st_stream_v4(p, pack8(v));
    } else if constexpr (cnt == 4) {
        kept::st_stream_v2(p, make_uint2(pack_bf16_rn(v[0], v[1]), pack_bf16_rn(v[2], v[3])));
    } else if constexpr (cnt == 2) {
        *reinterpret_cast<uint32_t *>(p) = pack_bf16_rn(v[0], v[1]);
    } else {
        *p = static_cast<uint16_t>(pack_bf16_rn(v[0], 0.f));
    }
}

template <int cnt>
__device__ __forceinline__ void store_vals(float *p, const float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < cnt; e += (cnt >= 4 ? 4 : cnt)) {
        if constexpr (cnt >= 4)
            *reinterpret_cast<float4 *>(p + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        else if constexpr (cnt == 2)
            *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
        else
            *p = v[0];
    }
}

template <typename FT>
struct FRaw;  // 8 values of F_out as loaded
template <>
struct FRaw<uint16_t> {
    uint4 a;
    __device__ void load(const uint16_t *p) { a = ptx::ld_stream_v4(p); }
    __device__ void zero() { a = make_uint4(0, 0, 0, 0); }
    __device__ void get(float (&f)[8]) const { unpack8(a, f); }
};
template <>
struct FRaw<float> {
    uint4 a, b;
    __device__ void load(const float *p) { a = ptx::ld_stream_v4(p); b = ptx::ld_stream_v4(p + 4); }
    __device__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ void get(float (&f)[8]) const
    {
        f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y);
        f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
        f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y);
        f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
    }
};

template <int n, typename FT, int kWarps>
__global__ void __launch_bounds__(kWarps * 32)
post_backward_kernel(const uint16_t *__restrict__ dX_next, const uint8_t *__restrict__ Xq,
                     const uint8_t *__restrict__ Xs, const FT *__restrict__ F_out,
                     const float *__restrict__ H_post, int64_t B, int64_t C,
                     FT *__restrict__ dF_out, float *__restrict__ dH_res,
                     float *__restrict__ dH_post)
{
    using S = Slots<n>;
    __shared__ float part[kWarps][3][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = lane & 3, slot = (lane >> 2) & (S::n2 - 1), tok = (lane >> 2) / S::n2;
    const int64_t nb = kept_blocks(C), groups = nb;
    ptx::pdl_wait();
    ptx::pdl_trigger();
    for (int64_t b0 = static_cast<int64_t>(blockIdx.x) * S::tokens; b0 < B;
         b0 += static_cast<int64_t>(gridDim.x) * S::tokens) {
        const int64_t b = b0 + tok;
        const bool have_tok = b < B && in_range(1101, b, 1, B);
        const bool have = have_tok && slot < n;
        const int64_t row = b * n + slot;
        const uint16_t *g_row = dX_next + row * C;
        const uint8_t *q_row = Xq + row * C;
        const uint8_t *s_row = Xs + row * nb;
        const FT *f_row = F_out + b * C;
        const float h = have ? __ldg(H_post + row) : 0.f;

        uint4 g;
        uint2 q;
        uint32_t E;
        FRaw<FT> fr;
        const auto load = [&](int64_t cg) {
            const int64_t c = cg * 32 + t * 8;
            const bool in = cg < groups && c < C;
            if (in && have && in_range(1102, c, 8, C)) {
                g = ptx::ld_stream_v4(g_row + c);
                q = kept::ld_stream_v2(q_row + c);
                E = __ldg(s_row + cg);
                fr.load(f_row + c);
            } else {
                g = make_uint4(0, 0, 0, 0);
                q = make_uint2(0, 0);
                E = kept::kScaleMin;
                fr.zero();
            }
        };
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        float dpost = 0.f;
        load(warp);
        for (int64_t cg = warp; cg < groups; cg += kWarps) {
            const uint4 x = kept::decode8_bf16(q, kept::scale_value(E));
            mma_16816(acc, x.x, x.y, g.x, g.y);
            mma_16816(acc, x.z, x.w, g.z, g.w);
            float v[8], f[8];
            unpack8(g, v);
            fr.get(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) dpost = fmaf(v[e], f[e], dpost);
            load(cg + kWarps);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= h;
            const int off = sum_over_slots<S::n2>(v, slot);
            const int64_t c = cg * 32 + t * 8 + off;
            if (have_tok && c < C && in_range(1103, c, 8 / S::n2, C))
                store_vals<8 / S::n2>(dF_out + b * C + c, v);
        }
        // over the four lanes of a slot, then over the warps
        dpost += __shfl_xor_sync(0xffffffffu, dpost, 1);
        dpost += __shfl_xor_sync(0xffffffffu, dpost, 2);
        part[warp][0][lane] = acc[0];
        part[warp][1][lane] = acc[1];
        part[warp][2][lane] = dpost;
        __syncthreads();
        if (warp < 3) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s += part[w][warp][lane];
            if (warp == 2) {
                if (have && t == 0 && in_range(1104, row, 1, B * n)) dH_post[row] = s;
            } else {
                // accumulator: row = the X slot of this lane's group, column = a G slot
                const int col = 2 * t + warp, i = col & (S::n2 - 1);
                if (have && i < n && col / S::n2 == tok && in_range(1105, (b * n + i) * n + slot, 1, B * n * n))
                    dH_res[(b * n + i) * n + slot] = s;
            }
        }
        __syncthreads();
    }
}

template <typename FT, int kWarps>
cudaError_t launch_w(const uint16_t *dX_next, const uint8_t *Xq, const uint8_t *Xs,
                     const FT *F_out, const float *H_post, int64_t B, int n, int64_t C, FT *dF_out,
                     float *dH_res, float *dH_post, cudaStream_t stream)
{
    switch (n) {
#define MHC_CASE(k)                                                                              \
    case k: {                                                                                    \
        const int64_t gs = (B + Slots<k>::tokens - 1) / Slots<k>::tokens;                        \
        const dim3 grid(static_cast<unsigned>(gs < 0x7fffffff ? gs : 0x7fffffff));               \
        return launch_pdl(post_backward_kernel<k, FT, kWarps>, grid, dim3(kWarps * 32), 0,       \
                          stream, dX_next, Xq, Xs, F_out, H_post, B, C, dF_out, dH_res, dH_post); \
    }
        MHC_CASE(1) MHC_CASE(2) MHC_CASE(3) MHC_CASE(4) MHC_CASE(5) MHC_CASE(6) MHC_CASE(7)
        MHC_CASE(8)
#undef MHC_CASE
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

template <typename FT>
cudaError_t launch_post_backward(const uint16_t *dX_next, const uint8_t *Xq, const uint8_t *Xs,
                                 const FT *F_out, const float *H_post, int64_t B, int n, int64_t C,
                                 FT *dF_out, float *dH_res, float *dH_post, int,
                                 cudaStream_t stream)
{
    return launch_w<FT, 8>(dX_next, Xq, Xs, F_out, H_post, B, n, C, dF_out, dH_res, dH_post,
                           stream);
}
template cudaError_t launch_post_backward<uint16_t>(const uint16_t *, const uint8_t *,
                                                    const uint8_t *, const uint16_t *,
                                                    const float *, int64_t, int, int64_t,
                                                    uint16_t *, float *, float *, int,
                                                    cudaStream_t);
template cudaError_t launch_post_backward<float>(const uint16_t *, const uint8_t *,
                                                 const uint8_t *, const float *, const float *,
                                                 int64_t, int, int64_t, float *, float *, float *,
                                                 int, cudaStream_t);

}  // namespace mhc
