// Root-mean-square norms at the entry of the layer function F, and their backward.
//
//   streams    H = Σ_i H_pre[i]·X[i]   (F_pre: step 4a)
//   residual   H = A + R
//   both       rstd = 1/sqrt(Σ_c H[c]²/C + eps),  Z[c] = H[c]·rstd·gain[c]
//
// with Z in bf16 or in the 8-bit form of kept.cuh.  H is held in fp32 registers from the
// mixing to the scaling, so the inputs are read once and each output is rounded once.
// Bound by memory.
//
// A group of G threads takes a token, a thread chunks of 8 channels g, g + G, ...; the
// sum of squares is added in a fixed order, by lane, warp and then warps in order.
#include <cuda_runtime.h>

#include <cstdint>

#include "check.cuh"
#include "mix.cuh"
#include "model.h"
#include "ptx.cuh"
#include "train/kept.cuh"

namespace mhc {
namespace {

constexpr int kMaxThreads = 512;

// How a token of C channels is laid over threads: `items` chunks of 8 channels a thread,
// `group` threads a token, `tokens` tokens a block.
struct Layout {
    int items, group, tokens;
};
Layout layout_of(int64_t C)
{
    const int c8 = static_cast<int>(C / 8);
    Layout l;
    l.items = c8 <= 256 ? 1 : c8 <= 1024 ? 2 : 4;
    l.group = (((c8 + l.items - 1) / l.items) + 31) / 32 * 32;
    l.tokens = l.group >= 256 ? 1 : 256 / l.group;
    return l;
}

// Sum of v over the threads of a group.  Every thread of the block calls it; `red` holds a
// value a warp and is not written again before every thread has passed the next call's
// barrier (callers alternate between two).
__device__ __forceinline__ float group_sum(float v, float *red, int first_warp, int warps)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < warps; ++w) s += red[first_warp + w];
    return s;
}

template <int n>  // streams, or 0: A + R
__device__ __forceinline__ void load_mixed(const NormArgs &a, int64_t b, int64_t c8, float (&f)[8])
{
    float t[8];
    if constexpr (n == 0) {
        unpack8(ptx::ld_stream_v4(a.X + b * a.C + c8 * 8), f);
        if (a.R != nullptr) {
            unpack8(ptx::ld_stream_v4(a.R + b * a.C + c8 * 8), t);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] += t[e];
        }
    } else {
        uint4 xv[n];
        float h[n];
#pragma unroll
        for (int i = 0; i < n; ++i) xv[i] = ptx::ld_stream_v4(a.X + (b * n + i) * a.C + c8 * 8);
#pragma unroll
        for (int i = 0; i < n; ++i) h[i] = ptx::ld_dep(a.H_pre + b * n + i);
        unpack8(xv[0], t);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = h[0] * t[e];
#pragma unroll
        for (int i = 1; i < n; ++i) {
            unpack8(xv[i], t);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = fmaf(h[i], t[e], f[e]);
        }
    }
}

__device__ __forceinline__ void load_gain(const float *gain, int64_t c8, float (&g)[8])
{
    const uint4 u = ptx::ld_dep_v4(gain + c8 * 8), v = ptx::ld_dep_v4(gain + c8 * 8 + 4);
    g[0] = __uint_as_float(u.x); g[1] = __uint_as_float(u.y);
    g[2] = __uint_as_float(u.z); g[3] = __uint_as_float(u.w);
    g[4] = __uint_as_float(v.x); g[5] = __uint_as_float(v.y);
    g[6] = __uint_as_float(v.z); g[7] = __uint_as_float(v.w);
}

template <int n, int ITEMS, bool Q8>
__global__ void __launch_bounds__(kMaxThreads) rmsnorm_kernel(const NormArgs a, int G, int T)
{
    __shared__ float red[2][kMaxThreads / 32];
    const int group = threadIdx.x / G, g = threadIdx.x % G, warps = G >> 5;
    const int64_t C8 = a.C >> 3, nb = kept_blocks(a.C);
    ptx::pdl_wait();
    ptx::pdl_trigger();
    int turn = 0;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * T; first < a.B;
         first += static_cast<int64_t>(gridDim.x) * T, turn ^= 1) {
        const int64_t b = first + group;
        const bool have = b < a.B && in_range(1501, b, 1, a.B);
        float f[ITEMS][8], ss = 0.f;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int64_t c8 = k * G + g;
            if (have && c8 < C8) {
                load_mixed<n>(a, b, c8, f[k]);
                if (a.H != nullptr) ptx::st_stream_v4(a.H + b * a.C + c8 * 8, pack8(f[k]));
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[k][e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(f[k][e], f[k][e], ss);
        }
        const float ms = group_sum(ss, red[turn], group * warps, warps) / static_cast<float>(a.C) + a.eps;
        const float rstd = ms != 0.f ? 1.0f / sqrtf(ms) : 0.f;
        if (a.rstd != nullptr && have && g == 0) a.rstd[b] = rstd;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int64_t c8 = k * G + g;
            const bool live = have && c8 < C8;
            float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (live) {
                float w[8];
                load_gain(a.gain, c8, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] = f[k][e] * rstd * w[e];
            }
            if constexpr (Q8) {
                uint32_t m = kept::amax8(z);
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const uint32_t E = kept::scale_code_f32(m);
                if (live) {
                    kept::st_stream_v2(a.Zq + b * a.C + c8 * 8, kept::encode8(z, E));
                    if ((c8 & 3) == 0) a.Zs[b * nb + (c8 >> 2)] = static_cast<uint8_t>(E);
                }
            } else if (live) {
                ptx::st_stream_v4(a.Z + b * a.C + c8 * 8, pack8(z));
            }
        }
    }
}

// Backward.  With t = gain·dZ and s = Σ_c t·H:
//   dH = rstd·(t − H·rstd²·s/C) + dH_skip,   dgain = Σ_b dZ·H·rstd
// The blocks walk the tokens; a thread meets the same channels in each of them, so it
// holds their share of dgain in fp32 registers.  A block's sums go to its row of the
// workspace, and a second launch adds the rows in order.
constexpr int kBackwardBlocks = 2;  // blocks an SM

template <int ITEMS>
__global__ void __launch_bounds__(kMaxThreads)
rmsnorm_backward_kernel(const NormBackwardArgs a, int G, int T, float *__restrict__ parts)
{
    __shared__ float red[2][kMaxThreads / 32];
    __shared__ float4 join[ITEMS == 1 ? 2 * kMaxThreads : 1];
    const int group = threadIdx.x / G, g = threadIdx.x % G, warps = G >> 5;
    const int64_t C8 = a.C >> 3;
    ptx::pdl_wait();
    ptx::pdl_trigger();
    float acc[ITEMS][8];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[k][e] = 0.f;
    int turn = 0;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * T; first < a.B;
         first += static_cast<int64_t>(gridDim.x) * T, turn ^= 1) {
        const int64_t b = first + group;
        const bool have = b < a.B && in_range(1511, b, 1, a.B);
        const float rstd = have ? ptx::ld_dep(a.rstd + b) : 0.f;
        uint4 dz[ITEMS], hv[ITEMS], sk[ITEMS];
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int64_t c8 = k * G + g;
            dz[k] = hv[k] = sk[k] = make_uint4(0, 0, 0, 0);
            if (have && c8 < C8) {
                dz[k] = ptx::ld_stream_v4(a.dZ + b * a.C + c8 * 8);
                hv[k] = ptx::ld_stream_v4(a.H + b * a.C + c8 * 8);
                if (a.dH_skip != nullptr) sk[k] = ptx::ld_stream_v4(a.dH_skip + b * a.C + c8 * 8);
            }
        }
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int64_t c8 = k * G + g;
            float d[8], h[8], w[8];
            unpack8(dz[k], d);
            unpack8(hv[k], h);
            if (c8 < C8) {
                load_gain(a.gain, c8, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s = fmaf(w[e] * d[e], h[e], s);
                    acc[k][e] = fmaf(d[e] * rstd, h[e], acc[k][e]);
                }
            }
        }
        const float sum = group_sum(s, red[turn], group * warps, warps);
        const float back = rstd * rstd * (sum / static_cast<float>(a.C));
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int64_t c8 = k * G + g;
            if (!have || c8 >= C8) continue;
            float d[8], h[8], w[8], o[8];
            unpack8(dz[k], d);
            unpack8(hv[k], h);
            unpack8(sk[k], o);
            load_gain(a.gain, c8, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = fmaf(rstd, fmaf(-h[e], back, w[e] * d[e]), o[e]);
            ptx::st_stream_v4(a.dH + b * a.C + c8 * 8, pack8(o));
        }
    }
    // the sums of a block's tokens, group by group
    if constexpr (ITEMS == 1) {
        join[2 * threadIdx.x] = make_float4(acc[0][0], acc[0][1], acc[0][2], acc[0][3]);
        join[2 * threadIdx.x + 1] = make_float4(acc[0][4], acc[0][5], acc[0][6], acc[0][7]);
        __syncthreads();
        if (group != 0) return;
        for (int k = 1; k < T; ++k) {
            const float4 u = join[2 * (k * G + g)], v = join[2 * (k * G + g) + 1];
            acc[0][0] += u.x; acc[0][1] += u.y; acc[0][2] += u.z; acc[0][3] += u.w;
            acc[0][4] += v.x; acc[0][5] += v.y; acc[0][6] += v.z; acc[0][7] += v.w;
        }
    }
    float *row = parts + static_cast<int64_t>(blockIdx.x) * a.C;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int64_t c8 = k * G + g;
        if (c8 >= C8 || !in_range(1512, c8 * 8, 8, a.C)) continue;
        *reinterpret_cast<float4 *>(row + c8 * 8) = make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3]);
        *reinterpret_cast<float4 *>(row + c8 * 8 + 4) = make_float4(acc[k][4], acc[k][5], acc[k][6], acc[k][7]);
    }
}

// dgain (+)= the rows of `parts`, by slices of rows and then slices in order.
constexpr int kJoinCols = 32, kJoinSlices = 8;
__global__ void __launch_bounds__(kJoinCols * kJoinSlices)
rmsnorm_join_kernel(const float *parts, int rows, int64_t C, int accumulate, float *dgain)
{
    __shared__ float part[kJoinSlices][kJoinCols];
    const int col = threadIdx.x % kJoinCols, slice = threadIdx.x / kJoinCols;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kJoinCols + col;
    ptx::pdl_wait();
    ptx::pdl_trigger();
    float s = 0.f;
    if (c < C)
#pragma unroll 4
        for (int r = slice; r < rows; r += kJoinSlices) s += ptx::ld_dep(parts + r * C + c);
    part[slice][col] = s;
    __syncthreads();
    if (slice != 0 || c >= C) return;
#pragma unroll
    for (int k = 1; k < kJoinSlices; ++k) s += part[k][col];
    dgain[c] = accumulate ? ptx::ld_dep(dgain + c) + s : s;
}

int backward_blocks(int64_t B, int64_t C, int num_sms)
{
    const Layout l = layout_of(C);
    const int64_t all = (B + l.tokens - 1) / l.tokens, most = static_cast<int64_t>(kBackwardBlocks) * num_sms;
    return static_cast<int>(all < most ? all : most);
}

template <int n, bool Q8>
cudaError_t launch_forward_n(const NormArgs &a, int num_sms, cudaStream_t stream)
{
    const Layout l = layout_of(a.C);
    const int64_t all = (a.B + l.tokens - 1) / l.tokens, most = int64_t{1} << 30;
    const dim3 grid(static_cast<unsigned>(all < most ? all : most)), block(l.group * l.tokens);
    switch (l.items) {
    case 1: return launch_pdl(rmsnorm_kernel<n, 1, Q8>, grid, block, 0, stream, a, l.group, l.tokens);
    case 2: return launch_pdl(rmsnorm_kernel<n, 2, Q8>, grid, block, 0, stream, a, l.group, l.tokens);
    default: return launch_pdl(rmsnorm_kernel<n, 4, Q8>, grid, block, 0, stream, a, l.group, l.tokens);
    }
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs &a, int num_sms, cudaStream_t stream)
{
    switch (a.n) {
#define MHC_CASE(k)                                                             \
    case k:                                                                     \
        return a.Zq != nullptr ? launch_forward_n<k, true>(a, num_sms, stream)  \
                               : launch_forward_n<k, false>(a, num_sms, stream);
        MHC_CASE(0) MHC_CASE(1) MHC_CASE(2) MHC_CASE(3) MHC_CASE(4) MHC_CASE(5) MHC_CASE(6)
        MHC_CASE(7) MHC_CASE(8)
#undef MHC_CASE
    default: return cudaErrorInvalidValue;
    }
}

size_t rmsnorm_backward_workspace_bytes(int64_t B, int64_t C, int num_sms)
{
    return static_cast<size_t>(backward_blocks(B, C, num_sms)) * C * sizeof(float);
}

cudaError_t launch_rmsnorm_backward(const NormBackwardArgs &a, void *workspace, int num_sms,
                                    cudaStream_t stream)
{
    const Layout l = layout_of(a.C);
    const int blocks = backward_blocks(a.B, a.C, num_sms);
    const dim3 grid(blocks), block(l.group * l.tokens);
    float *parts = static_cast<float *>(workspace);
    cudaError_t e;
    switch (l.items) {
    case 1: e = launch_pdl(rmsnorm_backward_kernel<1>, grid, block, 0, stream, a, l.group, l.tokens, parts); break;
    case 2: e = launch_pdl(rmsnorm_backward_kernel<2>, grid, block, 0, stream, a, l.group, l.tokens, parts); break;
    default: e = launch_pdl(rmsnorm_backward_kernel<4>, grid, block, 0, stream, a, l.group, l.tokens, parts); break;
    }
    if (e != cudaSuccess) return e;
    return launch_pdl(rmsnorm_join_kernel, dim3(static_cast<unsigned>((a.C + kJoinCols - 1) / kJoinCols)),
                      dim3(kJoinCols * kJoinSlices), 0, stream, parts, blocks, a.C, a.accumulate, a.dgain);
}

}  // namespace mhc
