// Keeping the n residual streams in 8 bits for the backward pass (the form is
// kept.cuh's), alone and together with the update that consumes them:
//
//   X_next[b][i][c] = Σ_j H_res[b][i][j]·X[b][j][c] + H_post[b][i]·F_out[b][c]
//   (codes, scales) = X as kept
//
// The update has X in registers anyway, so keeping it there costs the bytes of
// the codes and no second read of X; and X_next may then overwrite X.
//
// A thread owns 8 channels of one token in all n streams (128-bit accesses),
// so four neighbouring lanes hold a block of 32 channels and find its largest
// magnitude with two shuffles.  All kernels are bound by memory: at B=16384, n=4,
// C=7168 the update with the codes takes 384-400 us, 6.5-6.8 TB/s (a copy runs at 6.8),
// unpacking 200, 7.1 TB/s, packing 206, 6.9.  At n >= 5 the update with the codes is
// further from that: B=8192, n=8, C=4096 271 us, 5.2 TB/s (256 with F_out in fp32; the
// update alone, whose kernel walks tokens, 170): a CTA a token and two an SM.
#include <cuda_runtime.h>

#include <cstdint>

#include "check.cuh"
#include "kept.cuh"
#include "mix.cuh"
#include "ptx.cuh"
#include "train.h"

namespace mhc {
namespace {

constexpr int kMaxGridY = 65535;

// The largest magnitude over the four lanes of a block.
__device__ __forceinline__ uint32_t block_amax(uint32_t a)
{
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    return max(a, __shfl_xor_sync(0xffffffffu, a, 2));
}

// Codes and scale of 8 channels (chunk c8) of one stream row.  Every lane of
// the warp calls it; a lane without channels passes zeros and live = false.
__device__ __forceinline__ void keep8(const uint4 &x, bool live, int64_t row, int64_t c8,
                                      int64_t C, int64_t nb, uint8_t *Xq, uint8_t *Xs)
{
    const uint32_t E = kept::scale_code(block_amax(kept::amax8(x)));
    if (!live) return;
    kept::st_stream_v2(Xq + row * C + c8 * 8, kept::encode8(x, E));
    if ((c8 & 3) == 0) Xs[row * nb + (c8 >> 2)] = static_cast<uint8_t>(E);
}

template <int n, typename FT>
__global__ void __launch_bounds__(256, n <= 4 ? 4 : 2)
post_res_ckpt_kernel(const uint16_t *X, const FT *__restrict__ F_out,
                     const float *__restrict__ H_res, const float *__restrict__ H_post, int64_t B,
                     int64_t C, uint16_t *X_next, uint8_t *__restrict__ Xq,
                     uint8_t *__restrict__ Xs)
{
    __shared__ float hs[n * n + n];
    const int64_t C8 = C >> 3, nb = kept_blocks(C);
    const int64_t c8 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    ptx::pdl_wait();
    ptx::pdl_trigger();
    for (int64_t b = blockIdx.y; b < B; b += gridDim.y) {
        const bool tok_ok = in_range(1001, b, 1, B);
        const bool ok = c8 < C8 && tok_ok && in_range(1002, c8 * 8, 8, C);
        uint4 xv[n];
        float f[8];
        if (ok) {
#pragma unroll
            for (int j = 0; j < n; ++j) xv[j] = ptx::ld_stream_v4(X + (b * n + j) * C + c8 * 8);
            kept::load_f8(F_out + b * C + c8 * 8, f);
        } else {
#pragma unroll
            for (int j = 0; j < n; ++j) xv[j] = make_uint4(0, 0, 0, 0);
        }
        __syncthreads();  // the previous token's coefficients are no longer read
        for (int t = threadIdx.x; t < n * n + n; t += blockDim.x)
            if (tok_ok)
                hs[t] = t < n * n ? ptx::ld_dep(H_res + b * n * n + t) : ptx::ld_dep(H_post + b * n + (t - n * n));
        __syncthreads();
#pragma unroll
        for (int j = 0; j < n; ++j) keep8(xv[j], ok, b * n + j, c8, C, nb, Xq, Xs);
        if (ok) {
#pragma unroll
            for (int i = 0; i < n; ++i)
                ptx::st_stream_v4(X_next + (b * n + i) * C + c8 * 8, post_mix8<n>(hs, i, xv, f));
        }
    }
}

// Packing and unpacking alone: the rows of all tokens and streams are alike.  A
// thread takes its 8 channels of kRows neighbouring rows, all loads first: with
// one row a thread there were too few bytes in flight (unpacking B=16384, n=4,
// C=7168: 463 us, against a floor of 210).
constexpr int kRows = 4;

__global__ void __launch_bounds__(256)
ckpt_pack_kernel(const uint16_t *__restrict__ X, int64_t rows, int64_t C,
                 uint8_t *__restrict__ Xq, uint8_t *__restrict__ Xs)
{
    const int64_t C8 = C >> 3, nb = kept_blocks(C);
    const int64_t c8 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    ptx::pdl_wait();
    ptx::pdl_trigger();
    for (int64_t row = static_cast<int64_t>(blockIdx.y) * kRows; row < rows;
         row += static_cast<int64_t>(gridDim.y) * kRows) {
        uint4 x[kRows];
        bool ok[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            ok[k] = c8 < C8 && row + k < rows && in_range(1011, row + k, 1, rows);
            x[k] = ok[k] ? ptx::ld_stream_v4(X + (row + k) * C + c8 * 8) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) keep8(x[k], ok[k], row + k, c8, C, nb, Xq, Xs);
    }
}

__global__ void __launch_bounds__(256)
ckpt_unpack_kernel(const uint8_t *__restrict__ Xq, const uint8_t *__restrict__ Xs, int64_t rows,
                   int64_t C, uint16_t *__restrict__ X)
{
    const int64_t C8 = C >> 3, nb = kept_blocks(C);
    const int64_t c8 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    ptx::pdl_wait();
    ptx::pdl_trigger();
    if (c8 >= C8) return;
    for (int64_t row = static_cast<int64_t>(blockIdx.y) * kRows; row < rows;
         row += static_cast<int64_t>(gridDim.y) * kRows) {
        uint2 q[kRows];
        uint32_t E[kRows];
        bool ok[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            ok[k] = row + k < rows && in_range(1021, row + k, 1, rows);
            q[k] = make_uint2(0, 0);
            E[k] = kept::kScaleMin;
            if (!ok[k]) continue;
            q[k] = kept::ld_stream_v2(Xq + (row + k) * C + c8 * 8);
            E[k] = ptx::ld_dep(Xs + (row + k) * nb + (c8 >> 2));
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k)
            if (ok[k])
                ptx::st_stream_v4(X + (row + k) * C + c8 * 8,
                                  kept::decode8_bf16(q[k], E[k]));
    }
}

// Threads per block: a power of two that divides C/8 when one exists, otherwise 128.
int block_threads(int64_t C8)
{
    for (int t : {256, 128, 64, 32})
        if (C8 % t == 0) return t;
    return 128;
}

dim3 row_grid(int64_t rows, int64_t C8, int threads)
{
    const int64_t gx = (C8 + threads - 1) / threads;
    return dim3(static_cast<unsigned>(gx),
                static_cast<unsigned>(rows < kMaxGridY ? rows : kMaxGridY), 1);
}

}  // namespace

template <typename FT>
cudaError_t launch_post_res_ckpt(const uint16_t *X, const FT *F_out, const float *H_res,
                                 const float *H_post, int64_t B, int n, int64_t C,
                                 uint16_t *X_next, uint8_t *Xq, uint8_t *Xs, cudaStream_t stream)
{
    const int threads = block_threads(C / 8);
    const dim3 grid = row_grid(B, C / 8, threads);
    switch (n) {
#define MHC_CASE(k)                                                                            \
    case k:                                                                                    \
        return launch_pdl(post_res_ckpt_kernel<k, FT>, grid, dim3(threads), 0, stream, X,      \
                          F_out, H_res, H_post, B, C, X_next, Xq, Xs);
        MHC_CASE(1) MHC_CASE(2) MHC_CASE(3) MHC_CASE(4) MHC_CASE(5) MHC_CASE(6) MHC_CASE(7)
        MHC_CASE(8)
#undef MHC_CASE
    default: return cudaErrorInvalidValue;
    }
}
template cudaError_t launch_post_res_ckpt<uint16_t>(const uint16_t *, const uint16_t *,
                                                    const float *, const float *, int64_t, int,
                                                    int64_t, uint16_t *, uint8_t *, uint8_t *,
                                                    cudaStream_t);
template cudaError_t launch_post_res_ckpt<float>(const uint16_t *, const float *, const float *,
                                                 const float *, int64_t, int, int64_t, uint16_t *,
                                                 uint8_t *, uint8_t *, cudaStream_t);

cudaError_t launch_ckpt_pack(const uint16_t *X, int64_t B, int n, int64_t C, uint8_t *Xq,
                             uint8_t *Xs, cudaStream_t stream)
{
    const int threads = block_threads(C / 8);
    return launch_pdl(ckpt_pack_kernel, row_grid((B * n + kRows - 1) / kRows, C / 8, threads),
                      dim3(threads), 0, stream, X, B * n, C, Xq, Xs);
}

cudaError_t launch_ckpt_unpack(const uint8_t *Xq, const uint8_t *Xs, int64_t B, int n, int64_t C,
                               uint16_t *X, cudaStream_t stream)
{
    const int threads = block_threads(C / 8);
    return launch_pdl(ckpt_unpack_kernel, row_grid((B * n + kRows - 1) / kRows, C / 8, threads),
                      dim3(threads), 0, stream, Xq, Xs, B * n, C, X);
}

}  // namespace mhc
