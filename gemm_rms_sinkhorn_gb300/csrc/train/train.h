// Launchers of the training operators, shared between their translation units.
// Arguments have already been validated by train_api.cu when these run.
//
// Sites of the device index checks (check.cuh) here: 1000s ckpt.cu, 1100s
// post_backward.cu, 1200s pre_backward.cu and (1240s) streams.cu, 1300s
// phi_grad.cu, 1400s embed.cu.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "mhc_internal.h"

namespace mhc {

// Runs `set` the first time on each device (attributes of kernels are kept per
// device); the bits of `done` are devices.
template <typename F>
cudaError_t once_per_device(std::atomic<uint64_t> &done, F set)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
    if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
    if ((e = set()) == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// A tensor of `rank` dimensions, innermost first, densely packed, read in boxes of
// box[] elements of 1 or 2 bytes, whose rows are swizzled by their width where that
// is 32, 64 or 128 bytes (tensor_map.cu).  False when there is no such map.
bool encode_tensor(CUtensorMap *m, int esize, int rank, const void *base, const int64_t *dims,
                   const int *box);

constexpr int kKeptBlock = 32;  // channels that share a scale
__host__ __device__ inline int64_t kept_blocks(int64_t C)
{
    return (C + kKeptBlock - 1) / kKeptBlock;
}

// ---- X in 8 bits (ckpt.cu)
cudaError_t launch_ckpt_pack(const uint16_t *X, int64_t B, int n, int64_t C, uint8_t *Xq,
                             uint8_t *Xs, cudaStream_t stream);
cudaError_t launch_ckpt_unpack(const uint8_t *Xq, const uint8_t *Xs, int64_t B, int n, int64_t C,
                               uint16_t *X, cudaStream_t stream);
template <typename FT>  // uint16_t (bf16) or float
cudaError_t launch_post_res_ckpt(const uint16_t *X, const FT *F_out, const float *H_res,
                                 const float *H_post, int64_t B, int n, int64_t C,
                                 uint16_t *X_next, uint8_t *Xq, uint8_t *Xs, cudaStream_t stream);

// ---- backward of X_next = H_res·X + H_post ⊗ F_out (post_backward.cu)
template <typename FT>
cudaError_t launch_post_backward(const uint16_t *dX_next, const uint8_t *Xq, const uint8_t *Xs,
                                 const FT *F_out, const float *H_post, int64_t B, int n, int64_t C,
                                 FT *dF_out, float *dH_res, float *dH_post, int num_sms,
                                 cudaStream_t stream);

// Every wait of the dX and dφ kernels gives up after limit_ns of GPU time.  For tests of
// that, CTA 0 of one of them leaves its unit of this number without its copies.
struct Waits {
    uint64_t limit_ns = kWaitLimitNs;
    int64_t stall_dx = -1, stall_dphi = -1;
};

// ---- backward of steps 1-4a (pre_backward.cu)
struct PreBackwardArgs {
    const uint16_t *dX_next, *dF_pre;
    const uint8_t *Xq, *Xs;
    const uint16_t *phi_t;
    float a_pre, a_post, a_res;
    const float *bias;
    int iters;
    const float *Y, *r, *H_pre, *H_post, *H_res, *dH_res, *dH_post;
    int accumulate;
    int64_t B;
    int n;
    int64_t C;
    uint16_t *dX;
    float *dphi_t, *dbias, *dalpha;
};
// The Sinkhorn steps' history, indexed in 32 bits, takes up to 16 values a step and thread of 64.
constexpr int kMaxBackwardIters = (1 << 21) - 1;
size_t pre_backward_workspace_bytes(int64_t B, int n, int64_t C, int iters, int num_sms);
cudaError_t launch_pre_backward(const PreBackwardArgs &a, void *workspace, int num_sms,
                                cudaStream_t stream, const Waits &waits);

// ---- dX (streams.cu)
// k of the product dY·φ, padded to the tensor instruction's 16
__host__ __device__ constexpr int dy_cols(int n) { return (n * n + 2 * n + 15) / 16 * 16; }
// what mixes a token's streams: H_resᵀ [j][i], H_pre[j], s
__host__ __device__ constexpr int mix_vals(int n) { return n * n + n + 1; }
// Channels of a unit of streams.cu, and how φ is laid out for it: for each chunk of
// that many channels, rows (j, channel) of k in bf16, phi_image_row bytes each with
// the 16-byte pieces swizzled as the tensor cores read them; for n = 8 the k past
// 64 in rows of their own behind them.
__host__ __device__ constexpr int streams_width(int n) { return n <= 4 ? 64 : 32; }
__host__ __device__ constexpr int phi_image_row(int n)
{
    return dy_cols(n) <= 16 ? 32 : dy_cols(n) <= 32 ? 64 : 128;
}
__host__ __device__ constexpr int phi_image_row2(int n) { return dy_cols(n) > 64 ? 32 : 0; }
__host__ __device__ constexpr int64_t phi_image_bytes(int n)  // of a chunk
{
    return static_cast<int64_t>(n) * streams_width(n) * (phi_image_row(n) + phi_image_row2(n));
}
// dY as two bf16 terms that add up to it to 2^-16 of its size.
constexpr int kRowTerms = 2;
// What a row's 16-byte piece numbers are XORed with, in rows of `bytes`.
__host__ __device__ constexpr int swizzle_xor(int bytes, int row)
{
    return bytes == 128 ? row & 7 : bytes == 64 ? row >> 1 & 3 : bytes == 32 ? row >> 2 & 1 : 0;
}
struct StreamsArgs {
    const uint16_t *dX_next, *dF;
    const uint8_t *phi_img;    // [chunks][phi_image_bytes]
    const uint16_t *dY_rows;   // [kRowTerms][Bp][dy_cols], zeros past N
    const uint8_t *Xq, *Xs;
    const float *mix;          // [mix_vals][Bp]
    int64_t B, Bp, C;          // Bp: tokens, padded
    uint16_t *dX;
};
cudaError_t launch_streams(const StreamsArgs &s, int n, int num_sms, cudaStream_t stream,
                           const Waits &waits);
cudaError_t read_and_clear_streams_status(int *status);

// ---- dφ (phi_grad.cu)
// dY in three bf16 terms that add up to it (to about 2^-26 of its size): the hi
// terms of 16 columns in 16 rows, then their mid and low terms, for each 16
// columns (rows of columns past N hold anything); tokens contiguous and padded
// with zeros to a multiple of kPhiTokens.
constexpr int kPhiTerms = 3;
constexpr int kPhiTokens = 64;
__host__ __device__ constexpr int phi_term_row(int k, int term)
{
    return k / 16 * (16 * kPhiTerms) + term * 16 + k % 16;
}
__host__ __device__ constexpr int phi_term_rows(int N) { return (N + 15) / 16 * 16 * kPhiTerms; }
inline int64_t phi_grad_padded_tokens(int64_t B)
{
    return (B + kPhiTokens - 1) / kPhiTokens * kPhiTokens;
}
// Sums of dH̃ by CTA of what formed it, [ctas][N + 3] (columns, then the α), which
// the last launch adds up beside dφ's parts.
struct BiasSums {
    const float *part;
    int ctas;
    float *dbias, *dalpha;
};
size_t phi_grad_workspace_bytes(int64_t B, int n, int64_t C, int num_sms);
cudaError_t launch_phi_grad(const uint8_t *Xq, const uint8_t *Xs, const uint16_t *dY_terms,
                            int64_t B, int n, int64_t C, int accumulate, float *dphi_t,
                            void *workspace, const BiasSums &bs, int num_sms, cudaStream_t stream,
                            const Waits &waits);
cudaError_t read_and_clear_phi_grad_status(int *status);

// ---- token ids to streams and back (embed.cu)
template <typename T>  // the table's element: uint16_t (bf16) or float
cudaError_t launch_embed(const T *table, const int64_t *ids, float scale, int64_t V, int64_t B,
                         int n, int64_t C, uint16_t *X, cudaStream_t stream);
size_t embed_backward_workspace_bytes(int64_t V, int64_t B, int n, int64_t C);
cudaError_t launch_embed_backward(const uint16_t *dX, const int64_t *ids, float scale,
                                  int accumulate, int64_t V, int64_t B, int n, int64_t C,
                                  float *dtable, void *workspace, int num_sms,
                                  cudaStream_t stream);

}  // namespace mhc
