// Launchers of the training operators, shared between their translation units.
// Arguments have already been validated by train_api.cu when these run.
//
// Sites of the device index checks (check.cuh) here: 1000s ckpt.cu, 1100s
// post_backward.cu, 1200s pre_backward.cu, 1300s phi_grad.cu, 1400s embed.cu.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>

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
size_t pre_backward_workspace_bytes(int64_t B, int n, int64_t C, int iters, int num_sms);
cudaError_t launch_pre_backward(const PreBackwardArgs &a, void *workspace, int num_sms,
                                cudaStream_t stream);

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
size_t phi_grad_workspace_bytes(int64_t B, int n, int64_t C, int num_sms);
cudaError_t launch_phi_grad(const uint8_t *Xq, const uint8_t *Xs, const uint16_t *dY_terms,
                            int64_t B, int n, int64_t C, int accumulate, float *dphi_t,
                            void *workspace, int num_sms, cudaStream_t stream);
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
