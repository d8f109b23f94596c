// C ABI of the training operators (declared in include/mhc.h): argument
// validation on the host, then their kernels on the caller's stream.  No
// exception crosses this boundary and nothing here allocates device memory.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "host/args.h"
#include "mhc.h"
#include "mhc_testing.h"
#include "train.h"

using namespace mhc;

namespace {

size_t codes_bytes(int64_t B, int n, int64_t C) { return static_cast<size_t>(B * n * C); }
size_t scales_bytes(int64_t B, int n, int64_t C)
{
    return static_cast<size_t>(B * n * kept_blocks(C));
}

// The checks that follow the shape rules, in the order of the other calls:
// pointers, overlaps, device, memory.  `ws` (may be NULL): the workspace, which
// needs `need(num_sms)` bytes.
template <typename Need>
int check_buffers(const Buf *ins, int n_in, Buf *outs, int n_out, const void *alias_out,
                  const void *alias_in, Buf *ws, Need need, DeviceInfo *info)
{
    MHC_TRY(check_ptrs(ins, n_in));
    MHC_TRY(check_ptrs(outs, n_out));
    MHC_TRY(check_overlap(outs, n_out, ins, n_in, alias_out, alias_in));
    MHC_TRY(check_device(info));
    MHC_TRY(check_on_device(ins, n_in, *info));
    MHC_TRY(check_on_device(outs, n_out, *info));
    if (ws != nullptr) {
        const size_t bytes = need(info->num_sms);
        if (ws->p == nullptr || ws->bytes < bytes) return MHC_ERR_WORKSPACE;
        const Buf w = {ws->p, bytes};
        MHC_TRY(check_ptrs(&w, 1));
        MHC_TRY(check_overlap(&w, 1, ins, n_in, nullptr, nullptr));
        MHC_TRY(check_overlap(&w, 1, outs, n_out, nullptr, nullptr));
        MHC_TRY(check_on_device(&w, 1, *info));
    }
    return MHC_OK;
}

int check_buffers(const Buf *ins, int n_in, Buf *outs, int n_out, const void *alias_out,
                  const void *alias_in, DeviceInfo *info)
{
    return check_buffers(ins, n_in, outs, n_out, alias_out, alias_in, nullptr,
                         [](int) { return size_t{0}; }, info);
}

cudaStream_t cu(mhc_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Gradients of weights that no token touches: zero unless they are added to.
int zero_grads(const Buf *outs, int count, int accumulate, mhc_stream_t stream)
{
    if (accumulate) return MHC_OK;
    MHC_TRY(check_ptrs(outs, count));
    DeviceInfo info;
    MHC_TRY(check_device(&info));
    MHC_TRY(check_on_device(outs, count, info));
    for (int i = 0; i < count; ++i)
        if (cudaMemsetAsync(const_cast<void *>(outs[i].p), 0, outs[i].bytes, cu(stream)) !=
            cudaSuccess)
            return MHC_ERR_CUDA;
    return MHC_OK;
}

// Shape rules of the token table.
int check_table(int64_t V, int64_t B, int n, int64_t C, float scale)
{
    MHC_TRY(check_shape(B, n, C, true));
    if (V < 1 || !std::isfinite(scale)) return MHC_ERR_INVALID;
    if (V >= (int64_t{1} << 31)) return MHC_ERR_UNSUPPORTED;
    return MHC_OK;
}

template <typename T>
int embed_checked(const T *table, const int64_t *ids, float scale, int64_t V, int64_t B, int n,
                  int64_t C, mhc_bf16 *X, mhc_stream_t stream)
{
    MHC_TRY(check_table(V, B, n, C, scale));
    if (B == 0) return MHC_OK;
    const Buf ins[] = {{table, static_cast<size_t>(V * C) * sizeof(T)},
                       {ids, static_cast<size_t>(B) * 8}};
    Buf outs[] = {{X, bf16_bytes(B * n * C)}};
    DeviceInfo info;
    MHC_TRY(check_buffers(ins, 2, outs, 1, nullptr, nullptr, &info));
    return cuda_status(launch_embed(table, ids, scale, V, B, n, C, X, cu(stream)));
}

template <typename FT>
int post_res_ckpt_checked(const mhc_bf16 *X, const FT *F_out, const float *H_res,
                          const float *H_post, int64_t B, int n, int64_t C, mhc_bf16 *X_next,
                          uint8_t *Xq, uint8_t *Xs, mhc_stream_t stream)
{
    MHC_TRY(check_shape(B, n, C, true));
    if (B == 0) return MHC_OK;
    const Buf ins[] = {{X, bf16_bytes(B * n * C)},
                       {F_out, static_cast<size_t>(B * C) * sizeof(FT)},
                       {H_res, f32_bytes(B * n * n)}, {H_post, f32_bytes(B * n)}};
    Buf outs[] = {{X_next, bf16_bytes(B * n * C)}, {Xq, codes_bytes(B, n, C)},
                  {Xs, scales_bytes(B, n, C)}};
    DeviceInfo info;
    MHC_TRY(check_buffers(ins, 4, outs, 3, X_next, X, &info));
    return cuda_status(launch_post_res_ckpt(X, F_out, H_res, H_post, B, n, C, X_next, Xq, Xs,
                                            cu(stream)));
}

template <typename FT>
int post_backward_checked(const mhc_bf16 *dX_next, const uint8_t *Xq, const uint8_t *Xs,
                          const FT *F_out, const float *H_post, int64_t B, int n, int64_t C,
                          FT *dF_out, float *dH_res, float *dH_post, mhc_stream_t stream)
{
    MHC_TRY(check_shape(B, n, C, true));
    if (B == 0) return MHC_OK;
    const size_t f = static_cast<size_t>(B * C) * sizeof(FT);
    const Buf ins[] = {{dX_next, bf16_bytes(B * n * C)}, {Xq, codes_bytes(B, n, C)},
                       {Xs, scales_bytes(B, n, C)}, {F_out, f}, {H_post, f32_bytes(B * n)}};
    Buf outs[] = {{dF_out, f}, {dH_res, f32_bytes(B * n * n)}, {dH_post, f32_bytes(B * n)}};
    DeviceInfo info;
    MHC_TRY(check_buffers(ins, 5, outs, 3, nullptr, nullptr, &info));
    return cuda_status(launch_post_backward(dX_next, Xq, Xs, F_out, H_post, B, n, C, dF_out,
                                            dH_res, dH_post, info.num_sms, cu(stream)));
}

int pre_backward_checked(const PreBackwardArgs &a, void *workspace, size_t workspace_bytes,
                         mhc_stream_t stream, const Waits &waits)
{
    const int64_t B = a.B, C = a.C;
    const int n = a.n;
    MHC_TRY(check_shape(B, n, C, true));
    if (a.iters < 0) return MHC_ERR_INVALID;
    if (a.iters > kMaxBackwardIters) return MHC_ERR_UNSUPPORTED;
    const int N = num_coeffs(n);
    const int64_t K = n * C;
    Buf outs[] = {{a.dphi_t, f32_bytes(int64_t{N} * K)}, {a.dbias, f32_bytes(N)},
                  {a.dalpha, f32_bytes(3)}, {a.dX, bf16_bytes(B * K)}};
    if (B == 0) return zero_grads(outs, 3, a.accumulate, stream);
    const Buf ins[] = {{a.dX_next, bf16_bytes(B * K)}, {a.dF_pre, bf16_bytes(B * C)},
                       {a.Xq, codes_bytes(B, n, C)}, {a.Xs, scales_bytes(B, n, C)},
                       {a.phi_t, bf16_bytes(int64_t{N} * K)}, {a.bias, f32_bytes(N)},
                       {a.Y, f32_bytes(B * N)}, {a.r, f32_bytes(B)}, {a.H_pre, f32_bytes(B * n)},
                       {a.H_post, f32_bytes(B * n)}, {a.H_res, f32_bytes(B * n * n)},
                       {a.dH_res, f32_bytes(B * n * n)}, {a.dH_post, f32_bytes(B * n)}};
    Buf ws = {workspace, workspace_bytes};
    DeviceInfo info;
    MHC_TRY(check_buffers(
        ins, 13, outs, 4, a.dX, a.dX_next, &ws,
        [&](int sms) { return pre_backward_workspace_bytes(B, n, C, a.iters, sms); }, &info));
    return cuda_status(launch_pre_backward(a, workspace, info.num_sms, cu(stream), waits));
}

}  // namespace

extern "C" {

int mhc_embed(const mhc_bf16 *table, const int64_t *ids, float scale, int64_t V, int64_t B, int n,
              int64_t C, mhc_bf16 *X, mhc_stream_t stream)
{
    return embed_checked(table, ids, scale, V, B, n, C, X, stream);
}

int mhc_embed_f32(const float *table, const int64_t *ids, float scale, int64_t V, int64_t B,
                  int n, int64_t C, mhc_bf16 *X, mhc_stream_t stream)
{
    return embed_checked(table, ids, scale, V, B, n, C, X, stream);
}

size_t mhc_embed_backward_workspace_bytes(int64_t V, int64_t B, int n, int64_t C)
{
    if (check_table(V, B, n, C, 1.0f) != MHC_OK || B == 0) return 0;
    return embed_backward_workspace_bytes(V, B, n, C);
}

int mhc_embed_backward(const mhc_bf16 *dX, const int64_t *ids, float scale, int accumulate,
                       int64_t V, int64_t B, int n, int64_t C, float *dtable, void *workspace,
                       size_t workspace_bytes, mhc_stream_t stream)
{
    MHC_TRY(check_table(V, B, n, C, scale));
    Buf outs[] = {{dtable, f32_bytes(V * C)}};
    if (B == 0) return zero_grads(outs, 1, accumulate, stream);
    const Buf ins[] = {{dX, bf16_bytes(B * n * C)}, {ids, static_cast<size_t>(B) * 8}};
    Buf ws = {workspace, workspace_bytes};
    DeviceInfo info;
    MHC_TRY(check_buffers(ins, 2, outs, 1, nullptr, nullptr, &ws,
                          [&](int) { return embed_backward_workspace_bytes(V, B, n, C); }, &info));
    return cuda_status(launch_embed_backward(dX, ids, scale, accumulate != 0, V, B, n, C, dtable,
                                             workspace, info.num_sms, cu(stream)));
}

int mhc_ckpt_pack(const mhc_bf16 *X, int64_t B, int n, int64_t C, uint8_t *Xq, uint8_t *Xs,
                  mhc_stream_t stream)
{
    MHC_TRY(check_shape(B, n, C, true));
    if (B == 0) return MHC_OK;
    const Buf ins[] = {{X, bf16_bytes(B * n * C)}};
    Buf outs[] = {{Xq, codes_bytes(B, n, C)}, {Xs, scales_bytes(B, n, C)}};
    DeviceInfo info;
    MHC_TRY(check_buffers(ins, 1, outs, 2, nullptr, nullptr, &info));
    return cuda_status(launch_ckpt_pack(X, B, n, C, Xq, Xs, cu(stream)));
}

int mhc_ckpt_unpack(const uint8_t *Xq, const uint8_t *Xs, int64_t B, int n, int64_t C,
                    mhc_bf16 *X, mhc_stream_t stream)
{
    MHC_TRY(check_shape(B, n, C, true));
    if (B == 0) return MHC_OK;
    const Buf ins[] = {{Xq, codes_bytes(B, n, C)}, {Xs, scales_bytes(B, n, C)}};
    Buf outs[] = {{X, bf16_bytes(B * n * C)}};
    DeviceInfo info;
    MHC_TRY(check_buffers(ins, 2, outs, 1, nullptr, nullptr, &info));
    return cuda_status(launch_ckpt_unpack(Xq, Xs, B, n, C, X, cu(stream)));
}

int mhc_post_res_apply_ckpt(const mhc_bf16 *X, const mhc_bf16 *F_out, const float *H_res,
                            const float *H_post, int64_t B, int n, int64_t C, mhc_bf16 *X_next,
                            uint8_t *Xq, uint8_t *Xs, mhc_stream_t stream)
{
    return post_res_ckpt_checked(X, F_out, H_res, H_post, B, n, C, X_next, Xq, Xs, stream);
}

int mhc_post_res_apply_ckpt_f32(const mhc_bf16 *X, const float *F_out, const float *H_res,
                                const float *H_post, int64_t B, int n, int64_t C,
                                mhc_bf16 *X_next, uint8_t *Xq, uint8_t *Xs, mhc_stream_t stream)
{
    return post_res_ckpt_checked(X, F_out, H_res, H_post, B, n, C, X_next, Xq, Xs, stream);
}

int mhc_post_res_apply_backward(const mhc_bf16 *dX_next, const uint8_t *Xq, const uint8_t *Xs,
                                const mhc_bf16 *F_out, const float *H_post, int64_t B, int n,
                                int64_t C, mhc_bf16 *dF_out, float *dH_res, float *dH_post,
                                mhc_stream_t stream)
{
    return post_backward_checked(dX_next, Xq, Xs, F_out, H_post, B, n, C, dF_out, dH_res, dH_post,
                                 stream);
}

int mhc_post_res_apply_backward_f32(const mhc_bf16 *dX_next, const uint8_t *Xq, const uint8_t *Xs,
                                    const float *F_out, const float *H_post, int64_t B, int n,
                                    int64_t C, float *dF_out, float *dH_res, float *dH_post,
                                    mhc_stream_t stream)
{
    return post_backward_checked(dX_next, Xq, Xs, F_out, H_post, B, n, C, dF_out, dH_res, dH_post,
                                 stream);
}

size_t mhc_pre_backward_workspace_bytes(int64_t B, int n, int64_t C, int iters)
{
    DeviceInfo info;
    if (check_shape(B, n, C, true) != MHC_OK || iters < 0 || iters > kMaxBackwardIters || B == 0)
        return 0;
    if (current_device_info(&info) != cudaSuccess) return 0;
    return pre_backward_workspace_bytes(B, n, C, iters, info.num_sms);
}

#define MHC_PRE_BACKWARD_ARGS                                                                     \
    const mhc_bf16 *dX_next, const mhc_bf16 *dF_pre, const uint8_t *Xq, const uint8_t *Xs,        \
        const mhc_bf16 *phi_t, float alpha_pre, float alpha_post, float alpha_res,                \
        const float *bias, int iters, const float *Y, const float *r, const float *H_pre,         \
        const float *H_post, const float *H_res, const float *dH_res, const float *dH_post,       \
        int accumulate, int64_t B, int n, int64_t C, mhc_bf16 *dX, float *dphi_t, float *dbias,   \
        float *dalpha, void *workspace, size_t workspace_bytes, mhc_stream_t stream
#define MHC_PRE_BACKWARD_PASS                                                                     \
    PreBackwardArgs{dX_next, dF_pre, Xq, Xs, phi_t, alpha_pre, alpha_post, alpha_res, bias,       \
                    iters, Y, r, H_pre, H_post, H_res, dH_res, dH_post, accumulate != 0, B, n, C, \
                    dX, dphi_t, dbias, dalpha},                                                   \
        workspace, workspace_bytes, stream

int mhc_pre_backward(MHC_PRE_BACKWARD_ARGS)
{
    return pre_backward_checked(MHC_PRE_BACKWARD_PASS, Waits{});
}

int mhc_testing_pre_backward_stalled(MHC_PRE_BACKWARD_ARGS, int kernel, int64_t stall_unit,
                                     uint64_t wait_limit_ns)
{
    constexpr uint64_t lo = 1000000;
    Waits w;
    w.limit_ns = wait_limit_ns < lo ? lo : wait_limit_ns > kWaitLimitNs ? kWaitLimitNs : wait_limit_ns;
    (kernel == 0 ? w.stall_dx : w.stall_dphi) = stall_unit;
    return pre_backward_checked(MHC_PRE_BACKWARD_PASS, w);
}

#undef MHC_PRE_BACKWARD_ARGS
#undef MHC_PRE_BACKWARD_PASS

}  // extern "C"
