// C ABI of the operators at the entry of F and at the model's end (declared in
// include/mhc.h): argument validation on the host, then their kernels on the caller's
// stream.  No exception crosses this boundary and nothing here allocates device memory.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "host/args.h"
#include "mhc.h"
#include "model.h"

using namespace mhc;

namespace {

// Buffers of a call, without those that are NULL where that is allowed.
struct Bufs {
    Buf b[8];
    int count = 0;
    void add(const void *p, size_t bytes) { b[count++] = {p, bytes}; }
    void add_if(const void *p, size_t bytes)
    {
        if (p != nullptr) add(p, bytes);
    }
};

int check_norm_shape(int64_t B, int n, int64_t C)
{
    MHC_TRY(check_shape(B, n, C, true));
    return C > kNormMaxC ? MHC_ERR_UNSUPPORTED : MHC_OK;
}

bool bad_eps(float eps) { return !std::isfinite(eps) || eps < 0.f; }

// The rules of the four forward norms.  q8: whether Z is (Zq, Zs).
int norm_checked(const NormArgs &a, bool q8, mhc_stream_t stream)
{
    const int64_t B = a.B, C = a.C;
    MHC_TRY(check_norm_shape(B, a.n == 0 ? 1 : a.n, C));
    if (bad_eps(a.eps)) return MHC_ERR_INVALID;
    // without a residual the sum is A itself
    if (a.n == 0 && a.R == nullptr && a.H != nullptr) return MHC_ERR_INVALID;
    if (B == 0) return MHC_OK;
    Bufs ins, outs;
    ins.add(a.X, bf16_bytes(B * (a.n == 0 ? 1 : a.n) * C));
    if (a.n == 0)
        ins.add_if(a.R, bf16_bytes(B * C));
    else
        ins.add(a.H_pre, f32_bytes(B * a.n));
    ins.add(a.gain, f32_bytes(C));
    outs.add_if(a.H, bf16_bytes(B * C));
    outs.add_if(a.rstd, f32_bytes(B));
    if (q8) {
        outs.add(a.Zq, static_cast<size_t>(B * C));
        outs.add(a.Zs, static_cast<size_t>(B * kept_blocks(C)));
    } else {
        outs.add(a.Z, bf16_bytes(B * C));
    }
    // the sum may be exactly one of its terms
    const void *alias = a.n != 0 ? nullptr : a.H == a.R ? a.R : a.X;
    DeviceInfo info;
    MHC_TRY(check_buffers(ins.b, ins.count, outs.b, outs.count, a.n != 0 ? nullptr : a.H, alias, &info));
    return cuda_status(launch_rmsnorm(a, info.num_sms, cu(stream)));
}

template <typename T>
int distill_checked(const DistillArgs<T> &a, int64_t V, bool grad, mhc_stream_t stream)
{
    const int64_t B = a.B, ld = a.ld;
    if (B < 0 || V < 1 || a.K < 1 || ld < V) return MHC_ERR_INVALID;
    // up to 2^64, so that differences of logits times it are numbers
    if (!(a.inv_tau > 0.f) || !(a.inv_tau <= 0x1p64f)) return MHC_ERR_INVALID;
    if (B >= (int64_t{1} << 31) || V > kDistillMaxV || a.K > kDistillMaxK) return MHC_ERR_UNSUPPORTED;
    if (ld % 8 != 0 || ld > (int64_t{1} << 24)) return MHC_ERR_UNSUPPORTED;
    if (B == 0) return MHC_OK;
    const size_t rows = static_cast<size_t>(B) * static_cast<size_t>(ld) * sizeof(T);
    Bufs ins, outs;
    ins.add(a.z, rows);
    ins.add(a.ids, static_cast<size_t>(B) * a.K * 8);
    ins.add(a.t, f32_bytes(B * a.K));
    ins.add_if(a.t_lse, f32_bytes(B));
    if (grad) {
        ins.add(a.dloss, f32_bytes(B));
        outs.add_if(a.loss, f32_bytes(B));
        outs.add(a.dz, rows);
    } else {
        outs.add(a.loss, f32_bytes(B));
    }
    DeviceInfo info;
    MHC_TRY(check_buffers(ins.b, ins.count, outs.b, outs.count, a.dz, grad ? a.z : nullptr, &info));
    DistillArgs<T> d = a;
    d.V = static_cast<int>(V);
    return cuda_status(launch_distill(d, info.num_sms, cu(stream)));
}

}  // namespace

extern "C" {

int mhc_pre_apply_rmsnorm(const mhc_bf16 *X, const float *H_pre, const float *gain, float eps,
                          int64_t B, int n, int64_t C, mhc_bf16 *F_pre, float *rstd, mhc_bf16 *Z,
                          mhc_stream_t stream)
{
    if (n < 1) return MHC_ERR_UNSUPPORTED;
    return norm_checked({X, nullptr, H_pre, gain, eps, B, n, C, F_pre, rstd, Z, nullptr, nullptr},
                        false, stream);
}

int mhc_pre_apply_rmsnorm_q8(const mhc_bf16 *X, const float *H_pre, const float *gain, float eps,
                             int64_t B, int n, int64_t C, mhc_bf16 *F_pre, float *rstd, uint8_t *Zq,
                             uint8_t *Zs, mhc_stream_t stream)
{
    if (n < 1) return MHC_ERR_UNSUPPORTED;
    return norm_checked({X, nullptr, H_pre, gain, eps, B, n, C, F_pre, rstd, nullptr, Zq, Zs}, true,
                        stream);
}

int mhc_add_rmsnorm(const mhc_bf16 *A, const mhc_bf16 *R, const float *gain, float eps, int64_t B,
                    int64_t C, mhc_bf16 *H, float *rstd, mhc_bf16 *Z, mhc_stream_t stream)
{
    return norm_checked({A, R, nullptr, gain, eps, B, 0, C, H, rstd, Z, nullptr, nullptr}, false,
                        stream);
}

int mhc_add_rmsnorm_q8(const mhc_bf16 *A, const mhc_bf16 *R, const float *gain, float eps, int64_t B,
                       int64_t C, mhc_bf16 *H, float *rstd, uint8_t *Zq, uint8_t *Zs,
                       mhc_stream_t stream)
{
    return norm_checked({A, R, nullptr, gain, eps, B, 0, C, H, rstd, nullptr, Zq, Zs}, true, stream);
}

size_t mhc_rmsnorm_backward_workspace_bytes(int64_t B, int64_t C)
{
    DeviceInfo info;
    if (check_norm_shape(B, 1, C) != MHC_OK || B == 0) return 0;
    if (current_device_info(&info) != cudaSuccess) return 0;
    return rmsnorm_backward_workspace_bytes(B, C, info.num_sms);
}

int mhc_rmsnorm_backward(const mhc_bf16 *dZ, const mhc_bf16 *H, const float *gain, const float *rstd,
                         const mhc_bf16 *dH_skip, int accumulate, int64_t B, int64_t C, mhc_bf16 *dH,
                         float *dgain, void *workspace, size_t workspace_bytes, mhc_stream_t stream)
{
    MHC_TRY(check_norm_shape(B, 1, C));
    Buf outs[] = {{dgain, f32_bytes(C)}, {dH, bf16_bytes(B * C)}};
    if (B == 0) return zero_grads(outs, 1, accumulate, stream);
    Bufs ins;
    ins.add(dZ, bf16_bytes(B * C));
    ins.add(H, bf16_bytes(B * C));
    ins.add(gain, f32_bytes(C));
    ins.add(rstd, f32_bytes(B));
    ins.add_if(dH_skip, bf16_bytes(B * C));
    Buf ws = {workspace, workspace_bytes};
    DeviceInfo info;
    MHC_TRY(check_buffers(
        ins.b, ins.count, outs, 2, dH, dH == dZ ? dZ : dH_skip, &ws,
        [&](int sms) { return rmsnorm_backward_workspace_bytes(B, C, sms); }, &info));
    return cuda_status(launch_rmsnorm_backward(
        {dZ, H, gain, rstd, dH_skip, accumulate != 0, B, C, dH, dgain}, workspace, info.num_sms,
        cu(stream)));
}

int mhc_distill_loss(const mhc_bf16 *z, int64_t ld, const int64_t *ids, const float *t,
                     const float *t_lse, float inv_tau, int64_t B, int64_t V, int K, float *loss,
                     mhc_stream_t stream)
{
    return distill_checked<uint16_t>({z, ld, ids, t, t_lse, inv_tau, nullptr, B, 0, K, loss, nullptr},
                                     V, false, stream);
}

int mhc_distill_loss_f32(const float *z, int64_t ld, const int64_t *ids, const float *t,
                         const float *t_lse, float inv_tau, int64_t B, int64_t V, int K, float *loss,
                         mhc_stream_t stream)
{
    return distill_checked<float>({z, ld, ids, t, t_lse, inv_tau, nullptr, B, 0, K, loss, nullptr}, V,
                                  false, stream);
}

int mhc_distill_loss_backward(const mhc_bf16 *z, int64_t ld, const int64_t *ids, const float *t,
                              const float *t_lse, float inv_tau, const float *dloss, int64_t B,
                              int64_t V, int K, float *loss, mhc_bf16 *dz, mhc_stream_t stream)
{
    return distill_checked<uint16_t>({z, ld, ids, t, t_lse, inv_tau, dloss, B, 0, K, loss, dz}, V, true,
                                     stream);
}

int mhc_distill_loss_backward_f32(const float *z, int64_t ld, const int64_t *ids, const float *t,
                                  const float *t_lse, float inv_tau, const float *dloss, int64_t B,
                                  int64_t V, int K, float *loss, float *dz, mhc_stream_t stream)
{
    return distill_checked<float>({z, ld, ids, t, t_lse, inv_tau, dloss, B, 0, K, loss, dz}, V, true,
                                  stream);
}

}  // extern "C"
