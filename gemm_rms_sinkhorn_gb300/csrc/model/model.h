// Launchers of the operators at the entry of the layer function F and at the
// model's end: norms (rmsnorm.cu) and distillation (distill.cu).  Arguments have
// already been validated by model_api.cu when these run.
//
// Sites of the device index checks (check.cuh) here: 1500s rmsnorm.cu, 1600s
// distill.cu.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "mhc_internal.h"
#include "train/train.h"

namespace mhc {

// ---- norms (rmsnorm.cu)
// A token's channels stay in the registers of one block from the sum of squares to the
// scaling: 512 threads of 4 chunks of 8.
constexpr int64_t kNormMaxC = 16384;

struct NormArgs {
    const uint16_t *X;       // the streams [B][n][C]; a residual's sum: A [B][C]
    const uint16_t *R;       // a residual's sum: [B][C], or NULL
    const float *H_pre;      // the streams' weights [B][n]
    const float *gain;
    float eps;
    int64_t B;
    int n;                   // streams; 0: a residual's sum
    int64_t C;
    uint16_t *H;             // the mixed streams or the sum, NULL where it is not wanted
    float *rstd;             // likewise
    uint16_t *Z;             // bf16 out, or NULL and
    uint8_t *Zq, *Zs;        // the 8-bit form (kept.cuh)
};
cudaError_t launch_rmsnorm(const NormArgs &a, int num_sms, cudaStream_t stream);

struct NormBackwardArgs {
    const uint16_t *dZ, *H;
    const float *gain, *rstd;
    const uint16_t *dH_skip;  // or NULL
    int accumulate;
    int64_t B, C;
    uint16_t *dH;
    float *dgain;
};
size_t rmsnorm_backward_workspace_bytes(int64_t B, int64_t C, int num_sms);
cudaError_t launch_rmsnorm_backward(const NormBackwardArgs &a, void *workspace, int num_sms,
                                    cudaStream_t stream);

// ---- distillation (distill.cu)
constexpr int64_t kDistillMaxV = 1 << 18;
constexpr int kDistillMaxK = 1024;

template <typename T>  // the logits' element: uint16_t (bf16) or float
struct DistillArgs {
    const T *z;
    int64_t ld;
    const int64_t *ids;
    const float *t, *t_lse;  // t_lse: or NULL
    float inv_tau;
    const float *dloss;      // NULL: no gradient
    int64_t B;
    int V, K;
    float *loss;             // or NULL
    T *dz;
};
template <typename T>
cudaError_t launch_distill(const DistillArgs<T> &a, int num_sms, cudaStream_t stream);

}  // namespace mhc
