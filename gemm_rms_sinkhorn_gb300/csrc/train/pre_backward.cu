// Backward of everything before the layer function F: F_pre (§2.5 (1)), the
// coefficients with their Sinkhorn iteration (§2.3, §2.4) and the projection
// with its RMS (§2.1, §2.2), page "mHC 算法分析 & cutile 高效实现", and of the
// residual path of X_next.  G = dX_next, dF = dF_pre, X read as it was kept
// (kept.cuh), K = nC, N = n² + 2n:
//
//   dots    dH_pre[i] = Σ_c dF[c]·X[i][c]
//   coefs   dH̃_pre  = dH_pre·H_pre·(1 − H_pre)
//           dH̃_post = dH_post·H_post·(1 − H_post/2)
//           dH̃_res  = the Sinkhorn iteration's (below)
//           dbias = Σ_b dH̃,  dα_seg = Σ_b Σ_{k in seg} dH̃·Y/r
//           dY = α·dH̃/r,     s = −Σ_k dY·Y/(K·r²)       (r = sqrt(Σx²/K);
//                                                        r = 0: below)
//   streams dX[j] = Σ_i H_res[i][j]·G[i] + H_pre[j]·dF + Σ_k dY[k]·φ[k] + s·X[j]
//           (streams.cu)
//   phi     dφ_t[k] = Σ_b dY[b][k]·X[b]                  (phi_grad.cu)
//
// The sum over all channels in `dots` stands between F's gradient and dX, so
// the codes are read by dots and again by streams.
//
// Sinkhorn.  With A = exp(H̃_res) (rows shifted by their maximum, which changes
// no iterate), the iteration is u_t = 1/(A·v_{t−1}), v_t = 1/(Aᵀ·u_t), v_0 = 1,
// H_res = diag(u_T)·A·diag(v_T).  With R_t = diag(u_t)·A·diag(v_{t−1}), whose rows
// sum to 1, and P_t = diag(u_t)·A·diag(v_t), whose columns do, the gradients α of
// log u and β of log v are undone step by step into E = dH̃_res:
//
//   E = P_T·dH_res,  α_i = Σ_j E,  β_j = Σ_i E
//   for t = T … 1:  E −= P_t·β_j,   α_i −= Σ_j P_t·β_j
//                   E −= R_t·α_i,   β_j = −Σ_i R_t·α_i,   α = 0
//   (T = 0: E = A·dH_res)
//
// All factors are entries of the iterates, at most 1: wherever the forward is finite
// so is this (in terms of u, v and A alone, u·v and the squares of u and v overflow
// where H̃_res spreads by some 80).  The forward is run again, in the form that it has
// for this n, and what it goes through is kept: up to n = 4 the R_t (P_t is R_t over
// its column sums), else u_t and v_t, 2n values a step.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "check.cuh"
#include "kept.cuh"
#include "mix.cuh"
#include "ptx.cuh"
#include "train.h"

namespace mhc {
namespace {

// ------------------------------------------------------------------ dots

// Bound by the codes' bytes.  A lane takes 8 channels of all n streams, so dF is
// widened once for them; a block's scale multiplies its partial sum, not its
// values.  W warps share a token.  As many CTAs an SM as spill next to nothing: B=16384,
// n=4, C=7168 110 us, 6.5 TB/s, with five (48 registers), 147 with two; B=8191, n=8,
// C=4096 68 us with three and coefs beside it (its bytes take 50), 76 with two, 77
// with four, which spill.
constexpr int kDotWarps = 8;

//
// The CTAs past the tokens' lay φ_t [N][K] out for the product dY·φ (train.h).
template <int n, int W>
__global__ void __launch_bounds__(kDotWarps * 32, n <= 4 ? 5 : n == 5 ? 4 : 3)
dots_kernel(const uint16_t *__restrict__ dF, const uint8_t *__restrict__ Xq,
            const uint8_t *__restrict__ Xs, const uint16_t *__restrict__ phi_t, int64_t B,
            int64_t C, unsigned dot_ctas, float *__restrict__ dH_pre,
            uint8_t *__restrict__ phi_img)
{
    if (blockIdx.x >= dot_ctas) {
        constexpr int N = n * n + 2 * n, kCols = dy_cols(n);
        const int64_t K = n * C;
        const int64_t q = static_cast<int64_t>(blockIdx.x - dot_ctas) * (kDotWarps * 32) + threadIdx.x;
        ptx::pdl_wait();
        ptx::pdl_trigger();
        if (q >= K || !in_range(1203, q, 1, K)) return;
        constexpr int W = streams_width(n), RB = phi_image_row(n);
        const int64_t j = q / C, c = q - j * C;
        const int row = static_cast<int>(j) * W + static_cast<int>(c % W);
        uint8_t *img = phi_img + c / W * phi_image_bytes(n);
        uint32_t w[kCols / 2];  // all loads before the first store
#pragma unroll
        for (int k = 0; k < kCols; ++k) {
            const uint32_t v = k < N ? ptx::ld_dep(phi_t + k * K + q) : 0u;
            w[k / 2] = k % 2 == 0 ? v : w[k / 2] | v << 16;
        }
#pragma unroll
        for (int k8 = 0; k8 < kCols / 8; ++k8) {
            uint8_t *dst = k8 * 16 < RB ? img + row * RB + (k8 ^ swizzle_xor(RB, row)) * 16
                                        : img + n * W * RB + row * 32 +
                                              ((k8 - RB / 16) ^ swizzle_xor(32, row)) * 16;
            *reinterpret_cast<uint4 *>(dst) =
                make_uint4(w[k8 * 4], w[k8 * 4 + 1], w[k8 * 4 + 2], w[k8 * 4 + 3]);
        }
        return;
    }
    __shared__ float part[kDotWarps][n];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t nb = kept_blocks(C);
    ptx::pdl_wait();
    ptx::pdl_trigger();
    const int64_t b = static_cast<int64_t>(blockIdx.x) * (kDotWarps / W) + warp / W;
    const bool have = b < B && in_range(1201, b, 1, B);
    const uint16_t *f_row = dF + b * C;
    const uint8_t *q_row = Xq + b * n * C, *s_row = Xs + b * n * nb;
    const int C8 = static_cast<int>(C >> 3);
    uint2 q[n];
    uint4 f;
    uint32_t E[n];
    const auto load = [&](int c8) {
        const bool in = have && c8 < C8 && in_range(1202, c8 * 8, 8, C);
        f = in ? ptx::ld_stream_v4(f_row + c8 * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < n; ++i) {
            q[i] = in ? kept::ld_stream_v2(q_row + i * C + c8 * 8) : make_uint2(0, 0);
            E[i] = in ? ptx::ld_dep(s_row + i * nb + (c8 >> 2)) : kept::kScaleMin;
        }
    };
    float s[n];
#pragma unroll
    for (int i = 0; i < n; ++i) s[i] = 0.f;
    const int c0 = (warp % W) * 32 + lane;
    load(c0);
    for (int c8 = c0; c8 - lane < C8; c8 += W * 32) {
        uint64_t v[4], x[4];
        unpack8_pairs(f, v);
        float d[n], scale[n];
#pragma unroll
        for (int i = 0; i < n; ++i) {
            kept::codes8_pairs(q[i], x);
            uint64_t a = 0;
#pragma unroll
            for (int p = 0; p < 4; ++p) a = f2_fma(x[p], v[p], a);
            float lo, hi;
            f2_unpack(a, lo, hi);
            d[i] = lo + hi;
            scale[i] = kept::scale_value(E[i]);
        }
        load(c8 + W * 32);
#pragma unroll
        for (int i = 0; i < n; ++i) s[i] = fmaf(d[i], scale[i], s[i]);
    }
#pragma unroll
    for (int i = 0; i < n; ++i)
#pragma unroll
        for (int x = 16; x > 0; x /= 2) s[i] += __shfl_xor_sync(0xffffffffu, s[i], x);
    if constexpr (W == 1) {
        if (have && lane == 0)
#pragma unroll
            for (int i = 0; i < n; ++i) dH_pre[b * n + i] = s[i];
    } else {
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < n; ++i) part[warp][i] = s[i];
        __syncthreads();
        if (have && warp % W == 0 && lane < n) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) sum += part[warp + w][lane];
            dH_pre[b * n + lane] = sum;
        }
    }
}

// ----------------------------------------------------------------- coefs

// A thread per token.  What a token needs of Y, r, H and dH comes through shared
// memory, a row of odd length per token (read by a thread each from global memory,
// every request touches 32 lines), and the sums over tokens go back through it: by
// shuffles, five dependent ones per column, they took as long as the iteration.  Up
// to dH_pre nothing here depends on dots, so all that runs beside it.
// (B=8191, n=8, in the backward: 42 us read from global memory, 37 so; 40 with the
// iterates in place of u and v.)
constexpr int kCoefThreads = 64;
constexpr int kSmemMost = 200 * 1024;

// A token's staged row: Y, dH_res, H_res, H_pre, H_post, dH_post.
__host__ __device__ constexpr int coef_row(int n) { return (n * n + 2 * n + 2 * n * n + 3 * n) | 1; }
// dH̃ by column and the α's sums, by token.
__host__ __device__ constexpr int coef_sums(int n) { return (n * n + 2 * n + 3) * (kCoefThreads + 1); }
// What is kept of a step: R_t, or u_t and v_t.
__host__ __device__ constexpr int hist_vals(int n) { return n <= 4 ? n * n : 2 * n; }
inline size_t coef_smem(int n, int iters, bool with_hist)
{
    return sizeof(float) * (static_cast<size_t>(kCoefThreads) * coef_row(n) + coef_sums(n) +
                            (with_hist ? static_cast<size_t>(iters) * hist_vals(n) * kCoefThreads : 0));
}

struct CoefOut {
    float *mix;          // [mix_vals][padded tokens] (train.h)
    uint16_t *dY_rows;   // [kRowTerms][padded tokens][dy_cols] bf16, zeros past N
    uint16_t *dY_terms;  // bf16 terms of dY (train.h)
    float *part;         // [CTAs][N + 3]: Σ dH̃ by column, then by α
    float *hist;         // [CTAs][iters][hist_vals][threads], or NULL: in shared memory
};

template <int n>
__global__ void __launch_bounds__(kCoefThreads)
coefs_kernel(PreBackwardArgs a, const float *__restrict__ dH_pre, int64_t Bp, CoefOut o)
{
    constexpr int N = n * n + 2 * n, kCols = dy_cols(n), kRow = coef_row(n);
    static_assert(int64_t{kMaxBackwardIters} * hist_vals(n) * kCoefThreads < int64_t{1} << 31, "h_at");
    constexpr int kS = kCoefThreads + 1;
    extern __shared__ float smem_f[];
    float *rows = smem_f, *sums = rows + kCoefThreads * kRow;  // sums: [N + 3][kS]
    float *hist = o.hist ? o.hist + static_cast<int64_t>(blockIdx.x) * a.iters * hist_vals(n) * kCoefThreads
                         : sums + coef_sums(n);
    hist += threadIdx.x;
    const auto h_at = [&](int t, int k) -> float & { return hist[(t * hist_vals(n) + k) * kCoefThreads]; };
    float total[(N + 3 + kCoefThreads - 1) / kCoefThreads] = {};  // of columns threadIdx.x, + 64

    // the rows of a token block, element by element in the order of global memory
    const auto stage = [&](int64_t b0) {
        const int live = static_cast<int>(a.B - b0 < kCoefThreads ? a.B - b0 : kCoefThreads);
        const auto take = [&](const float *src, int len, int at) {
            if (live <= 0 || !in_range(1213, b0, live, a.B)) return;
            for (int x = threadIdx.x; x < live * len; x += kCoefThreads)
                ptx::cp_async4(rows + x / len * kRow + at + x % len, src + b0 * len + x);
        };
        take(a.Y, N, 0);
        take(a.dH_res, n * n, N);
        take(a.H_res, n * n, N + n * n);
        take(a.H_pre, n, N + 2 * n * n);
        take(a.H_post, n, N + 2 * n * n + n);
        take(a.dH_post, n, N + 2 * n * n + 2 * n);
        ptx::cp_async_commit();
        ptx::cp_async_wait_all();
        __syncthreads();
    };
    // (inputs: the kernel before this one does not write them, and lets this one start only
    // when what preceded the call had finished, so they may be read ahead of the wait)
    bool waited = false;

    const float inv_K = 1.0f / (static_cast<float>(n) * static_cast<float>(a.C));
    for (int64_t b0 = static_cast<int64_t>(blockIdx.x) * kCoefThreads; b0 < Bp;
         b0 += static_cast<int64_t>(gridDim.x) * kCoefThreads) {
        const int64_t b = b0 + threadIdx.x;
        const bool live = b < a.B && in_range(1211, b, 1, a.B);
        const float r = live ? __ldg(a.r + b) : 0.f, inv_r = inv_norm(r);
        stage(b0);
        const float *y = rows + threadIdx.x * kRow, *row_D = y + N, *row_H = row_D + n * n;
        const float *row_hp = row_H + n * n, *row_hq = row_hp + n, *row_dq = row_hq + n;
        float A[n][n], E[n][n];  // E: dH_res, then dH̃_res
        if (live) {
#pragma unroll
            for (int i = 0; i < n; ++i)
#pragma unroll
                for (int j = 0; j < n; ++j) {
                    const int k = 2 * n + i * n + j;
                    A[i][j] = a.a_res * y[k] * inv_r + __ldg(a.bias + k);
                    E[i][j] = row_D[i * n + j];
                }
            if (a.iters > 0) {
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    float mx = A[i][0];
#pragma unroll
                    for (int j = 1; j < n; ++j) mx = fmaxf(mx, A[i][j]);
#pragma unroll
                    for (int j = 0; j < n; ++j) A[i][j] = expf(A[i][j] - mx);
                }
                // back from the iterate P = u·A·v: α and β are the gradients of log u and log v
                float al[n], be[n];
                const auto row_col_sums = [&] {
#pragma unroll
                    for (int i = 0; i < n; ++i) al[i] = tree_sum<n>(E[i]);
#pragma unroll
                    for (int j = 0; j < n; ++j) {
                        float p[n];
#pragma unroll
                        for (int i = 0; i < n; ++i) p[i] = E[i][j];
                        be[j] = tree_sum<n>(p);
                    }
                };
                if constexpr (n <= 4) {
                    for (int t = 0; t < a.iters; ++t) {
#pragma unroll
                        for (int i = 0; i < n; ++i) {
                            const float inv = recip_approx(tree_sum<n>(A[i]));
#pragma unroll
                            for (int j = 0; j < n; ++j) h_at(t, i * n + j) = A[i][j] *= inv;
                        }
#pragma unroll
                        for (int j = 0; j < n; ++j) {
                            float p[n];
#pragma unroll
                            for (int i = 0; i < n; ++i) p[i] = A[i][j];
                            const float inv = recip_approx(tree_sum<n>(p));
#pragma unroll
                            for (int i = 0; i < n; ++i) A[i][j] *= inv;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < n; ++i)
#pragma unroll
                        for (int j = 0; j < n; ++j) E[i][j] *= A[i][j];
                    row_col_sums();
                    float N_R[n][n], N_inv[n];  // R_t and 1 over its column sums, a step ahead
                    const auto next = [&](int t) {
#pragma unroll
                        for (int i = 0; i < n; ++i)
#pragma unroll
                            for (int j = 0; j < n; ++j) N_R[i][j] = h_at(t, i * n + j);
#pragma unroll
                        for (int j = 0; j < n; ++j) {
                            float p[n];
#pragma unroll
                            for (int i = 0; i < n; ++i) p[i] = N_R[i][j];
                            N_inv[j] = recip_approx(tree_sum<n>(p));
                        }
                    };
                    next(a.iters - 1);
                    for (int t = a.iters - 1; t >= 0; --t) {
                        float R[n][n], g[n];
#pragma unroll
                        for (int j = 0; j < n; ++j) {
                            g[j] = N_inv[j] * be[j];
#pragma unroll
                            for (int i = 0; i < n; ++i) R[i][j] = N_R[i][j];
                        }
                        next(t > 0 ? t - 1 : 0);
#pragma unroll
                        for (int i = 0; i < n; ++i) {
                            float p[n];
#pragma unroll
                            for (int j = 0; j < n; ++j) p[j] = R[i][j] * g[j];
                            al[i] -= tree_sum<n>(p);
#pragma unroll
                            for (int j = 0; j < n; ++j) E[i][j] = fmaf(-R[i][j], g[j] + al[i], E[i][j]);
                        }
#pragma unroll
                        for (int j = 0; j < n; ++j) {
                            float p[n];
#pragma unroll
                            for (int i = 0; i < n; ++i) p[i] = R[i][j] * al[i];
                            be[j] = -tree_sum<n>(p);
                        }
#pragma unroll
                        for (int i = 0; i < n; ++i) al[i] = 0.f;
                    }
                } else {
                    float u[n], v[n];
#pragma unroll
                    for (int j = 0; j < n; ++j) v[j] = 1.0f;
                    for (int t = 0; t < a.iters; ++t) {
#pragma unroll
                        for (int i = 0; i < n; ++i) {
                            float p[n];
#pragma unroll
                            for (int j = 0; j < n; ++j) p[j] = A[i][j] * v[j];
                            h_at(t, i) = u[i] = recip_approx(tree_sum<n>(p));
                        }
#pragma unroll
                        for (int j = 0; j < n; ++j) {
                            float p[n];
#pragma unroll
                            for (int i = 0; i < n; ++i) p[i] = __fmul_rn(u[i], A[i][j]);
                            h_at(t, n + j) = v[j] = recip_approx(tree_sum<n>(p));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < n; ++i)
#pragma unroll
                        for (int j = 0; j < n; ++j) E[i][j] *= (u[i] * A[i][j]) * v[j];
                    row_col_sums();
                    for (int t = a.iters - 1; t >= 0; --t) {
                        // u and v are u_t and v_t; (u·A)·v before the gradient's factor, as u
                        // and v may be large
                        float to_v[n], to_u[n];
#pragma unroll
                        for (int k = 0; k < n; ++k) {
                            to_v[k] = t > 0 ? h_at(t - 1, n + k) : 1.0f;
                            to_u[k] = h_at(t > 0 ? t - 1 : 0, k);
                        }
#pragma unroll
                        for (int i = 0; i < n; ++i)
#pragma unroll
                            for (int j = 0; j < n; ++j) {
                                const float P = (u[i] * A[i][j]) * v[j];
                                E[i][j] = fmaf(-P, be[j], E[i][j]);
                                al[i] = fmaf(-P, be[j], al[i]);
                            }
#pragma unroll
                        for (int j = 0; j < n; ++j) be[j] = 0.f;
#pragma unroll
                        for (int i = 0; i < n; ++i)
#pragma unroll
                            for (int j = 0; j < n; ++j) {
                                const float R = (u[i] * A[i][j]) * to_v[j];
                                E[i][j] = fmaf(-R, al[i], E[i][j]);
                                be[j] = fmaf(-R, al[i], be[j]);
                            }
#pragma unroll
                        for (int k = 0; k < n; ++k) {
                            al[k] = 0.f;
                            v[k] = to_v[k];
                            u[k] = to_u[k];
                        }
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < n; ++i)
#pragma unroll
                    for (int j = 0; j < n; ++j) E[i][j] *= expf(A[i][j]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < n; ++i)
#pragma unroll
                for (int j = 0; j < n; ++j) E[i][j] = 0.f;
        }

        if (!waited) {
            ptx::pdl_wait();  // dH_pre
            ptx::pdl_trigger();
            waited = true;
        }
        float dh[n];
#pragma unroll
        for (int i = 0; i < n; ++i) dh[i] = live ? ptx::ld_dep(dH_pre + b * n + i) : 0.f;
        float *mix = o.mix + b;
        uint4 *row = reinterpret_cast<uint4 *>(o.dY_rows + b * kCols);
        uint4 *row_mid = reinterpret_cast<uint4 *>(o.dY_rows + (Bp + b) * kCols);
        const bool in = b < Bp && in_range(1212, b, 1, Bp);
        if (in) {
#pragma unroll
            for (int i = 0; i < n; ++i)
#pragma unroll
                for (int j = 0; j < n; ++j) mix[(j * n + i) * Bp] = live ? row_H[i * n + j] : 0.f;
        }
        float sx = 0.f, da[3] = {0.f, 0.f, 0.f};
        uint32_t packed[4] = {0, 0, 0, 0}, packed_mid[4] = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < kCols; ++k) {
            uint32_t hi = 0, mid = 0;
            if (k < N) {
                float d = 0.f;  // dH̃ of column k
                if (k < n) {
                    if (live) {
                        const float h = row_hp[k];
                        mix[(n * n + k) * Bp] = h;
                        d = dh[k] * h * (1.0f - h);
                    }
                } else if (k < 2 * n) {
                    if (live) d = row_dq[k - n] * row_hq[k - n] * (1.0f - 0.5f * row_hq[k - n]);
                } else {
                    d = E[(k - 2 * n) / n][(k - 2 * n) % n];
                }
                const float yk = live ? y[k] : 0.f;
                const float alpha = k < n ? a.a_pre : k < 2 * n ? a.a_post : a.a_res;
                da[k < n ? 0 : k < 2 * n ? 1 : 2] += d * (yk * inv_r);
                const float dy = alpha * d * inv_r;
                sx = fmaf(-dy, yk, sx);
                sums[k * kS + threadIdx.x] = d;
                // dY as two bf16 terms for dX, to 2^-16, where the sum that it enters is
                // rounded to bf16 (one term, 2^-8, would show wherever φ's rows cancel),
                // and as three for dφ, which is kept in fp32
                hi = pack_bf16_rn(dy, 0.f) & 0xFFFFu;
                const float rest = dy - bf16_lo(hi);
                mid = pack_bf16_rn(rest, 0.f) & 0xFFFFu;
                const uint32_t low = pack_bf16_rn(rest - bf16_lo(mid), 0.f) & 0xFFFFu;
                if (in) {
                    uint16_t *dst = o.dY_terms + static_cast<int64_t>(phi_term_row(k, 0)) * Bp + b;
                    dst[0] = static_cast<uint16_t>(hi);
                    dst[16 * Bp] = static_cast<uint16_t>(mid);
                    dst[32 * Bp] = static_cast<uint16_t>(low);
                }
            }
            const int w = k % 8 / 2;
            packed[w] = k % 2 == 0 ? hi : packed[w] | (hi << 16);
            packed_mid[w] = k % 2 == 0 ? mid : packed_mid[w] | (mid << 16);
            if (k % 8 == 7 && in) {
                row[k / 8] = make_uint4(packed[0], packed[1], packed[2], packed[3]);
                row_mid[k / 8] = make_uint4(packed_mid[0], packed_mid[1], packed_mid[2], packed_mid[3]);
            }
        }
        sx = sx * inv_r * inv_r * inv_K;
        // A token of zeros (padding): the forward takes Y/r as 0, so φ and the α get nothing
        // from it.  Its coefficients jump at X = 0; where they are asked to move, dX has no
        // value, and nowhere else.
        if (live && r == 0.f) {
            bool moved = false;
            for (int k = 0; k < N; ++k)
                moved |= (k < n ? a.a_pre : k < 2 * n ? a.a_post : a.a_res) * sums[k * kS + threadIdx.x] != 0.f;
            if (moved) sx = __int_as_float(0x7FC00000);
        }
        if (in) mix[(n * n + n) * Bp] = sx;
#pragma unroll
        for (int e = 0; e < 3; ++e) sums[(N + e) * kS + threadIdx.x] = da[e];
        __syncthreads();
        // a thread per column, in the order of the tokens
#pragma unroll
        for (int x = 0; x < (N + 3 + kCoefThreads - 1) / kCoefThreads; ++x) {
            const int k = x * kCoefThreads + threadIdx.x;
            if (k < N + 3) {
                float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
                for (int t = 0; t < kCoefThreads; t += 4)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[e] += sums[k * kS + t + e];
                total[x] += (s[0] + s[1]) + (s[2] + s[3]);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int x = 0; x < (N + 3 + kCoefThreads - 1) / kCoefThreads; ++x) {
        const int k = x * kCoefThreads + threadIdx.x;
        if (k < N + 3) o.part[static_cast<int64_t>(blockIdx.x) * (N + 3) + k] = total[x];
    }
}

// -------------------------------------------------------------- launches

struct Ws {
    float *dH_pre, *mix, *part, *hist;
    uint16_t *dY_rows, *dY_terms;
    uint8_t *phi_img;
    void *phi;
    int64_t ctas;      // of coefs_kernel
    size_t coef_smem;  // its dynamic shared memory
    size_t total;
};

Ws carve(void *base, int64_t B, int n, int64_t C, int iters, int num_sms)
{
    const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const int N = num_coeffs(n);
    const int64_t Bp = phi_grad_padded_tokens(B);
    Ws w{};
    uint8_t *p = static_cast<uint8_t *>(base);
    size_t at = 0;
    const auto take = [&](size_t bytes) { uint8_t *r = p + at; at += up(bytes); return r; };
    const size_t hist = static_cast<size_t>(iters) * hist_vals(n) * kCoefThreads * sizeof(float);
    const bool in_smem = coef_smem(n, iters, true) <= static_cast<size_t>(kSmemMost);
    w.coef_smem = coef_smem(n, iters, in_smem);
    const int64_t most = (in_smem ? 16 : 2) * static_cast<int64_t>(num_sms);
    const int64_t need = (Bp + kCoefThreads - 1) / kCoefThreads;
    w.ctas = need < most ? need : most;
    w.dH_pre = reinterpret_cast<float *>(take(static_cast<size_t>(B) * n * 4));
    w.mix = reinterpret_cast<float *>(take(static_cast<size_t>(Bp) * mix_vals(n) * 4));
    w.part = reinterpret_cast<float *>(take(static_cast<size_t>(w.ctas) * (N + 3) * 4));
    w.dY_rows = reinterpret_cast<uint16_t *>(take(static_cast<size_t>(Bp) * kRowTerms * dy_cols(n) * 2));
    w.phi_img = take(static_cast<size_t>((C + streams_width(n) - 1) / streams_width(n) *
                                         phi_image_bytes(n)));
    w.dY_terms = reinterpret_cast<uint16_t *>(take(static_cast<size_t>(Bp) * phi_term_rows(N) * 2));
    w.hist = nullptr;
    if (!in_smem)
        w.hist = reinterpret_cast<float *>(take(static_cast<size_t>(w.ctas) * hist));
    w.phi = take(phi_grad_workspace_bytes(B, n, C, num_sms));
    w.total = at;
    return w;
}

template <int n>
cudaError_t launch_n(const PreBackwardArgs &a, const Ws &w, int num_sms, cudaStream_t stream,
                     const Waits &waits)
{
    const int64_t Bp = phi_grad_padded_tokens(a.B);
    // a warp a token once there are tokens for some warps on every SM, else a CTA a token
    const bool many = a.B >= 16 * static_cast<int64_t>(num_sms);
    const int64_t dot_ctas = many ? (a.B + kDotWarps - 1) / kDotWarps : a.B;
    const int64_t phi_ctas = (n * a.C + kDotWarps * 32 - 1) / (kDotWarps * 32);
    cudaError_t e = launch_pdl(many ? dots_kernel<n, 1> : dots_kernel<n, kDotWarps>,
                               dim3(static_cast<unsigned>(dot_ctas + phi_ctas)),
                               dim3(kDotWarps * 32), 0, stream, a.dF_pre, a.Xq, a.Xs, a.phi_t, a.B,
                               a.C, static_cast<unsigned>(dot_ctas), w.dH_pre, w.phi_img);
    if (e != cudaSuccess) return e;
    const CoefOut o{w.mix, w.dY_rows, w.dY_terms, w.part, w.hist};
    static std::atomic<uint64_t> configured{0};
    e = once_per_device(configured, [] {
        return cudaFuncSetAttribute(coefs_kernel<n>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kSmemMost);
    });
    if (e != cudaSuccess) return e;
    e = launch_pdl(coefs_kernel<n>, dim3(static_cast<unsigned>(w.ctas)), dim3(kCoefThreads),
                   w.coef_smem, stream, a, w.dH_pre, Bp, o);
    if (e != cudaSuccess) return e;
    e = launch_streams(StreamsArgs{a.dX_next, a.dF_pre, w.phi_img, w.dY_rows, a.Xq, a.Xs, w.mix, a.B,
                                   Bp, a.C, a.dX}, n, num_sms, stream, waits);
    if (e != cudaSuccess) return e;
    const BiasSums bs{w.part, static_cast<int>(w.ctas), a.dbias, a.dalpha};
    return launch_phi_grad(a.Xq, a.Xs, w.dY_terms, a.B, n, a.C, a.accumulate, a.dphi_t, w.phi, bs,
                           num_sms, stream, waits);
}

}  // namespace

size_t pre_backward_workspace_bytes(int64_t B, int n, int64_t C, int iters, int num_sms)
{
    return B > 0 ? carve(nullptr, B, n, C, iters, num_sms).total : 0;
}

cudaError_t launch_pre_backward(const PreBackwardArgs &a, void *workspace, int num_sms,
                                cudaStream_t stream, const Waits &waits)
{
    const Ws w = carve(workspace, a.B, a.n, a.C, a.iters, num_sms);
    switch (a.n) {
#define MHC_CASE(k) \
    case k: return launch_n<k>(a, w, num_sms, stream, waits);
        MHC_CASE(1) MHC_CASE(2) MHC_CASE(3) MHC_CASE(4) MHC_CASE(5) MHC_CASE(6) MHC_CASE(7)
        MHC_CASE(8)
#undef MHC_CASE
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace mhc
