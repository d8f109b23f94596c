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
// One pass over G, the codes and F_out, bound by their bytes.  Two forms; where
// several warps share a token their sums are added in warp order, so that results
// do not depend on timing:
//
//   n <= 4  a lane takes 8 channels of all streams: n² + 2n packed multiply-adds
//           a channel pair, accumulators in registers.  B=4096, n=4, C=4096, F in fp32:
//           57 us, its bytes take 50; a token 4 us.
//   n >= 5  those would be n² register pairs.  Here a warp takes 32 channels of
//           all streams, stream g at lanes 4g .. 4g+3, 8 channels a lane, as the
//           operands of mma.m16n8k16: X's rows and, below them, F_out's against
//           G's columns give dH_res and dH_post, on values that are exact in
//           bf16; the block's scale multiplies the product of its 32 channels.
//           dF_out is a product too, of G transposed in registers with H_post in
//           three bf16 terms (2^-26).  tcgen05's smallest tile is 128 rows and
//           has its operands in shared memory; this work is 8 rows a token.
#include <cuda_runtime.h>

#include <cstdint>

#include "check.cuh"
#include "kept.cuh"
#include "mix.cuh"
#include "mma.cuh"
#include "ptx.cuh"
#include "train.h"

namespace mhc {
namespace {

constexpr int kWarps = 8;
constexpr int kDepth = 2;  // channel groups that a warp of the n >= 5 form has in flight

// Eight values of F_out or dF_out, in bf16 or fp32.
struct Raw8 {
    uint4 a, b;  // b: fp32's second half
};
__device__ __forceinline__ void load_raw(Raw8 &r, const uint16_t *p) { r.a = ptx::ld_stream_v4(p); }
__device__ __forceinline__ void load_raw(Raw8 &r, const float *p)
{
    r.a = ptx::ld_stream_v4(p);
    r.b = ptx::ld_stream_v4(p + 4);
}
__device__ __forceinline__ void raw_pairs(const Raw8 &r, const uint16_t *, uint64_t (&f)[4])
{
    unpack8_pairs(r.a, f);
}
__device__ __forceinline__ void raw_pairs(const Raw8 &r, const float *, uint64_t (&f)[4])
{
    f[0] = (static_cast<uint64_t>(r.a.y) << 32) | r.a.x;
    f[1] = (static_cast<uint64_t>(r.a.w) << 32) | r.a.z;
    f[2] = (static_cast<uint64_t>(r.b.y) << 32) | r.b.x;
    f[3] = (static_cast<uint64_t>(r.b.w) << 32) | r.b.z;
}
__device__ __forceinline__ void store8(uint16_t *p, const uint64_t (&v)[4])
{
    ptx::st_stream_v4(p, pack8_pairs(v));
}
__device__ __forceinline__ void store8(float *p, const uint64_t (&v)[4])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint64_t x = v[2 * h], y = v[2 * h + 1];
        ptx::st_stream_v4(p + 4 * h, make_uint4(static_cast<uint32_t>(x), static_cast<uint32_t>(x >> 32),
                                                static_cast<uint32_t>(y), static_cast<uint32_t>(y >> 32)));
    }
}

template <int n, typename FT, int W>
__global__ void __launch_bounds__(kWarps * 32)
post_backward_kernel(const uint16_t *__restrict__ dX_next, const uint8_t *__restrict__ Xq,
                     const uint8_t *__restrict__ Xs, const FT *__restrict__ F_out,
                     const float *__restrict__ H_post, int64_t B, int64_t C,
                     FT *__restrict__ dF_out, float *__restrict__ dH_res,
                     float *__restrict__ dH_post)
{
    constexpr int kSums = n * n + n;  // dH_res row-major, then dH_post
    __shared__ float part[kWarps][kSums];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t nb = kept_blocks(C);
    const int C8 = static_cast<int>(C >> 3);
    ptx::pdl_wait();
    ptx::pdl_trigger();
    const int64_t b = static_cast<int64_t>(blockIdx.x) * (kWarps / W) + warp / W;
    const bool have = b < B && in_range(1101, b, 1, B);
    const uint16_t *g_row = dX_next + b * n * C;
    const uint8_t *q_row = Xq + b * n * C, *s_row = Xs + b * n * nb;
    const FT *f_row = F_out + b * C;
    float h[n];
#pragma unroll
    for (int i = 0; i < n; ++i) h[i] = have ? ptx::ld_dep(H_post + b * n + i) : 0.f;

    uint64_t acc[n][n], post[n];
#pragma unroll
    for (int i = 0; i < n; ++i) {
        post[i] = 0;
#pragma unroll
        for (int j = 0; j < n; ++j) acc[i][j] = 0;
    }
    const int c0 = (warp % W) * 32 + lane;
    for (int c8 = c0; have && c8 < C8; c8 += W * 32) {
        if (!in_range(1102, c8 * 8, 8, C)) break;
        uint4 gv[n];
        uint2 q[n];
        uint32_t E[n];
        Raw8 fr;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            gv[i] = ptx::ld_stream_v4(g_row + i * C + c8 * 8);
            q[i] = kept::ld_stream_v2(q_row + i * C + c8 * 8);
            E[i] = ptx::ld_dep(s_row + i * nb + (c8 >> 2));
        }
        load_raw(fr, f_row + c8 * 8);
        uint64_t g[n][4], f[4], df[4];
#pragma unroll
        for (int i = 0; i < n; ++i) unpack8_pairs(gv[i], g[i]);
        raw_pairs(fr, f_row, f);
#pragma unroll
        for (int p = 0; p < 4; ++p) df[p] = 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const uint64_t hh = f2_pack(h[i], h[i]);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                df[p] = f2_fma(hh, g[i][p], df[p]);
                post[i] = f2_fma(g[i][p], f[p], post[i]);
            }
        }
        store8(dF_out + b * C + c8 * 8, df);
#pragma unroll
        for (int j = 0; j < n; ++j) {
            float x[8];
            kept::decode8(q[j], kept::scale_value(E[j]), x);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint64_t xp = f2_pack(x[2 * p], x[2 * p + 1]);
#pragma unroll
                for (int i = 0; i < n; ++i) acc[i][j] = f2_fma(g[i][p], xp, acc[i][j]);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
        float lo, hi;
        f2_unpack(k < n * n ? acc[k / n][k % n] : post[k - n * n], lo, hi);
        float s = lo + hi;
#pragma unroll
        for (int x = 16; x > 0; x /= 2) s += __shfl_xor_sync(0xffffffffu, s, x);
        if (lane == 0) part[warp][k] = s;
    }
    if constexpr (W == 1) __syncwarp(); else __syncthreads();
    if (!have || warp % W != 0) return;
    for (int k = lane; k < kSums; k += 32) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) s += part[warp + w][k];
        if (k < n * n) dH_res[b * n * n + k] = s; else dH_post[b * n + (k - n * n)] = s;
    }
}

// bf16 terms hi, mid, low of an fp32 value, as the low halves of words.
__device__ __forceinline__ void split3(float v, uint32_t &hi, uint32_t &mid, uint32_t &low)
{
    hi = pack_bf16_rn(v, 0.f);
    const float r = v - bf16_lo(hi);
    mid = pack_bf16_rn(r, 0.f);
    low = pack_bf16_rn(r - bf16_lo(mid), 0.f);
}

// At B=8192, n=8, C=4096 180 us, 5.3 TB/s; its bytes take 140.  Three CTAs an SM (80
// registers) and two neighbouring channel groups read together (two CTAs with four
// groups 197, four with one 216; with a warp's groups apart 24 more).  G as the left
// operand of dF_out's product takes two products a group; as the right operand, of
// which H_post fills one row in 16, eight: 189.  What bounds it is the latency of its
// loads at 24 warps an SM: a third fewer L1 wavefronts for the scales gained nothing.
// With F_out in fp32 215 us, its bytes take 160: every stream's lanes load F_out again.
template <int n, typename FT>
__global__ void __launch_bounds__(kWarps * 32, 3)
post_backward_wide_kernel(const uint16_t *__restrict__ dX_next, const uint8_t *__restrict__ Xq,
                          const uint8_t *__restrict__ Xs, const FT *__restrict__ F_out,
                          const float *__restrict__ H_post, int64_t B, int64_t C,
                          FT *__restrict__ dF_out, float *__restrict__ dH_res,
                          float *__restrict__ dH_post)
{
    constexpr bool kF32 = sizeof(FT) == 4;
    __shared__ float part[kWarps][4][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;  // stream; 8 channels of a group of 32
    const int64_t nb = kept_blocks(C);
    const int groups = static_cast<int>(nb);
    ptx::pdl_wait();
    ptx::pdl_trigger();
    const int64_t b = blockIdx.x;
    const bool have_tok = b < B && in_range(1111, b, 1, B);
    const bool have = have_tok && g < n;
    const uint16_t *g_row = dX_next + (b * n + g) * C + t * 8;
    const uint8_t *q_row = Xq + (b * n + g) * C + t * 8, *s_row = Xs + (b * n + g) * nb;
    const FT *f_row = F_out + b * C + t * 8;
    FT *df_row = dF_out + b * C;

    const float hp0 = have_tok && 2 * t < n ? ptx::ld_dep(H_post + b * n + 2 * t) : 0.f;
    const float hp1 = have_tok && 2 * t + 1 < n ? ptx::ld_dep(H_post + b * n + 2 * t + 1) : 0.f;
    const int c_out = g / 2 * 8 + t * 2 + g % 2;  // the channel of a group that the lane writes

    // kDepth groups are in flight: a slot is loaded again as soon as it is used
    struct Slot {
        uint4 g;
        uint2 q;
        uint32_t E;
        Raw8 f;
    } slots[kDepth];
#pragma unroll
    for (int x = 0; x < kDepth; ++x) {
        slots[x].g = slots[x].f.a = slots[x].f.b = make_uint4(0, 0, 0, 0);
        slots[x].q = make_uint2(0, 0);
        slots[x].E = kept::kScaleMin;
    }
    const int whole = static_cast<int>(C >> 5);  // groups with all their channels
    const bool have_f = kF32 ? have : have_tok && g == 0;  // bf16: F_out is row 8 of the left operand
    const auto load = [&](Slot &x, int cg) {
        if (cg < whole && in_range(1112, cg * 32 + t * 8, 8, C)) {
            // (a lane without a stream keeps its zeros)
            if (have) {
                x.g = ptx::ld_stream_v4(g_row + cg * 32);
                x.q = kept::ld_stream_v2(q_row + cg * 32);
                x.E = ptx::ld_dep(s_row + cg);
            }
            if (have_f) load_raw(x.f, f_row + cg * 32);
        } else if (cg < groups) {
            const bool in = cg * 32 + t * 8 < C;
            x.g = in && have ? ptx::ld_stream_v4(g_row + cg * 32) : make_uint4(0, 0, 0, 0);
            x.q = in && have ? kept::ld_stream_v2(q_row + cg * 32) : make_uint2(0, 0);
            // every lane scales its row's sums, also where its own channels are past C
            x.E = have ? ptx::ld_dep(s_row + cg) : kept::kScaleMin;
            x.f.a = x.f.b = make_uint4(0, 0, 0, 0);
            if (in && have_f) load_raw(x.f, f_row + cg * 32);
        }
    };
    if (have_tok)
#pragma unroll
        for (int x = 0; x < kDepth; ++x) load(slots[x], warp * kDepth + x);
    // H_post as a product's right operand: the even columns hi at k = 0 .. 7 and mid at
    // 8 .. 15, the odd ones low, so that a lane's two columns add up to dF_out
    uint32_t a[3], e[3];
    split3(hp0, a[0], a[1], a[2]);
    split3(hp1, e[0], e[1], e[2]);
    const uint32_t h0 = g % 2 == 0 ? __byte_perm(a[0], e[0], 0x5410) : __byte_perm(a[2], e[2], 0x5410);
    const uint32_t h1 = g % 2 == 0 ? __byte_perm(a[1], e[1], 0x5410) : 0;
    float acc[2] = {0.f, 0.f}, post[2] = {0.f, 0.f};
    const auto use = [&](Slot &s, int cg) {
        const uint4 x = kept::codes8_bf16(s.q);
        const float scale = kept::scale_value(s.E);
        const uint4 gw = s.g;
        const Raw8 fr = s.f;
        load(s, cg + kDepth * kWarps);
        float d[4];
        if constexpr (kF32) {
            mma_16816_new(d, x.x, 0u, x.y, 0u, gw.x, gw.y);
            mma_16816(d, x.z, 0u, x.w, 0u, gw.z, gw.w);
            uint64_t v[4], f[4], a = 0;
            unpack8_pairs(gw, v);
            raw_pairs(fr, f_row, f);
#pragma unroll
            for (int p = 0; p < 4; ++p) a = f2_fma(v[p], f[p], a);
            float lo, hi;
            f2_unpack(a, lo, hi);
            post[0] += lo + hi;
        } else {
            mma_16816_new(d, x.x, fr.a.x, x.y, fr.a.y, gw.x, gw.y);
            mma_16816(d, x.z, fr.a.z, x.w, fr.a.w, gw.z, gw.w);
            post[0] += d[2];
            post[1] += d[3];
        }
        acc[0] = fmaf(d[0], scale, acc[0]);
        acc[1] = fmaf(d[1], scale, acc[1]);
        // dF_out: G transposed is the left operand, its row r of word w the channel
        // 8·(r/2) + 2w + r%2, against which every column pair holds H_post
        uint32_t m[4];
        const uint32_t word[4] = {gw.x, gw.y, gw.z, gw.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) m[w] = transpose_8x8(word[w]);
        float o[2][4];
        mma_16816_new(o[0], m[0], m[1], m[0], m[1], h0, h1);
        mma_16816_new(o[1], m[2], m[3], m[2], m[3], h0, h1);
        const float lo = t < 2 ? o[0][0] + o[0][1] : o[1][0] + o[1][1];
        const float hi = t < 2 ? o[0][2] + o[0][3] : o[1][2] + o[1][3];
        const float v = t % 2 == 0 ? lo : hi;  // word t
        const int c = cg * 32 + c_out;
        if constexpr (kF32) {
            if (c < C) __stcs(df_row + c, v);
        } else {
            const float next = __shfl_xor_sync(0xffffffffu, v, 4);
            if (g % 2 == 0 && c < C)
                __stcs(reinterpret_cast<uint32_t *>(df_row + c), pack_bf16_rn(v, next));
        }
    };
    if (have_tok) {
        for (int cg = warp * kDepth; cg < groups; cg += kDepth * kWarps)
#pragma unroll
            for (int x = 0; x < kDepth; ++x)
                if (cg + x < groups) use(slots[x], cg + x);
    }
    if constexpr (kF32) {
        post[0] += __shfl_xor_sync(0xffffffffu, post[0], 1);
        post[0] += __shfl_xor_sync(0xffffffffu, post[0], 2);
    }
    part[warp][0][lane] = acc[0];
    part[warp][1][lane] = acc[1];
    part[warp][2][lane] = post[0];
    part[warp][3][lane] = post[1];
    __syncthreads();
    if (!have_tok || warp != 0) return;
    float s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        s[k] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s[k] += part[w][k][lane];
    }
    // product rows: X's stream g (dH_res) and F_out (dH_post); columns: G's stream 2t + e
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = 2 * t + e;
        if (i < n && g < n) dH_res[(b * n + i) * n + g] = s[e];
        if (!kF32 && i < n && g == 0) dH_post[b * n + i] = s[2 + e];
    }
    if (kF32 && t == 0 && g < n) dH_post[b * n + g] = s[2];
}

}  // namespace

template <typename FT>
cudaError_t launch_post_backward(const uint16_t *dX_next, const uint8_t *Xq, const uint8_t *Xs,
                                 const FT *F_out, const float *H_post, int64_t B, int n, int64_t C,
                                 FT *dF_out, float *dH_res, float *dH_post, int num_sms,
                                 cudaStream_t stream)
{
    // n <= 4: a warp a token once there are tokens for some warps on every SM, else a
    // CTA a token.  n >= 5: always a CTA a token, whose warps read neighbouring 64-byte
    // pieces of a row together (a warp a token: 267 us at B=8192, n=8, C=4096).
    const bool many = n <= 4 && B >= 16 * static_cast<int64_t>(num_sms);
    const dim3 grid(static_cast<unsigned>(many ? (B + kWarps - 1) / kWarps : B));
    switch (n) {
#define MHC_CASE(k, few, all)                                                                    \
    case k:                                                                                      \
        return launch_pdl(many ? all : few, grid, dim3(kWarps * 32), 0, stream, dX_next, Xq, Xs, \
                          F_out, H_post, B, C, dF_out, dH_res, dH_post);
        MHC_CASE(1, (post_backward_kernel<1, FT, kWarps>), (post_backward_kernel<1, FT, 1>))
        MHC_CASE(2, (post_backward_kernel<2, FT, kWarps>), (post_backward_kernel<2, FT, 1>))
        MHC_CASE(3, (post_backward_kernel<3, FT, kWarps>), (post_backward_kernel<3, FT, 1>))
        MHC_CASE(4, (post_backward_kernel<4, FT, kWarps>), (post_backward_kernel<4, FT, 1>))
        MHC_CASE(5, (post_backward_wide_kernel<5, FT>), (post_backward_wide_kernel<5, FT>))
        MHC_CASE(6, (post_backward_wide_kernel<6, FT>), (post_backward_wide_kernel<6, FT>))
        MHC_CASE(7, (post_backward_wide_kernel<7, FT>), (post_backward_wide_kernel<7, FT>))
        MHC_CASE(8, (post_backward_wide_kernel<8, FT>), (post_backward_wide_kernel<8, FT>))
#undef MHC_CASE
    default: return cudaErrorInvalidValue;
    }
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
