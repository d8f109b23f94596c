// dφ_t[k][q] = Σ_b dY[b][k]·X[b][q] on the tensor cores, X read as it was kept
// (kept.cuh) and dY given as three bf16 terms (train.h): the products of bf16
// values are exact, so with fp32 accumulation dφ has fp32's accuracy, which
// one bf16 rounding of dY (2^-9) would not have.
//
// A tall, skinny product: K = nC rows (the channels), 3N columns, summed over
// the tokens.  A CTA takes strips of 256 channels and blocks
// of 64 tokens, the (strip, block) units dealt out in equal contiguous ranges,
// one CTA per SM:
//
//   warp 18     TMA: the codes (64 rows of 256 bytes) into a ring of their own, up
//               to four units ahead;
//   warps 0-15  read them there, write the bf16 values to a stage's A tile and hand
//               it over.  (Codes loaded to registers ahead of use, in place of the
//               ring: 180 us at B=16384, n=4, C=7168 against 158.)  The scales are
//               loaded between hand-overs;
//   warp 16     TMA: the dY terms of the block (B tile);
//   warp 17     tcgen05.mma, M = 128 channels (two accumulators), N = 3n² + 6n
//               columns padded to 48, K = 16 tokens.
//
// Every kFlush units the sixteen warps read the accumulators (tcgen05.ld) and
// add them to the workspace's fp32 sums, each value always by the same thread,
// so in a fixed order.  The accumulator drops what is below its last bit at each
// step (a bias towards zero: over 16384 tokens in one chain dφ was 9.1e-6 off,
// in chains of kFlush · 64 tokens 7e-7); these additions round.
//
// Channels are contiguous in the codes, so A is written MN-major: a unit's tile
// is [4 × 64 channels][8 × 8 tokens], each 64 × 8 part 1 KB with the 128-byte
// swizzle.  A second launch adds the strips' parts in the order of the tokens.
//
// Time: B=16384, n=4, C=7168 158 us for 470 MB of codes (70 us at the copy rate);
// B=8191, n=8, C=4096 112 us.  Bound by shared-memory traffic, some 132 KB a unit
// (codes in and out, the A tile in, the tensor cores' reads of A and B), whose parts
// add up: without decoding 121 us, with a quarter of the products 144, with neither
// 86-91.  Decoding once for two accumulators' columns (157), a deeper B ring (167)
// and A written K-major (188) gained nothing.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "check.cuh"
#include "kept.cuh"
#include "mhc_internal.h"
#include "ptx.cuh"
#include "train.h"

namespace mhc {
namespace {

constexpr int kStrip = 256;
constexpr int kTok = kPhiTokens;
constexpr int kLoadWarps = 16;
constexpr int kRowsEach = kTok / kLoadWarps;  // tokens of a unit that a load warp takes
constexpr int kFlush = 16;                    // units in one accumulation chain
constexpr int kThreads = (kLoadWarps + 3) * 32;
constexpr int kRawBytes = kStrip * kTok;  // a unit's codes
constexpr int kABytes = kStrip * kTok * 2;  // 32 KB
constexpr int kStatusTimeout = -5;          // MHC_ERR_TIMEOUT

__device__ int g_phi_status;

template <int n>
struct Cfg {
    static constexpr int N = n * n + 2 * n;
    static constexpr int NT = phi_term_rows(N);  // columns
    static constexpr int kBBytes = NT * kTok * 2;
    static constexpr int kStage = kABytes + kBBytes;
    static constexpr int kStages = n <= 7 ? 3 : 2;
    static constexpr int kRaw = n == 7 ? 3 : 4;  // units of codes in flight
    static constexpr int kSmem = 1024 + kStages * kStage + kRaw * kRawBytes + 256;
    static constexpr int kTmemCols = 2 * NT <= 128 ? 128 : 2 * NT <= 256 ? 256 : 512;
    static_assert(NT <= 256 && NT % 16 == 0, "MMA N for M = 128");
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

// The units (strip, token block), strip-major, in `grid` equal ranges.
struct Units {
    int64_t total, blocks;  // units; token blocks of a strip
    int grid;
    __host__ __device__ int64_t lo(int c) const { return total * c / grid; }
    __host__ __device__ int owner(int64_t u) const
    {
        return static_cast<int>(((u + 1) * grid - 1) / total);
    }
};

// MN-major operand with the 128-byte swizzle: 64 elements × 8 per 1 KB part;
// parts along M/N `lead` bytes apart, along K `stride` bytes.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t lead, uint32_t stride)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(lead >> 4) << 16;
    d |= static_cast<uint64_t>(stride >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// kTma: the codes can be copied by TMA, whose row strides are multiples of 16 bytes.
template <int n, bool kTma>
__global__ void __launch_bounds__(kThreads, 1)
phi_grad_kernel(const __grid_constant__ CUtensorMap tm_y,
                const __grid_constant__ CUtensorMap tm_x, const uint8_t *__restrict__ Xq,
                const uint8_t *__restrict__ Xs, int64_t B, int64_t C, Units un,
                float *__restrict__ part, uint64_t limit_ns, int64_t stall)
{
    using Cf = Cfg<n>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *raw = smem + Cf::kStages * Cf::kStage;
    uint64_t *full = reinterpret_cast<uint64_t *>(raw + Cf::kRaw * kRawBytes);
    uint64_t *raw_full = full + Cf::kStages, *raw_empty = raw_full + Cf::kRaw;
    uint64_t *empty = raw_empty + Cf::kRaw;
    uint64_t *acc_full = empty + Cf::kStages, *acc_empty = acc_full + 1, *drain = acc_empty + 1;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x;
    const int64_t K = n * C, nb = kept_blocks(C);
    const int64_t u0 = un.lo(cta), u1 = un.lo(cta + 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < Cf::kStages; ++s) {
            ptx::mbar_init(&full[s], kLoadWarps + 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < Cf::kRaw; ++s) {
            ptx::mbar_init(&raw_full[s], 1);
            ptx::mbar_init(&raw_empty[s], kLoadWarps);
        }
        ptx::mbar_init(acc_full, 1);
        ptx::mbar_init(acc_empty, kLoadWarps);
        ptx::mbar_init(drain, 1);
        *abort = 0;
        ptx::fence_barrier_init();
        ptx::prefetch_tensormap(&tm_y);
    }
    if (warp == kLoadWarps + 1) ptx::tmem_alloc<Cf::kTmemCols>(tmem_holder);
    ptx::tc_fence_before();
    __syncwarp();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    ptx::pdl_wait();

    const auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (ptx::mbar_wait_bounded(bar, parity, abort, limit_ns)) return true;
        *abort = 1;
        atomicExch(&g_phi_status, kStatusTimeout);
        return false;
    };

    if (warp < kLoadWarps) {
        // lane: 8 channels of the strip; warp: tokens warp, warp + 16, ... of the block
        const int blocks = static_cast<int>(un.blocks);
        const int64_t row_q = kLoadWarps * K, row_E = kLoadWarps * n * nb;  // to its next token
        int l_block = static_cast<int>(u0 % un.blocks);
        int64_t l_strip = u0 / un.blocks, l_left = u1 - u0;
        const uint8_t *l_q = nullptr, *l_E = nullptr;  // of its first token of the next unit
        bool l_in = false;
        const auto enter = [&] {
            const int64_t q = l_strip * kStrip + lane * 8, i = q / C, c = q - i * C;
            const int64_t b = static_cast<int64_t>(l_block) * kTok + warp;
            l_in = q < K;
            l_q = Xq + b * K + q;
            l_E = Xs + (b * n + i) * nb + (c >> 5);
        };
        enter();
        uint32_t E[kRowsEach];
        uint2 q[kRowsEach];
        // the scales (and without TMA the codes) of the next unit of the CTA's range
        const auto load = [&] {
            const int64_t rows = B - static_cast<int64_t>(l_block) * kTok;
#pragma unroll
            for (int e = 0; e < kRowsEach; ++e, l_q += row_q, l_E += row_E) {
                const bool ok = l_left > 0 && l_in && warp + kLoadWarps * e < rows &&
                                in_range(1301, l_q - Xq, 8, B * K);
                E[e] = ok ? ptx::ld_dep(l_E) : kept::kScaleMin;
                if constexpr (!kTma) q[e] = ok ? kept::ld_stream_v2(l_q) : make_uint2(0, 0);
            }
            --l_left;
            if (++l_block == blocks) {
                l_block = 0;
                ++l_strip;
                enter();
            }
        };
        const uint32_t at = static_cast<uint32_t>((lane >> 3) * 8192 + (warp >> 3) * 1024 +
                                                  (warp & 7) * 128 + (((lane & 7) ^ (warp & 7)) << 4));
        // the accumulators' side: channel half·128 + quarter·32 + lane, every other 16 columns
        const int quarter = warp & 3, half = warp >> 2 & 1, m0 = warp >> 3;
        const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                               static_cast<uint32_t>(half * Cf::NT);
        int stage = 0, slot = 0, chain = 0, in_chain = 0;
        uint32_t phase = 0, raw_phase = 0;
        int64_t s_strip = l_strip;  // of the unit being stored
        int s_block = l_block;
        bool fresh = true;  // no chain of this strip has been stored
        // the tile of one unit into its stage
        const auto step = [&](bool end) {
            // (warp-uniform: the loads of the accumulators are warp-collective)
            bool ok = wait(&empty[stage], phase ^ 1);
            if constexpr (kTma) ok = ok && wait(&raw_full[slot], raw_phase);
            if (!__all_sync(0xffffffffu, ok)) return false;
            if constexpr (kTma) {
                const uint8_t *src = raw + slot * kRawBytes + warp * kStrip + lane * 8;
#pragma unroll
                for (int e = 0; e < kRowsEach; ++e)
                    q[e] = *reinterpret_cast<const uint2 *>(src + e * (kLoadWarps * kStrip));
            }
            uint8_t *dst = smem + stage * Cf::kStage + at;
#pragma unroll
            for (int e = 0; e < kRowsEach; ++e)
                *reinterpret_cast<uint4 *>(dst + e * (kLoadWarps / 8) * 1024) =
                    kept::decode8_bf16(q[e], E[e]);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(&full[stage]);
                if (kTma) ptx::mbar_arrive(&raw_empty[slot]);
            }
            if (++stage == Cf::kStages) { stage = 0; phase ^= 1; }
            if (++slot == Cf::kRaw) { slot = 0; raw_phase ^= 1; }
            load();
            const bool last = end || s_block + 1 == blocks;
            if (++in_chain == kFlush || last) {
                in_chain = 0;
                if (!__all_sync(0xffffffffu, wait(acc_full, chain & 1))) return false;
                ++chain;
                ptx::tc_fence_after();
                float *dst_p = part + (cta + s_strip) * static_cast<int64_t>(Cf::N) * kStrip +
                               half * 128 + quarter * 32 + lane;
                const bool ok = in_range(1302, cta + s_strip, 1, un.grid + un.total / un.blocks);
#pragma unroll 1
                for (int m = m0; m < Cf::NT / 48; m += 2) {
                    float s[16], v[16];
                    ptx::tmem_ld_16(taddr + m * 48 + 32, s);  // the low terms first
                    ptx::tmem_ld_16(taddr + m * 48 + 16, v);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[e] += v[e];
                    ptx::tmem_ld_16(taddr + m * 48, v);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int k = m * 16 + e;
                        if (k >= Cf::N || !ok) break;
                        // this thread alone writes the value, in the order of the chains
                        if (fresh) dst_p[k * kStrip] = s[e] + v[e];
                        else atomicAdd(dst_p + k * kStrip, s[e] + v[e]);
                    }
                    __syncwarp();
                }
                fresh = last;
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(acc_empty);
            }
            if (++s_block == blocks) {
                s_block = 0;
                ++s_strip;
            }
            return true;
        };
        load();
        for (int64_t left = u1 - u0; left > 0; --left)
            if (!step(left == 1)) break;
    } else if (warp == kLoadWarps) {
        if (lane == 0) {
            const uint64_t pol = ptx::policy_evict_last();  // every strip reads them
            int stage = 0;
            uint32_t phase = 0;
            for (int64_t u = u0; u < u1; ++u) {
                if (!wait(&empty[stage], phase ^ 1)) break;
                if (u - u0 != stall || cta != 0) {  // a test's (train.h)
                    ptx::mbar_arrive_expect_tx(&full[stage], Cf::kBBytes);
                    ptx::tma_load_2d(smem + stage * Cf::kStage + kABytes, &tm_y,
                                     static_cast<int32_t>(u % un.blocks * kTok), 0, &full[stage], pol);
                }
                if (++stage == Cf::kStages) { stage = 0; phase ^= 1; }
            }
        }
    } else if (warp == kLoadWarps + 2) {
        if (kTma && lane == 0) {
            const uint64_t pol = ptx::policy_evict_first();
            int slot = 0;
            uint32_t phase = 0;
            int64_t strip = u0 / un.blocks;
            int block = static_cast<int>(u0 % un.blocks);
            for (int64_t left = u1 - u0; left > 0; --left) {
                if (!wait(&raw_empty[slot], phase ^ 1)) break;
                ptx::mbar_arrive_expect_tx(&raw_full[slot], kRawBytes);
                ptx::tma_load_2d(raw + slot * kRawBytes, &tm_x, static_cast<int32_t>(strip * kStrip),
                                 static_cast<int32_t>(block) * kTok, &raw_full[slot], pol);
                if (++slot == Cf::kRaw) { slot = 0; phase ^= 1; }
                if (++block == un.blocks) {
                    block = 0;
                    ++strip;
                }
            }
        }
    } else {
        if (lane == 0) {
            constexpr uint32_t idesc = ptx::idesc_bf16_f32(128, Cf::NT) | (1u << 15);  // A MN-major
            int stage = 0, chain = 0, in_chain = 0;
            uint32_t phase = 0;
            int64_t block = u0 % un.blocks;
            for (int64_t u = u0; u < u1; ++u) {
                if (in_chain == 0 && !wait(acc_empty, (chain & 1) ^ 1)) break;
                if (!wait(&full[stage], phase)) break;
                ptx::tc_fence_after();
                const uint32_t a = ptx::smem_u32(smem + stage * Cf::kStage);
                const uint64_t b_desc = ptx::smem_desc_sw128(a + kABytes);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int ks = 0; ks < kTok / 16; ++ks)
                        ptx::mma_bf16(tmem + static_cast<uint32_t>(h * Cf::NT),
                                      desc_mn_sw128(a + h * 16384 + ks * 2048, 8192, 1024),
                                      b_desc + 2 * ks, idesc, in_chain == 0 && ks == 0 ? 0u : 1u);
                ptx::mma_commit(&empty[stage]);
                if (++stage == Cf::kStages) { stage = 0; phase ^= 1; }
                const bool last = u + 1 == u1 || block + 1 == un.blocks;
                if (++block == un.blocks) block = 0;
                if (++in_chain == kFlush || last) {
                    in_chain = 0;
                    ++chain;
                    ptx::mma_commit(acc_full);
                }
            }
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (*abort) {  // set before the barrier or never, so every thread sees the same
        // Copies and products of a warp that had finished before another gave up may be
        // under way too, so this comes after all of them.
        if (warp == kLoadWarps && lane == 0) ptx::let_copies_land();
        if (warp == kLoadWarps + 1 && lane == 0) {  // every MMA issued has to end before TMEM is freed
            ptx::mma_commit(drain);
            volatile int never = 0;
            ptx::mbar_wait_bounded(drain, 0, &never, limit_ns);
        }
        __syncwarp();
        __syncthreads();
    }
    ptx::pdl_trigger();
    if (warp == kLoadWarps + 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc<Cf::kTmemCols>(tmem);
    }
}

// Adds each strip's parts in the order of the CTAs, which is that of the tokens.
// The CTAs past the strips add dbias and dα, a warp per value (in a launch of their
// own they cost 2 us and a launch).
constexpr int kJoinCols = 4;  // columns of dφ_t that a CTA of 64 × 4 threads adds
__global__ void __launch_bounds__(64 * kJoinCols)
phi_join_kernel(const float *__restrict__ part, int N, int64_t K, Units un, int accumulate,
                float *__restrict__ dphi_t, BiasSums bs)
{
    ptx::pdl_wait();
    ptx::pdl_trigger();
    const int64_t strips = un.total / un.blocks;
    if (blockIdx.x >= strips) {
        const int lane = threadIdx.x & 31;
        const int k = blockIdx.y * 2 * kJoinCols + threadIdx.y * 2 + (threadIdx.x >> 5);
        if (k >= N + 3 || !in_range(1313, k, 1, N + 3)) return;
        float s = 0.f;
        for (int c = lane; c < bs.ctas; c += 32) s += ptx::ld_dep(bs.part + static_cast<int64_t>(c) * (N + 3) + k);
#pragma unroll
        for (int x = 16; x > 0; x /= 2) s += __shfl_xor_sync(0xffffffffu, s, x);
        if (lane != 0) return;
        float *dst = k < N ? bs.dbias + k : bs.dalpha + (k - N);
        *dst = accumulate ? *dst + s : s;
        return;
    }
    const int64_t strip = blockIdx.x;
    const int first = un.owner(strip * un.blocks), last = un.owner((strip + 1) * un.blocks - 1);
    const int64_t q = strip * kStrip + threadIdx.x * 4;
    if (q >= K) return;
    const int k = blockIdx.y * kJoinCols + threadIdx.y;
    if (k < N) {
        if (!in_range(1311, k * K + q, 4, N * K) ||
            !in_range(1312, first + strip, last - first + 1, un.grid + strips))
            return;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int c = first; c <= last; ++c) {
            const uint4 v = ptx::ld_dep_v4(part + ((c + strip) * N + k) * kStrip + threadIdx.x * 4);
            s.x += __uint_as_float(v.x); s.y += __uint_as_float(v.y);
            s.z += __uint_as_float(v.z); s.w += __uint_as_float(v.w);
        }
        float4 *dst = reinterpret_cast<float4 *>(dphi_t + k * K + q);
        if (accumulate) {
            const float4 o = *dst;
            s = make_float4(o.x + s.x, o.y + s.y, o.z + s.z, o.w + s.w);
        }
        *dst = s;
    }
}

Units make_units(int64_t B, int n, int64_t C, int num_sms)
{
    Units u;
    u.blocks = (B + kTok - 1) / kTok;
    const int64_t strips = (n * C + kStrip - 1) / kStrip;
    u.total = strips * u.blocks;
    u.grid = static_cast<int>(u.total < num_sms ? u.total : num_sms);
    return u;
}

template <int n>
cudaError_t launch_n(const CUtensorMap &tm, const uint8_t *Xq, const uint8_t *Xs, int64_t B,
                     int64_t C, const Units &un, int accumulate, float *dphi_t, float *part,
                     const BiasSums &bs, cudaStream_t stream, const Waits &waits)
{
    using Cf = Cfg<n>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = once_per_device(configured, [] {
        const cudaError_t c = cudaFuncSetAttribute(
            phi_grad_kernel<n, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::kSmem);
        return c != cudaSuccess ? c
                                : cudaFuncSetAttribute(phi_grad_kernel<n, false>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       Cf::kSmem);
    });
    if (e != cudaSuccess) return e;
    CUtensorMap tx = tm;
    const bool tma = n * C % 16 == 0;
    const int64_t dims[2] = {n * C, B};
    const int box[2] = {kStrip, kTok};
    if (tma && !encode_tensor(&tx, 1, 2, Xq, dims, box)) return cudaErrorInvalidValue;
    e = launch_pdl(tma ? phi_grad_kernel<n, true> : phi_grad_kernel<n, false>, dim3(un.grid),
                   dim3(kThreads), Cf::kSmem, stream, tm, tx, Xq, Xs, B, C, un, part, waits.limit_ns,
                   waits.stall_dphi);
    if (e != cudaSuccess) return e;
    const int64_t K = n * C;
    return launch_pdl(phi_join_kernel,
                      dim3(static_cast<unsigned>((K + kStrip - 1) / kStrip) + 1,
                           (Cf::N + kJoinCols - 1) / kJoinCols), dim3(64, kJoinCols),
                      0, stream, part, Cf::N, K, un, accumulate, dphi_t, bs);
}

}  // namespace

size_t phi_grad_workspace_bytes(int64_t B, int n, int64_t C, int num_sms)
{
    const Units u = make_units(B, n, C, num_sms);
    return static_cast<size_t>(u.grid + u.total / u.blocks) * num_coeffs(n) * kStrip * 4;
}

cudaError_t launch_phi_grad(const uint8_t *Xq, const uint8_t *Xs, const uint16_t *dY_terms,
                            int64_t B, int n, int64_t C, int accumulate, float *dphi_t,
                            void *workspace, const BiasSums &bs, int num_sms, cudaStream_t stream,
                            const Waits &waits)
{
    const Units un = make_units(B, n, C, num_sms);
    CUtensorMap tm;
    const int N = num_coeffs(n);
    const uint32_t rows = static_cast<uint32_t>(phi_term_rows(N));
    if (!make_tmap(&tm, dY_terms, static_cast<uint64_t>(phi_grad_padded_tokens(B)), rows, rows))
        return cudaErrorInvalidValue;
    float *part = static_cast<float *>(workspace);
    switch (n) {
#define MHC_CASE(k) \
    case k: return launch_n<k>(tm, Xq, Xs, B, C, un, accumulate, dphi_t, part, bs, stream, waits);
        MHC_CASE(1) MHC_CASE(2) MHC_CASE(3) MHC_CASE(4) MHC_CASE(5) MHC_CASE(6) MHC_CASE(7)
        MHC_CASE(8)
#undef MHC_CASE
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t read_and_clear_phi_grad_status(int *status)
{
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return e;
    int v = 0, zero = 0;
    if ((e = cudaMemcpyFromSymbol(&v, g_phi_status, sizeof v)) != cudaSuccess) return e;
    if ((e = cudaMemcpyToSymbol(g_phi_status, &zero, sizeof zero)) != cudaSuccess) return e;
    *status = v;
    return cudaSuccess;
}

}  // namespace mhc
