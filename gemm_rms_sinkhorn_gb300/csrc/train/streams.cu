// dX of the mHC layer: the residual path, F_pre, the projection and its RMS in
// one pass (formulas in pre_backward.cu, which forms what this kernel takes):
//
//   dX[j] = Σ_i H_res[i][j]·G[i] + H_pre[j]·dF + Σ_k dY[k]·φ[k] + s·X[j]
//
// Bound by memory: G, the codes of X and dF in, dX out.  A unit is 64 tokens × W
// channels (64, or 32 for n >= 5) of all n streams; a CTA per SM takes a
// contiguous range of units, the channels of a token tile in order.
//
//   warp 8    TMA loads of a unit into a stage of the ring: G and the codes (a
//             box per stream) and dF;
//   warp 11   φ for those n·W channels (one bulk copy of an image laid out beforehand)
//             into a buffer of its own, which is free again after the product;
//   warp 9    tcgen05.mma, N = n·W channels, K = N_coef padded to 16, for each of dY's
//             two bf16 terms against the same φ: dY·φ into
//             TMEM, whose lanes are the tokens, each twice (M = 128): lanes 0-63
//             are read for the lower half of the channels, 64-127 for the upper;
//   warps 0-7 two groups of four warps, each half of a lane's channels.  A thread
//             has one token: its H_res, H_pre and s stay in registers for the whole
//             tile, and its row of every operand is in shared memory or TMEM, so
//             nothing is exchanged.  dX overwrites G in the stage;
//   warp 10   TMA stores of dX, and hands the stage back.
//
// Time: B=16384, n=4, C=7168 421-445 us (385 for its bytes; the copies alone, without
// the mixing, 416-438); B=8191, n=8, C=4096 315-319 us (208 for its bytes, the copies
// alone 260).  At n = 4 memory is the bound.  At n = 8 the copies take 1600 rows of 32
// or 64 bytes a unit, at 2.8 clocks a row, and two stages do not hide a unit's load,
// mixing and store from one another (with three, when one warp made all copies, 7/8 less
// arithmetic gave 28 us of 350, no codes 31).
//
// dY's second term (the first alone leaves 2^-8 of dY in the result) costs no time up to
// n = 5 and 1 % of the backward at n = 6.  At n = 8 its rows take the third stage's
// place; φ copied by a warp of its own, which no longer waits behind the stages, makes
// up for that (the backward at B=8191, C=4096: 540 us with one term, three stages and
// one warp for all copies, 518 so; φ in parts of two streams, with three stages, 586).
//
// How it came to this (B=16384, n=4, C=7168).  With the operands read from global
// memory in the layout of warp-level products, a 128-bit request touches 8 lines and
// L1 is at its limit: 623 us.  With 128 tokens × 32 channels by TMA, rows are 64 bytes
// (32 of codes): L2 lines were evicted between a row's chunks under evict_first (2.5 GB
// read in place of 1.7): 640 us, and 490 without that hint; 64 × 64: 450.  Copying with
// cp.async in four warps in place of TMA: 494.  A warp of its own for the scales was no
// faster; words of four scales were (n = 8: 355 -> 349), and φ outside the stages
// (n = 8: 374 -> 355).
//
// For n >= 6 a mixing thread needs more than its share of registers (H_res is 64 of
// them at n = 8), and the other warps give theirs up (n = 8: 654 -> 418 us then); up to
// n = 5 it does not, and the exchange costs 10 %.
//
// Codes can only be copied by TMA where C % 16 == 0 (16-byte row strides);
// otherwise the threads read them from global memory (the backward at B=8192: C=4104
// 555-565 us at n=4 and 797-800 at n=8, C=4096 222-228 and 519-524).
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "check.cuh"
#include "kept.cuh"
#include "mhc_internal.h"
#include "mix.cuh"
#include "ptx.cuh"
#include "train.h"

namespace mhc {
namespace {

constexpr int kTok = 64;           // tokens of a tile
constexpr int kLanes = 128;        // TMEM lanes, threads of a group: each token twice
constexpr int kGroups = 2;         // groups of 128 threads that share a unit's channels
constexpr int kThreads = kGroups * kLanes + 4 * 32;
// registers of a mixing thread and of the others where they are shared out anew; as
// launched every thread has 168: 256·232 + 128·40 = 384·168
constexpr int kRegsMix = 232, kRegsRest = 40;
constexpr int kStatusTimeout = -5; // MHC_ERR_TIMEOUT
constexpr int kRingBudget = 223 * 1024;

__device__ int g_streams_status;

template <int n>
struct Cfg {
    static constexpr int N = n * n + 2 * n;
    static constexpr int kCols = dy_cols(n);           // k of the product
    static constexpr int W = streams_width(n);         // channels of a unit
    static constexpr int RB = phi_image_row(n);        // bytes of a k row
    static constexpr int RB2 = phi_image_row2(n);      // n = 8: k = 64 .. 79 apart
    static constexpr int NC = n * W;                   // product columns
    static constexpr int GB = W * 2;                   // bytes of a row of G
    static constexpr int kBBytes = NC * (RB + RB2), kGBytes = n * kTok * GB;
    static constexpr int kXBytes = n * kTok * W, kFBytes = kTok * GB;
    static constexpr int kStage = kGBytes + kXBytes + kFBytes;
    static constexpr bool kShareRegs = n >= 6;
    static constexpr int kATerm = kLanes * (RB + RB2), kABytes = kRowTerms * kATerm;
    // buffers of φ: two where that costs no stage
    static constexpr int fit(int phi) { return (kRingBudget - kABytes - phi * kBBytes) / kStage; }
    static constexpr int kPhi = fit(2) == fit(1) || fit(2) >= 6 ? 2 : 1;
    static constexpr int kStages = fit(kPhi) < 6 ? fit(kPhi) : 6;
    static constexpr int kAcc = 512 / NC < 4 ? 512 / NC : 4;  // accumulators in TMEM
    static constexpr int kEach = W / 2 / kGroups;      // channels of a thread
    static constexpr int kSmem = 1024 + kABytes + kPhi * kBBytes + kStages * kStage + 512;
    static_assert(kStages >= 2 && kAcc >= 2 && kSmem <= 227 * 1024, "shared memory, TMEM");
    static_assert(kStage % 1024 == 0 && kBBytes % 1024 == 0 && kABytes % 1024 == 0 &&
                  kXBytes % 1024 == 0, "swizzle atoms");
    static_assert(NC % 16 == 0 && NC <= 256, "MMA N for M = 128");
};

// Tensor maps: G and dX {C, n, B}, the codes {C, n, B}, dF {C, B} and dY {k,
// tokens, terms} (and from k = 64 on).
struct Maps {
    CUtensorMap g, dx, x, f, y, y2;
};

// K-major operand with rows of RB bytes under the swizzle of that width: 8-row
// groups 8·RB bytes apart.
template <int RB>
__device__ __forceinline__ uint64_t desc_k_major(uint32_t saddr)
{
    constexpr uint64_t kType = RB == 128 ? 2 : RB == 64 ? 4 : 6;
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (uint64_t{1} << 16) |
           (static_cast<uint64_t>(8 * RB / 16) << 32) | (uint64_t{1} << 46) | (kType << 61);
}

// Byte offset of 16-byte chunk `ch` of row `row` in such a layout.
template <int RB>
__device__ __forceinline__ uint32_t swizzled(int row, int ch)
{
    return static_cast<uint32_t>(row * RB + (ch ^ swizzle_xor(RB, row)) * 16);
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *m, int32_t x, int32_t y,
                                            int32_t z, uint64_t *bar, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(ptx::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(ptx::smem_u32(bar)), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap *m, int32_t x, int32_t y, int32_t z,
                                             const void *src)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(x), "r"(y), "r"(z), "r"(ptx::smem_u32(src))
                 : "memory");
}

// 32 lanes × 8 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld_8(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

// A unit's token tile and channel chunk, stepped through.
struct Unit {
    int64_t tile;
    int chunk, chunks;
    __device__ Unit(int64_t u, int chunks_)
        : tile(u / chunks_), chunk(static_cast<int>(u % chunks_)), chunks(chunks_)
    {
    }
    __device__ void step(int by)
    {
        for (chunk += by; chunk >= chunks; chunk -= chunks) ++tile;
    }
};

template <int n, bool kTmaX>
__global__ void __launch_bounds__(kThreads, 1)
streams_kernel(const __grid_constant__ Maps maps, const uint8_t *__restrict__ phi_img,
               const uint8_t *__restrict__ Xq,
               const uint8_t *__restrict__ Xs, const float *__restrict__ mix, int64_t B,
               int64_t Bp, int64_t C, int chunks, int64_t units, uint64_t limit_ns, int64_t stall)
{
    using Cf = Cfg<n>;
    constexpr int W = Cf::W, kEach = Cf::kEach;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *a_tile = smem, *phi = smem + Cf::kABytes, *ring = phi + Cf::kPhi * Cf::kBBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(ring + Cf::kStages * Cf::kStage);
    uint64_t *empty = full + Cf::kStages, *done = empty + Cf::kStages;
    uint64_t *acc_full = done + Cf::kStages, *acc_empty = acc_full + Cf::kAcc;
    uint64_t *phi_full = acc_empty + Cf::kAcc, *phi_empty = phi_full + Cf::kPhi;
    uint64_t *a_full = phi_empty + Cf::kPhi, *a_empty = a_full + 1, *drain = a_empty + 1;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t nb = kept_blocks(C);
    const int64_t u0 = units * blockIdx.x / gridDim.x;
    const uint32_t count = static_cast<uint32_t>(units * (blockIdx.x + 1) / gridDim.x - u0);

    if (threadIdx.x == 0) {
        for (int s = 0; s < Cf::kStages; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
            ptx::mbar_init(&done[s], 4 * kGroups);
        }
        for (int a = 0; a < Cf::kAcc; ++a) {
            ptx::mbar_init(&acc_full[a], 1);
            ptx::mbar_init(&acc_empty[a], 4 * kGroups);
        }
        for (int p = 0; p < Cf::kPhi; ++p) {
            ptx::mbar_init(&phi_full[p], 1);
            ptx::mbar_init(&phi_empty[p], 1);
        }
        ptx::mbar_init(a_full, 1);
        ptx::mbar_init(a_empty, 1);
        ptx::mbar_init(drain, 1);
        *abort = 0;
        ptx::fence_barrier_init();
    }
    if (warp == 9) ptx::tmem_alloc<512>(tmem_holder);
    ptx::tc_fence_before();
    __syncwarp();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    ptx::pdl_wait();

    const auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (ptx::mbar_wait_bounded(bar, parity, abort, limit_ns)) return true;
        *abort = 1;
        atomicExch(&g_streams_status, kStatusTimeout);
        return false;
    };

    if constexpr (Cf::kShareRegs) {
        if (warp < 8)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMix));
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    }
    if (warp < 8) {
        // ------------------------------------------------------------- mix
        const int group = warp >> 2, row = threadIdx.x & (kTok - 1);
        // this thread's channels of a unit
        const int ch0 = (threadIdx.x >> 6 & 1) * (W / 2) + group * kEach;
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        float h[n * n], hp[n], sx = 0.f;  // h[j·n + i] = H_res[i][j]
        int64_t have_tile = -1;
        // The next unit's scales, loaded a turn ahead; four blocks at a time where a row
        // of them can be read in words (a byte each touches as many lines).
        const bool words = nb % 4 == 0;
        Unit at_E(u0, chunks);
        uint32_t E[n], it_E = 0;
        const auto load_E = [&] {
            const int64_t b = at_E.tile * kTok + row;
            const int blk = (at_E.chunk * W + ch0) / 32;
            if (!words || it_E == 0 || blk % 4 < (W + 31) / 32) {
                const bool in = it_E < count && b < B && blk < nb;
                const int64_t at = b * n * nb + (words ? blk / 4 * 4 : blk);
#pragma unroll
                for (int j = 0; j < n; ++j) {
                    E[j] = kept::kScaleMin * 0x01010101u;
                    if (in && in_range(1241, at + j * nb, words ? 4 : 1, B * n * nb))
                        E[j] = words ? ptx::ld_dep(reinterpret_cast<const uint32_t *>(Xs + at + j * nb))
                                     : ptx::ld_dep(Xs + at + j * nb);
                }
            }
            at_E.step(1);
            ++it_E;
        };
        load_E();
        Unit un(u0, chunks);
        for (uint32_t it = 0; it < count; ++it, un.step(1)) {
            const int chunk = un.chunk;
            const int64_t b = un.tile * kTok + row;
            if (un.tile != have_tile) {
                have_tile = un.tile;
                const bool in = b < Bp && in_range(1242, b, 1, Bp);
#pragma unroll
                for (int k = 0; k < n * n; ++k) h[k] = in ? ptx::ld_dep(mix + k * Bp + b) : 0.f;
#pragma unroll
                for (int k = 0; k < n; ++k) hp[k] = in ? ptx::ld_dep(mix + (n * n + k) * Bp + b) : 0.f;
                sx = in ? ptx::ld_dep(mix + (n * n + n) * Bp + b) : 0.f;
            }
            const int byte = words ? (chunk * W + ch0) / 32 % 4 * 8 : 0;
            float sc[n];
#pragma unroll
            for (int j = 0; j < n; ++j) sc[j] = sx * kept::scale_value(E[j] >> byte & 0xFF);
            load_E();
            const uint32_t s = it % Cf::kStages, a = it % Cf::kAcc;
            const bool ok = wait(&full[s], it / Cf::kStages & 1) && wait(&acc_full[a], it / Cf::kAcc & 1);
            if (!__all_sync(0xffffffffu, ok)) break;  // what follows is warp-collective
            ptx::tc_fence_after();
            const uint32_t gs = ptx::smem_u32(ring + s * Cf::kStage);
            const uint32_t xs = gs + Cf::kGBytes, fs = xs + Cf::kXBytes;
            const uint32_t taddr = tmem + lane_base + static_cast<uint32_t>(a * Cf::NC);
            constexpr int J = n <= 4 ? n : n == 5 ? 3 : 2;  // streams of dX formed together
#pragma unroll
            for (int c8 = 0; c8 < kEach / 8; ++c8) {  // 8 channels at a time
                const int cc = ch0 / 8 + c8;
                const uint32_t at = swizzled<Cf::GB>(row, cc);
                uint64_t gp[n][4], f[4];
#pragma unroll
                for (int i = 0; i < n; ++i) unpack8_pairs(lds128(gs + i * (kTok * Cf::GB) + at), gp[i]);
                unpack8_pairs(lds128(fs + at), f);
#pragma unroll
                for (int j0 = 0; j0 < n; j0 += J) {
                    uint32_t p[J][8];
                    uint2 q[J];
#pragma unroll
                    for (int jj = 0; jj < J; ++jj)
                        if (j0 + jj < n) {
                            tmem_ld_8(taddr + (j0 + jj) * W + cc * 8, p[jj]);
                            if constexpr (kTmaX) {
                                q[jj] = lds64(xs + (j0 + jj) * (kTok * W) + swizzled<W>(row, cc / 2) +
                                              (cc & 1) * 8);
                            } else {
                                const int64_t c = static_cast<int64_t>(chunk) * W + cc * 8;
                                q[jj] = b < B && c < C
                                            ? kept::ld_stream_v2(Xq + (b * n + j0 + jj) * C + c)
                                            : make_uint2(0, 0);
                            }
                        }
                    ptx::tmem_ld_wait();
                    uint64_t acc[J][4], w[4];
#pragma unroll
                    for (int jj = 0; jj < J; ++jj)
                        if (j0 + jj < n) {
                            const uint64_t hh = f2_pack(hp[j0 + jj], hp[j0 + jj]);
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                acc[jj][x] = f2_fma(hh, f[x],
                                                    f2_pack(__uint_as_float(p[jj][2 * x]),
                                                            __uint_as_float(p[jj][2 * x + 1])));
                        }
#pragma unroll
                    for (int i = 0; i < n; ++i) {
#pragma unroll
                        for (int jj = 0; jj < J; ++jj)
                            if (j0 + jj < n) {
                                const uint64_t hh = f2_pack(h[(j0 + jj) * n + i], h[(j0 + jj) * n + i]);
#pragma unroll
                                for (int x = 0; x < 4; ++x) acc[jj][x] = f2_fma(hh, gp[i][x], acc[jj][x]);
                            }
                    }
#pragma unroll
                    for (int jj = 0; jj < J; ++jj)
                        if (j0 + jj < n) {
                            const int j = j0 + jj;
                            const uint64_t ss = f2_pack(sc[j], sc[j]);
                            kept::codes8_pairs(q[jj], w);
#pragma unroll
                            for (int x = 0; x < 4; ++x) acc[jj][x] = f2_fma(ss, w[x], acc[jj][x]);
                            sts128(gs + j * (kTok * Cf::GB) + at, pack8_pairs(acc[jj]));
                        }
                }
            }
            ptx::tc_fence_before();
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // dX, for the TMA store
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(&acc_empty[a]);
                ptx::mbar_arrive(&done[s]);
            }
        }
    } else if (warp == 8) {
        // ------------------------------------------------------- TMA loads
        if (lane == 0) {
            const uint64_t once = ptx::policy_evict_normal();
            int64_t have_tile = -1;
            uint32_t tiles = 0;
            Unit un(u0, chunks);
            for (uint32_t it = 0; it < count; ++it, un.step(1)) {
                const int32_t c0 = un.chunk * W, b0 = static_cast<int32_t>(un.tile * kTok);
                const uint32_t s = it % Cf::kStages;
                if (!wait(&empty[s], (it / Cf::kStages & 1) ^ 1)) break;
                if (it == stall && blockIdx.x == 0) continue;  // a test's (train.h)
                uint8_t *st = ring + s * Cf::kStage;
                ptx::mbar_arrive_expect_tx(&full[s], kTmaX ? Cf::kStage : Cf::kStage - Cf::kXBytes);
#pragma unroll 1
                for (int i = 0; i < n; ++i) {
                    tma_load_3d(st + i * (kTok * Cf::GB), &maps.g, c0, i, b0, &full[s], once);
                    if constexpr (kTmaX)
                        tma_load_3d(st + Cf::kGBytes + i * (kTok * W), &maps.x, c0, i, b0, &full[s], once);
                }
                ptx::tma_load_2d(st + Cf::kGBytes + Cf::kXBytes, &maps.f, c0, b0, &full[s], once);
                if (un.tile != have_tile) {
                    have_tile = un.tile;
                    if (!wait(a_empty, (tiles & 1) ^ 1)) break;
                    ++tiles;
                    ptx::mbar_arrive_expect_tx(a_full, Cf::kABytes);
                    for (int h = 0; h < 2 * kRowTerms; ++h) {  // each term's rows, twice
                        uint8_t *a = a_tile + h / 2 * Cf::kATerm;
                        tma_load_3d(a + h % 2 * kTok * Cf::RB, &maps.y, 0, b0, h / 2, a_full, once);
                        if constexpr (Cf::RB2 != 0)
                            tma_load_3d(a + kLanes * Cf::RB + h % 2 * kTok * Cf::RB2, &maps.y2, 64, b0,
                                        h / 2, a_full, once);
                    }
                }
            }
        }
    } else if (warp == 11) {
        // ----------------------------------------------------- copies of φ
        if (lane == 0) {
            const uint64_t keep = ptx::policy_evict_last();
            Unit un(u0, chunks);
            for (uint32_t it = 0; it < count; ++it, un.step(1)) {
                const uint32_t p = it % Cf::kPhi;
                if (!wait(&phi_empty[p], (it / Cf::kPhi & 1) ^ 1)) break;
                ptx::mbar_arrive_expect_tx(&phi_full[p], Cf::kBBytes);
                ptx::bulk_load(phi + p * Cf::kBBytes, phi_img + static_cast<int64_t>(un.chunk) * Cf::kBBytes,
                               Cf::kBBytes, &phi_full[p], keep);
            }
        }
    } else if (warp == 9) {
        // ------------------------------------------------------------- MMA
        if (lane == 0) {
            constexpr uint32_t idesc = ptx::idesc_bf16_f32(kLanes, Cf::NC);
            int64_t have_tile = -1;
            uint32_t tiles = 0;
            Unit un(u0, chunks);
            for (uint32_t it = 0; it < count; ++it, un.step(1)) {
                if (un.tile != have_tile) {
                    have_tile = un.tile;
                    if (!wait(a_full, tiles & 1)) break;
                    ++tiles;
                }
                const uint32_t p = it % Cf::kPhi, a = it % Cf::kAcc;
                if (!wait(&acc_empty[a], (it / Cf::kAcc & 1) ^ 1)) break;
                if (!wait(&phi_full[p], it / Cf::kPhi & 1)) break;
                ptx::tc_fence_after();
                const uint32_t d = tmem + static_cast<uint32_t>(a * Cf::NC);
                const uint32_t b_at = ptx::smem_u32(phi + p * Cf::kBBytes);
                const uint64_t bd = desc_k_major<Cf::RB>(b_at);
                constexpr int kMain = Cf::RB2 != 0 ? 4 : Cf::kCols / 16;
#pragma unroll
                for (int term = kRowTerms - 1; term >= 0; --term) {  // the small one first
                    const uint32_t a_at = ptx::smem_u32(a_tile + term * Cf::kATerm);
                    const uint64_t ad = desc_k_major<Cf::RB>(a_at);
#pragma unroll
                    for (int k = 0; k < kMain; ++k)
                        ptx::mma_bf16(d, ad + 2 * k, bd + 2 * k, idesc, term < kRowTerms - 1 || k > 0);
                    if constexpr (Cf::RB2 != 0)
                        ptx::mma_bf16(d, desc_k_major<32>(a_at + kLanes * Cf::RB),
                                      desc_k_major<32>(b_at + Cf::NC * Cf::RB), idesc, 1);
                }
                if (it + Cf::kPhi < count) ptx::mma_commit(&phi_empty[p]);
                if (it + 1 < count && un.chunk + 1 == chunks) ptx::mma_commit(a_empty);
                ptx::mma_commit(&acc_full[a]);
            }
        }
    } else if (warp == 10) {
        // ------------------------------------------------------ TMA stores
        if (lane == 0) {
            Unit un(u0, chunks);
            for (uint32_t it = 0; it < count; ++it, un.step(1)) {
                const int32_t c0 = un.chunk * W;
                const uint32_t s = it % Cf::kStages;
                if (!wait(&done[s], it / Cf::kStages & 1)) break;
#pragma unroll 1
                for (int j = 0; j < n; ++j)
                    tma_store_3d(&maps.dx, c0, j, static_cast<int32_t>(un.tile * kTok),
                                 ring + s * Cf::kStage + j * (kTok * Cf::GB));
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                ptx::mbar_arrive(&empty[s]);
            }
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (*abort) {  // set before the barrier or never, so every thread sees the same
        // Copies and products of a warp that had finished before another gave up may be
        // under way too, so this comes after all of them.
        if (warp == 8 && lane == 0) ptx::let_copies_land();
        if (warp == 9 && lane == 0) {  // every MMA issued has to end before TMEM is freed
            ptx::mma_commit(drain);
            volatile int never = 0;
            ptx::mbar_wait_bounded(drain, 0, &never, limit_ns);
        }
        __syncwarp();
        __syncthreads();
    }
    ptx::pdl_trigger();
    if (warp == 9) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc<512>(tmem);
    }
}

template <int n>
cudaError_t launch_n(const StreamsArgs &s, int num_sms, cudaStream_t stream, const Waits &waits)
{
    using Cf = Cfg<n>;
    const bool tma_x = s.C % 16 == 0;
    Maps m;
    const int64_t g_dims[3] = {s.C, n, s.B}, f_dims[2] = {s.C, s.B};
    const int64_t y_dims[3] = {Cf::kCols, s.Bp, kRowTerms};
    const int g_box[3] = {Cf::W, 1, kTok}, f_box[2] = {Cf::W, kTok};
    const int y_box[3] = {Cf::RB / 2, kTok, 1}, y2_box[3] = {16, kTok, 1};
    bool ok = encode_tensor(&m.g, 2, 3, s.dX_next, g_dims, g_box) && encode_tensor(&m.dx, 2, 3, s.dX, g_dims, g_box) &&
              encode_tensor(&m.f, 2, 2, s.dF, f_dims, f_box) && encode_tensor(&m.y, 2, 3, s.dY_rows, y_dims, y_box);
    if (ok && tma_x) ok = encode_tensor(&m.x, 1, 3, s.Xq, g_dims, g_box);
    if (ok && Cf::RB2 != 0) ok = encode_tensor(&m.y2, 2, 3, s.dY_rows, y_dims, y2_box);
    if (!ok) return cudaErrorInvalidValue;
    if (!tma_x) m.x = m.g;  // not used
    if (Cf::RB2 == 0) m.y2 = m.y;
    static std::atomic<uint64_t> configured{0};
    const cudaError_t e = once_per_device(configured, [] {
        const cudaError_t c = cudaFuncSetAttribute(
            streams_kernel<n, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::kSmem);
        return c != cudaSuccess ? c
                                : cudaFuncSetAttribute(streams_kernel<n, false>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       Cf::kSmem);
    });
    if (e != cudaSuccess) return e;
    const int64_t chunks = (s.C + Cf::W - 1) / Cf::W;
    const int64_t units = (s.B + kTok - 1) / kTok * chunks;
    return launch_pdl(tma_x ? streams_kernel<n, true> : streams_kernel<n, false>,
                      dim3(static_cast<unsigned>(units < num_sms ? units : num_sms)), dim3(kThreads),
                      Cf::kSmem, stream, m, s.phi_img, s.Xq, s.Xs, s.mix, s.B, s.Bp, s.C,
                      static_cast<int>(chunks), units, waits.limit_ns, waits.stall_dx);
}

}  // namespace

cudaError_t launch_streams(const StreamsArgs &s, int n, int num_sms, cudaStream_t stream,
                           const Waits &waits)
{
    switch (n) {
#define MHC_CASE(k) \
    case k: return launch_n<k>(s, num_sms, stream, waits);
        MHC_CASE(1) MHC_CASE(2) MHC_CASE(3) MHC_CASE(4) MHC_CASE(5) MHC_CASE(6) MHC_CASE(7)
        MHC_CASE(8)
#undef MHC_CASE
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t read_and_clear_streams_status(int *status)
{
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return e;
    int v = 0, zero = 0;
    if ((e = cudaMemcpyFromSymbol(&v, g_streams_status, sizeof v)) != cudaSuccess) return e;
    if ((e = cudaMemcpyToSymbol(g_streams_status, &zero, sizeof zero)) != cudaSuccess) return e;
    *status = v;
    return cudaSuccess;
}

}  // namespace mhc
