// Root-mean-square norms at the entry of the layer function F, and their backward.
//
//   streams    H = Σ_i H_pre[i]·X[i]   (F_pre: step 4a)
//   residual   H = A + R
//   both       rstd = 1/sqrt(Σ_c H[c]²/C + eps),  Z[c] = H[c]·rstd·gain[c]
//
// with Z in bf16 or in the 8-bit form of kept.cuh.  H is held in fp32 registers from the
// mixing to the scaling, so the inputs are read once and each output is rounded once.
// Bound by memory.  Of the copy rate of 6.78 TB/s: 8 streams, 8191 tokens of 4096 98 us, 1.0; a
// residual, 16384 tokens of 7168 148 us, 0.94; 4 streams, 16384 of 7168 in 8 bits with the
// unpacking behind it 209 us, 0.92; the backward of 16384 tokens of 7168 148 us, 0.94.  One
// token: 3.1 us with the unpacking, in a graph.  A alone, 16384 tokens of 7168: 77 us, 0.90, but
// in 8 bits 91, 0.58.
//
// Blocks walk the tokens.  A group of G threads takes a token, a thread chunks of 8 channels
// g, g + G, ... of it, the same ones in every token.  It copies the chunks of the next tokens
// into shared memory itself and alone reads them: copies are in flight while the block adds
// up its squares and writes, and nothing else waits for them.  The sum of squares is added
// in a fixed order, by lane, warp and then over the warps.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "check.cuh"
#include "mix.cuh"
#include "model.h"
#include "ptx.cuh"
#include "train/kept.cuh"

namespace mhc {
namespace {

constexpr int kMaxThreads = 512;

// How a token of C channels is laid over threads: `items` chunks of 8 channels a thread,
// `group` threads a token, `tokens` tokens a block of `most` threads.  The backward, where a
// block ends with its row of the workspace, takes blocks of 512: 16384 tokens of 2048 47 us,
// 57 with 256.
struct Layout {
    int items, group, tokens;
};
constexpr int kForwardThreads = 256, kBackwardThreads = kMaxThreads;
Layout layout_of(int64_t C, int most)
{
    const int c8 = static_cast<int>(C / 8);
    Layout l;
    l.items = c8 <= 256 ? 1 : c8 <= 1024 ? 2 : 4;
    l.group = (((c8 + l.items - 1) / l.items) + 31) / 32 * 32;
    l.tokens = l.group >= most ? 1 : most / l.group;  // one with 4 chunks a thread
    return l;
}

constexpr int kMaxWarps = kMaxThreads / 32;

// Sum of v over the threads of a group: a tree over lanes, then one over its warps.  Every
// thread of the block calls it; `red` holds a value a warp and is not written again before
// every thread has passed the next call's barrier (callers alternate between two).
__device__ __forceinline__ float group_sum(float v, float *red, int first_warp, int warps)
{
    static_assert(kMaxWarps == 16, "four steps join the warps");
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (lane & 15) < warps ? red[first_warp + (lane & 15)] : 0.f;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// 1/sqrt(ms): the approximation's 2 units in the last place and a Newton step.  0 where ms is
// 0 (a row of zeros with eps = 0) or infinite.
__device__ __forceinline__ float inverse_root(float ms)
{
    if (ms == 0.f) return 0.f;
    const float y = rsqrtf(ms);
    return y == 0.f ? 0.f : fmaf(0.5f * y, fmaf(-(ms * y), y, 1.f), y);
}

// Chunks that a thread has room for, of P pieces of 16 bytes each: what it has read of one
// makes room for the one that many on.  More in flight is mostly not better (us back to back,
// with one / two / four): 3 streams, 16384 tokens of 4096 98 / 104 / 107; 4 streams, 16384 of 2048
// 50.5 / 50.0 / 50.7; 5 streams, 8191 of 4096 68 / 70 / 70; a residual, 16384 of 2048 43 / 46 / 48;
// but 4 streams, 4096 of 16384 104 / 102 / 100 and 2 streams, 16384 of 4096 84 / 86 / 88, which
// have the other's.  Two are where a chunk is small (one stream, 16384 of 4096 69 / 65 / 67; a
// residual, 16384 of 7168 152 / 148 / 152, in 8 bits 149 / 127 / 140) and where blocks are few (8
// streams, 8191 of 4096 99.5 / 98.5, 4096 of 7168 86 / 85, of 16384 203 / 197, there with one block
// an SM).  A norm of A alone goes by the residual's: 16384 of 7168 98 / 77 / 80, 8192 of 16384
// 118 / 98 / 83, but of 2048 26 / 23 / 23.  The backward, with a gradient past the norm, 16384 of
// 7168 with one 161, with two 148.
__host__ __device__ constexpr int slots_of(int P, int items)
{
    return P == 1 || P == 8 || (P == 2 && items > 1) ? 2 : 1;
}
constexpr int kBackwardSlots = 2;
// The gain of a thread's channels stays in shared memory, but where those are many.
__host__ __device__ constexpr bool gain_kept(int items) { return items <= 2; }
// A thread's pieces of shared memory, with room for `slots` chunks of P.
__host__ __device__ constexpr int smem_pieces(int P, int items, int slots)
{
    return slots * P + (gain_kept(items) ? 2 * items : 0);
}

__device__ __forceinline__ void load_gain(const float *gain, int64_t c8, uint4 &u, uint4 &v)
{
    u = ptx::ld_dep_v4(gain + c8 * 8);
    v = ptx::ld_dep_v4(gain + c8 * 8 + 4);
}
__device__ __forceinline__ void f32_pairs(const uint4 &u, const uint4 &v, uint64_t (&t)[4])
{
    t[0] = f2_pack(__uint_as_float(u.x), __uint_as_float(u.y));
    t[1] = f2_pack(__uint_as_float(u.z), __uint_as_float(u.w));
    t[2] = f2_pack(__uint_as_float(v.x), __uint_as_float(v.y));
    t[3] = f2_pack(__uint_as_float(v.z), __uint_as_float(v.w));
}

template <int n, int ITEMS, bool Q8>  // n: streams, or 0: A + R
__global__ void __launch_bounds__(kMaxThreads, 2) rmsnorm_kernel(const NormArgs a, int G, int T)
{
    constexpr int P = n == 0 ? 2 : n, kSlots = slots_of(P, ITEMS), kWeights = n == 0 ? 1 : n;
    constexpr int kRooms = kSlots < ITEMS ? 1 : kSlots / ITEMS;  // whole tokens
    __shared__ float red[2][kMaxWarps];
    extern __shared__ __align__(16) uint4 dyn[];  // [smem_pieces][blockDim]
    const int stride = blockDim.x, group = threadIdx.x / G, g = threadIdx.x % G, warps = G >> 5;
    const int C = static_cast<int>(a.C), C8 = C >> 3, nb = static_cast<int>(kept_blocks(C));
    const uint32_t B = static_cast<uint32_t>(a.B), step = gridDim.x * T;
    const float inv_C = 1.0f / static_cast<float>(C);
    uint4 *const mine = dyn + threadIdx.x, *const gain = mine + kSlots * P * stride;
    bool live[ITEMS];  // whether the thread has such a chunk
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) live[k] = k * G + g < C8;
    // chunk k of token b, whose streams begin at `row`
    const int64_t in_step = static_cast<int64_t>(step) * (n == 0 ? 1 : n) * C;
    // 8 bits: what is read is marked to leave L2 first and the codes are stored plainly, so
    // that the kernel that reads them next finds some there (B = 16384, n = 4, C = 7168, with
    // the unpacking 221 us without, 209 with).  In bf16 it is all the same: n = 8, 8191 tokens of
    // 4096 took 99 us either way.
    const uint64_t policy = Q8 ? ptx::policy_evict_first() : 0;
    const auto copy = [&](uint4 *dst, const uint16_t *src) {
        if constexpr (Q8)
            ptx::cp_async16(dst, src, policy);
        else
            ptx::cp_async16(dst, src);
    };
    const auto fetch = [&](uint4 *slot, uint32_t b, int64_t row, int k) {
        if (b < B && live[k] && in_range(1501, b, 1, a.B)) {
            const uint16_t *x = a.X + row + (k * G + g) * 8;
            copy(slot, x);
            if constexpr (n == 0) {
                if (a.R != nullptr) copy(slot + stride, a.R + row + (k * G + g) * 8);
            } else {
#pragma unroll
                for (int i = 1; i < n; ++i) copy(slot + i * stride, x += C);
            }
        }
        ptx::cp_async_commit();
    };
    uint32_t b = blockIdx.x * T + group;
    const int64_t row0 = static_cast<int64_t>(b) * (n == 0 ? 1 : n) * C;
    ptx::pdl_wait();
    ptx::pdl_trigger();
#pragma unroll
    for (int u = 0; u < kSlots; ++u)
        fetch(mine + u * P * stride, b + u / ITEMS * step, row0 + u / ITEMS * in_step, u % ITEMS);
    if constexpr (gain_kept(ITEMS)) {
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (live[k]) load_gain(a.gain, k * G + g, gain[2 * k * stride], gain[(2 * k + 1) * stride]);
    }
    float h_next[kWeights];
    const auto weights = [&](uint32_t b) {
        if constexpr (n > 0) {
            const float *h = a.H_pre + static_cast<int64_t>(b) * n;
#pragma unroll
            for (int i = 0; i < n; ++i) h_next[i] = b < B ? ptx::ld_dep(h + i) : 0.f;
        }
    };
    weights(b);
    int turn = 0, room = 0;
    int64_t in_row = row0;
    for (uint32_t first = blockIdx.x * T; first < B; first += step, b += step, in_row += in_step, turn ^= 1) {
        const bool have = b < B;
        const int64_t row = static_cast<int64_t>(b) * C;
        uint4 *const slots = mine + room * P * ITEMS * stride;
        room = room + 1 == kRooms ? 0 : room + 1;
        float h[kWeights];
#pragma unroll
        for (int i = 0; i < kWeights; ++i) h[i] = h_next[i];
        weights(b + step);
        uint64_t f[ITEMS][4], ss = 0;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            uint4 *const x = slots + k % kSlots * P * stride;
            ptx::cp_async_wait_but<kSlots - 1>();
#pragma unroll
            for (int p = 0; p < 4; ++p) f[k][p] = 0;
            if (have && live[k]) {
                uint64_t t[4];
                if constexpr (n == 0) {
                    unpack8_pairs(x[0], f[k]);
                    if (a.R != nullptr) {
                        unpack8_pairs(x[stride], t);
#pragma unroll
                        for (int p = 0; p < 4; ++p) f[k][p] = f2_add(f[k][p], t[p]);
                    }
                } else {  // as pre_mix8 does, to the bit
                    unpack8_pairs(x[0], t);
#pragma unroll
                    for (int p = 0; p < 4; ++p) f[k][p] = f2_mul(f2_pack(h[0], h[0]), t[p]);
#pragma unroll
                    for (int i = 1; i < n; ++i) {
                        unpack8_pairs(x[i * stride], t);
#pragma unroll
                        for (int p = 0; p < 4; ++p) f[k][p] = f2_fma(f2_pack(h[i], h[i]), t[p], f[k][p]);
                    }
                }
                if (a.H != nullptr) ptx::st_stream_v4(a.H + row + (k * G + g) * 8, pack8_pairs(f[k]));
            }
            // into the same place: its values have been read
            fetch(x, b + (k + kSlots) / ITEMS * step, in_row + (k + kSlots) / ITEMS * in_step, (k + kSlots) % ITEMS);
#pragma unroll
            for (int p = 0; p < 4; ++p) ss = f2_fma(f[k][p], f[k][p], ss);
        }
        float lo, hi;
        f2_unpack(ss, lo, hi);
        const float rstd = inverse_root(fmaf(group_sum(lo + hi, red[turn], group * warps, warps), inv_C, a.eps));
        if (a.rstd != nullptr && have && g == 0) a.rstd[b] = rstd;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const bool ok = have && live[k];
            uint64_t z[4] = {0, 0, 0, 0};
            if (ok) {
                uint4 u, v;
                if constexpr (gain_kept(ITEMS))
                    u = gain[2 * k * stride], v = gain[(2 * k + 1) * stride];
                else
                    load_gain(a.gain, k * G + g, u, v);
                uint64_t w[4];
                f32_pairs(u, v, w);
#pragma unroll
                for (int p = 0; p < 4; ++p) z[p] = f2_mul(f2_mul(f[k][p], f2_pack(rstd, rstd)), w[p]);
            }
            if constexpr (Q8) {
                uint32_t m = kept::amax8(z);
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const uint32_t E = kept::scale_code_f32(m);
                if (ok) {
                    *reinterpret_cast<uint2 *>(a.Zq + row + (k * G + g) * 8) = kept::encode8(z, E);
                    if ((g & 3) == 0)  // G is a multiple of 32
                        a.Zs[static_cast<int64_t>(b) * nb + ((k * G + g) >> 2)] = static_cast<uint8_t>(E);
                }
            } else if (ok) {
                ptx::st_stream_v4(a.Z + row + (k * G + g) * 8, pack8_pairs(z));
            }
        }
    }
}

// Backward.  With t = gain·dZ and s = Σ_c t·H:
//   dH = rstd·(t − H·rstd²·s/C) + dH_skip,   dgain = Σ_b dZ·H·rstd
// The blocks walk the tokens; a thread meets the same channels in each of them, so it
// holds their share of dgain in fp32 registers.  A block's sums go to its row of the
// workspace, and a second launch adds the rows in order.
// Blocks an SM: as many as are resident at 64 registers a thread, or 128 with 4 chunks.
int blocks_per_sm(int items) { return items <= 2 ? 2 : 1; }

template <int ITEMS, bool SKIP>
__global__ void __launch_bounds__(kMaxThreads, ITEMS <= 2 ? 2 : 1)
rmsnorm_backward_kernel(const NormBackwardArgs a, int G, int T, float *__restrict__ parts)
{
    constexpr int P = SKIP ? 3 : 2, kSlots = kBackwardSlots;
    constexpr int kRooms = kSlots < ITEMS ? 1 : kSlots / ITEMS;
    __shared__ float red[2][kMaxWarps];
    extern __shared__ __align__(16) uint4 dyn[];  // [smem_pieces][blockDim]
    const int stride = blockDim.x, group = threadIdx.x / G, g = threadIdx.x % G, warps = G >> 5;
    const int C = static_cast<int>(a.C), C8 = C >> 3;
    const uint32_t B = static_cast<uint32_t>(a.B), step = gridDim.x * T;
    const float inv_C = 1.0f / static_cast<float>(C);
    uint4 *const mine = dyn + threadIdx.x, *const gain = mine + kSlots * P * stride;
    bool live[ITEMS];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) live[k] = k * G + g < C8;
    const int64_t row_step = static_cast<int64_t>(step) * C;
    const auto fetch = [&](uint4 *slot, uint32_t b, int64_t row, int k) {
        if (b < B && live[k] && in_range(1511, b, 1, a.B)) {
            const int64_t at = row + (k * G + g) * 8;
            ptx::cp_async16(slot, a.dZ + at);
            ptx::cp_async16(slot + stride, a.H + at);
            if constexpr (SKIP) ptx::cp_async16(slot + 2 * stride, a.dH_skip + at);
        }
        ptx::cp_async_commit();
    };
    uint32_t b = blockIdx.x * T + group;
    int64_t row = static_cast<int64_t>(b) * C;
    ptx::pdl_wait();
    ptx::pdl_trigger();
#pragma unroll
    for (int u = 0; u < kSlots; ++u)
        fetch(mine + u * P * stride, b + u / ITEMS * step, row + u / ITEMS * row_step, u % ITEMS);
    if constexpr (gain_kept(ITEMS)) {
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (live[k]) load_gain(a.gain, k * G + g, gain[2 * k * stride], gain[(2 * k + 1) * stride]);
    }
    const auto the_gain = [&](int k, uint64_t (&w)[4]) {
        uint4 u, v;
        if constexpr (gain_kept(ITEMS))
            u = gain[2 * k * stride], v = gain[(2 * k + 1) * stride];
        else
            load_gain(a.gain, k * G + g, u, v);
        f32_pairs(u, v, w);
    };
    uint64_t acc[ITEMS][4];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
#pragma unroll
        for (int p = 0; p < 4; ++p) acc[k][p] = 0;
    const auto the_rstd = [&](uint32_t b) { return b < B ? ptx::ld_dep(a.rstd + b) : 0.f; };
    float rstd_next = the_rstd(b);
    int turn = 0, room = 0;
    for (uint32_t first = blockIdx.x * T; first < B; first += step, b += step, row += row_step, turn ^= 1) {
        const bool have = b < B;
        uint4 *const slots = mine + room * P * ITEMS * stride;
        room = room + 1 == kRooms ? 0 : room + 1;
        const float rstd = rstd_next;
        rstd_next = the_rstd(b + step);
        const uint64_t rr = f2_pack(rstd, rstd);
        uint4 dz[ITEMS], hv[ITEMS], sk[ITEMS];
        uint64_t ss = 0;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            uint4 *const x = slots + k % kSlots * P * stride;
            ptx::cp_async_wait_but<kSlots - 1>();
            dz[k] = hv[k] = sk[k] = make_uint4(0, 0, 0, 0);
            if (have && live[k]) {
                dz[k] = x[0];
                hv[k] = x[stride];
                if constexpr (SKIP) sk[k] = x[2 * stride];
                uint64_t d[4], h[4], w[4];
                unpack8_pairs(dz[k], d);
                unpack8_pairs(hv[k], h);
                the_gain(k, w);
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    ss = f2_fma(f2_mul(w[p], d[p]), h[p], ss);
                    acc[k][p] = f2_fma(f2_mul(d[p], rr), h[p], acc[k][p]);
                }
            }
            fetch(x, b + (k + kSlots) / ITEMS * step, row + (k + kSlots) / ITEMS * row_step, (k + kSlots) % ITEMS);
        }
        float lo, hi;
        f2_unpack(ss, lo, hi);
        const float sum = group_sum(lo + hi, red[turn], group * warps, warps);
        const float back = -(rstd * (rstd * (sum * inv_C)));  // rstd² alone may be past fp32: tiny rows, eps = 0
        const uint64_t bb = f2_pack(back, back);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            if (!have || !live[k]) continue;
            uint64_t d[4], h[4], w[4], o[4];
            unpack8_pairs(dz[k], d);
            unpack8_pairs(hv[k], h);
            unpack8_pairs(sk[k], o);
            the_gain(k, w);
#pragma unroll
            for (int p = 0; p < 4; ++p) o[p] = f2_fma(rr, f2_fma(h[p], bb, f2_mul(w[p], d[p])), o[p]);
            ptx::st_stream_v4(a.dH + row + (k * G + g) * 8, pack8_pairs(o));
        }
    }
    // the sums of a block's tokens, group by group
    float4 sum[ITEMS][2];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            f2_unpack(acc[k][2 * p], sum[k][p].x, sum[k][p].y);
            f2_unpack(acc[k][2 * p + 1], sum[k][p].z, sum[k][p].w);
        }
    if constexpr (gain_kept(ITEMS)) {
        if (T > 1) {  // through the places of the gain
#pragma unroll
            for (int k = 0; k < ITEMS; ++k)
#pragma unroll
                for (int p = 0; p < 2; ++p) reinterpret_cast<float4 *>(gain)[(2 * k + p) * stride] = sum[k][p];
            __syncthreads();
            if (group != 0) return;
            for (int t = 1; t < T; ++t)
#pragma unroll
                for (int k = 0; k < ITEMS; ++k)
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const float4 u = reinterpret_cast<const float4 *>(gain)[(2 * k + p) * stride + t * G];
                        sum[k][p].x += u.x; sum[k][p].y += u.y; sum[k][p].z += u.z; sum[k][p].w += u.w;
                    }
        }
    }
    float *part = parts + static_cast<int64_t>(blockIdx.x) * C;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int c8 = k * G + g;
        if (!live[k] || !in_range(1512, c8 * 8, 8, a.C)) continue;
        *reinterpret_cast<float4 *>(part + c8 * 8) = sum[k][0];
        *reinterpret_cast<float4 *>(part + c8 * 8 + 4) = sum[k][1];
    }
}

// dgain (+)= the rows of `parts`, by slices of rows and then slices in order.  304 rows of
// 7168 are 9 MB, in L2: what counts is how many loads are in flight.  128 rows take 3.5 us
// (4.5 with 8 columns a block and 32 slices, 5.0 with 32 columns and 32 slices).
constexpr int kJoinCols = 32, kJoinSlices = 16;
__global__ void __launch_bounds__(kJoinCols * kJoinSlices)
rmsnorm_join_kernel(const float *parts, int rows, int64_t C, int accumulate, float *dgain)
{
    __shared__ float part[kJoinSlices][kJoinCols];
    const int col = threadIdx.x % kJoinCols, slice = threadIdx.x / kJoinCols;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kJoinCols + col;
    ptx::pdl_wait();
    ptx::pdl_trigger();
    float s = 0.f;
    if (c < C)
        for (int r0 = slice; r0 < rows; r0 += 8 * kJoinSlices) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int r = r0 + u * kJoinSlices;
                v[u] = r < rows ? ptx::ld_dep(parts + r * C + c) : 0.f;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) s += v[u];
        }
    part[slice][col] = s;
    __syncthreads();
    if (slice != 0 || c >= C || !in_range(1521, c, 1, C)) return;
#pragma unroll
    for (int k = 1; k < kJoinSlices; ++k) s += part[k][col];
    dgain[c] = accumulate ? ptx::ld_dep(dgain + c) + s : s;
}

int backward_blocks(int64_t B, int64_t C, int num_sms)
{
    const Layout l = layout_of(C, kBackwardThreads);
    const int64_t all = (B + l.tokens - 1) / l.tokens, most = static_cast<int64_t>(blocks_per_sm(l.items)) * num_sms;
    return static_cast<int>(all < most ? all : most);
}

// Launches `kernel` with so many pieces of shared memory a thread; blocks: how many, or 0: as
// many as are resident at once.
template <typename Args, typename... More>
cudaError_t launch_walking(void (*kernel)(const Args, int, int, More...), std::atomic<uint64_t> &done,
                           std::atomic<int> *resident, int pieces, const Layout &l, int64_t B, int blocks, int num_sms,
                           cudaStream_t stream, const Args &a, More... more)
{
    const int threads = l.group * l.tokens;
    const size_t smem = static_cast<size_t>(pieces) * threads * 16;
    cudaError_t e = once_per_device(done, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, pieces * kMaxThreads * 16);
    });
    if (e != cudaSuccess) return e;
    const int64_t all = (B + l.tokens - 1) / l.tokens;
    if (blocks == 0) {
        int each = resident[threads / 32].load(std::memory_order_relaxed);
        if (each == 0) {
            if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&each, kernel, threads, smem)) != cudaSuccess) return e;
            if (each < 1) each = 1;
            resident[threads / 32].store(each, std::memory_order_relaxed);
        }
        const int64_t most = static_cast<int64_t>(each) * num_sms;
        blocks = static_cast<int>(all < most ? all : most);
    }
    return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(threads), smem, stream, a, l.group, l.tokens,
                      more...);
}

template <int n, int ITEMS, bool Q8>
cudaError_t launch_forward_as(const NormArgs &a, int num_sms, cudaStream_t stream)
{
    constexpr int P = n == 0 ? 2 : n, pieces = smem_pieces(P, ITEMS, slots_of(P, ITEMS));
    static std::atomic<uint64_t> done{0};
    static std::atomic<int> resident[kMaxThreads / 32 + 1];
    return launch_walking(rmsnorm_kernel<n, ITEMS, Q8>, done, resident, pieces, layout_of(a.C, kForwardThreads), a.B, 0,
                          num_sms, stream, a);
}

template <int n, bool Q8>
cudaError_t launch_forward_n(const NormArgs &a, int num_sms, cudaStream_t stream)
{
    switch (layout_of(a.C, kForwardThreads).items) {
    case 1: return launch_forward_as<n, 1, Q8>(a, num_sms, stream);
    case 2: return launch_forward_as<n, 2, Q8>(a, num_sms, stream);
    default: return launch_forward_as<n, 4, Q8>(a, num_sms, stream);
    }
}

template <int ITEMS, bool SKIP>
cudaError_t launch_backward_as(const NormBackwardArgs &a, int blocks, float *parts, int num_sms, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    return launch_walking(rmsnorm_backward_kernel<ITEMS, SKIP>, done, nullptr, smem_pieces(SKIP ? 3 : 2, ITEMS, kBackwardSlots),
                          layout_of(a.C, kBackwardThreads), a.B, blocks, num_sms, stream, a, parts);
}

template <bool SKIP>
cudaError_t launch_backward_skip(const NormBackwardArgs &a, int blocks, float *parts, int num_sms, cudaStream_t stream)
{
    switch (layout_of(a.C, kBackwardThreads).items) {
    case 1: return launch_backward_as<1, SKIP>(a, blocks, parts, num_sms, stream);
    case 2: return launch_backward_as<2, SKIP>(a, blocks, parts, num_sms, stream);
    default: return launch_backward_as<4, SKIP>(a, blocks, parts, num_sms, stream);
    }
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs &a, int num_sms, cudaStream_t stream)
{
    switch (a.n) {
#define MHC_CASE(k)                                                             \
    case k:                                                                     \
        return a.Zq != nullptr ? launch_forward_n<k, true>(a, num_sms, stream)  \
                               : launch_forward_n<k, false>(a, num_sms, stream);
        MHC_CASE(0) MHC_CASE(1) MHC_CASE(2) MHC_CASE(3) MHC_CASE(4) MHC_CASE(5) MHC_CASE(6)
        MHC_CASE(7) MHC_CASE(8)
#undef MHC_CASE
    default: return cudaErrorInvalidValue;
    }
}

size_t rmsnorm_backward_workspace_bytes(int64_t B, int64_t C, int num_sms)
{
    return static_cast<size_t>(backward_blocks(B, C, num_sms)) * C * sizeof(float);
}

cudaError_t launch_rmsnorm_backward(const NormBackwardArgs &a, void *workspace, int num_sms,
                                    cudaStream_t stream)
{
    const int blocks = backward_blocks(a.B, a.C, num_sms);
    float *parts = static_cast<float *>(workspace);
    const cudaError_t e = a.dH_skip != nullptr ? launch_backward_skip<true>(a, blocks, parts, num_sms, stream)
                                               : launch_backward_skip<false>(a, blocks, parts, num_sms, stream);
    if (e != cudaSuccess) return e;
    return launch_pdl(rmsnorm_join_kernel, dim3(static_cast<unsigned>((a.C + kJoinCols - 1) / kJoinCols)),
                      dim3(kJoinCols * kJoinSlices), 0, stream, parts, blocks, a.C, a.accumulate, a.dgain);
}

}  // namespace mhc
