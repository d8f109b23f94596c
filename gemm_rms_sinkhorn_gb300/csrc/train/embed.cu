// Token ids to the n residual streams, and the table's gradient.
//
//   X[b][i][c]   = scale·T[ids[b]][c]                         for every stream i
//   dT[v][c]     = scale·Σ_{b: ids[b] = v} Σ_i dX[b][i][c]    fp32
//
// An id outside [0, V) is padding: its row of X is zero and it adds to no row
// of dT.
//
// The gradient is a sum by token id, and token counts are very uneven (a few
// ids make up much of a batch, most of the table does not occur), so it runs
// over the positions sorted by id, in three launches:
//
//   sort   CTA k owns a range of table rows.  It reads all ids, keeps those of
//          its range in their order, and counts those below it, which is where
//          its part of the sorted list starts: a stable counting sort with no
//          exchange between CTAs.  (Reading B ids per CTA is L2 traffic, a few
//          percent of the time of the rows of dX that follow.)  Rows of its range that do not
//          occur it sets to zero, so the table is written once.
//   sum    the sorted list is cut into chunks of 16 or 32 positions, whatever the
//          ids, so every CTA has the same work.  A run of one id that lies in a
//          chunk is written; a run that a chunk's edge cuts leaves its sums in
//          the workspace (one before the edge, one after).
//   join   adds the pieces of the cut runs, in the order of the chunks.
//
// All sums are fp32 in the order of the positions, so results do not depend on
// timing.  There are no atomics on sums.
//
// Both are bound by memory.  X at B=16384, n=4, C=7168 from 32000 fp32 rows: 170 us
// (207 for its bytes if no id came twice; repeated rows come from L2); a token 1.7 us.
// dT at B=16384, n=4, C=4096, V=32000: 190 us, its bytes take 156: sort with the zero
// rows 75, sum 92, join 15 and the gaps between the launches; 64 tokens 9 us.
#include <cuda_runtime.h>

#include <cstdint>

#include "check.cuh"
#include "kept.cuh"
#include "mix.cuh"
#include "ptx.cuh"
#include "train.h"

namespace mhc {
namespace {

constexpr int kMaxGridY = 65535;
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxRange = 512;  // table rows of a sorting CTA, at most
constexpr int kMostChunk = 32;  // sorted positions of a summing CTA, at most

__device__ __forceinline__ uint4 scaled8(const uint16_t *p, float scale)
{
    float f[8];
    unpack8(ptx::ld_dep_v4(p), f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= scale;
    return pack8(f);
}
__device__ __forceinline__ uint4 scaled8(const float *p, float scale)
{
    const uint4 a = ptx::ld_dep_v4(p), b = ptx::ld_dep_v4(p + 4);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(w[e]) * scale;
    return pack8(f);
}

template <typename T>
__global__ void __launch_bounds__(256)
embed_kernel(const T *__restrict__ table, const int64_t *__restrict__ ids, float scale, int64_t V,
             int64_t B, int n, int64_t C, uint16_t *__restrict__ X)
{
    const int64_t C8 = C >> 3;
    const int64_t c8 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    ptx::pdl_wait();
    ptx::pdl_trigger();
    if (c8 >= C8) return;
    for (int64_t b = blockIdx.y; b < B; b += gridDim.y) {
        if (!in_range(1401, b, 1, B)) continue;
        const int64_t id = ptx::ld_dep(ids + b);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (id >= 0 && id < V) v = scaled8(table + id * C + c8 * 8, scale);
        uint16_t *x = X + b * n * C + c8 * 8;
        for (int i = 0; i < n; ++i) ptx::st_stream_v4(x + i * C, v);
    }
}

// Workspace of the gradient: the number of positions that are not padding,
// the sorted positions and their rows, and two rows of sums per chunk.
struct GradWs {
    int *count, *pos, *row;
    int *last;    // [chunks]: where the run that starts in a chunk and is cut by its end, ends
                  // (a chunk), or -1 where there is none
    float *part;  // [chunks][2][C]: the run cut by the chunk's start, then by its end
    int chunk;    // positions of a chunk
};

// Positions of a chunk: 32 halve the cut runs' pieces (B=16384, C=4096: 187 us
// against 191 with 16), 16 halve the chain of loads where there are few CTAs (64
// tokens: 10 us against 12).
int chunk_of(int64_t B, int64_t C) { return B * C >= (int64_t{1} << 24) ? kMostChunk : 16; }
__host__ __device__ inline int64_t chunks_of(int64_t positions, int chunk)
{
    return (positions + chunk - 1) / chunk;
}

size_t carve(GradWs &w, void *base, int64_t B, int64_t C)
{
    const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    uint8_t *p = static_cast<uint8_t *>(base);
    size_t at = 0;
    w.count = reinterpret_cast<int *>(p + at);
    at += 256;
    w.chunk = chunk_of(B, C);
    w.pos = reinterpret_cast<int *>(p + at);
    at += up(static_cast<size_t>(B) * 4);
    w.row = reinterpret_cast<int *>(p + at);
    at += up(static_cast<size_t>(B) * 4);
    w.last = reinterpret_cast<int *>(p + at);
    at += up(static_cast<size_t>(chunks_of(B, w.chunk)) * 4);
    w.part = reinterpret_cast<float *>(p + at);
    at += up(static_cast<size_t>(chunks_of(B, w.chunk)) * 2 * static_cast<size_t>(C) * 4);
    return at;
}

__global__ void __launch_bounds__(kSortThreads, 2)
embed_sort_kernel(const int64_t *__restrict__ ids, int64_t V, int64_t B, int64_t C, int range,
                  int accumulate, GradWs ws, float *__restrict__ dtable)
{
    __shared__ int hist[kSortWarps][kMaxRange];  // counts, then where each warp's next one goes
    __shared__ int total[kMaxRange];
    __shared__ int sums[kSortWarps], below_w[kSortWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t v0 = static_cast<int64_t>(blockIdx.x) * range;
    const int64_t v1 = v0 + range < V ? v0 + range : V;
    const int rows = static_cast<int>(v1 - v0);
    for (int r = threadIdx.x; r < kSortWarps * kMaxRange; r += kSortThreads) (&hist[0][0])[r] = 0;
    __syncthreads();
    ptx::pdl_wait();
    ptx::pdl_trigger();

    // each warp counts a stretch of the positions
    const int64_t per = ((B + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    const int64_t lo = per * warp < B ? per * warp : B;
    const int64_t hi = lo + per < B ? lo + per : B;
    int below = 0, mine = 0;
#pragma unroll 4
    for (int64_t b = lo + lane; b < hi; b += 32) {
        const int64_t id = ptx::ld_dep(ids + b);
        below += id >= 0 && id < v0;
        if (id >= v0 && id < v1) {
            atomicAdd(&hist[warp][static_cast<int>(id - v0)], 1);
            ++mine;
        }
    }
    mine = __reduce_add_sync(0xffffffffu, mine);
    below = __reduce_add_sync(0xffffffffu, below);
    if (lane == 0) below_w[warp] = below;
    __syncthreads();

    // where each (row, warp) starts: rows in order, the warps' stretches in order
    const int r = threadIdx.x;  // kMaxRange == kSortThreads: a thread per row
    int cnt = 0;
    if (r < rows)
        for (int w = 0; w < kSortWarps; ++w) cnt += hist[w][r];
    total[r] = cnt;
    int incl = cnt;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int up = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += up;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int base = 0, all = 0;
    for (int w = 0; w < kSortWarps; ++w) {
        base += below_w[w] + (w < warp ? sums[w] : 0);
        all += below_w[w] + sums[w];
    }
    if (r < rows) {
        int at = base + incl - cnt;
        // this row's positions are [at, at + cnt): each chunk whose end lies among them
        const int k1 = (at + cnt - 1) / ws.chunk;
        for (int k = at / ws.chunk; cnt > 0 && k <= k1; ++k)
            if ((k + 1) * static_cast<int64_t>(ws.chunk) <= at + cnt && in_range(1413, k, 1, chunks_of(B, ws.chunk)))
                ws.last[k] = k == at / ws.chunk && k < k1 ? k1 : -1;
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = hist[w][r];
            hist[w][r] = at;
            at += c;
        }
    }
    if (v1 == V && threadIdx.x == 0) *ws.count = all;
    __syncthreads();

    if (mine > 0) {
        for (int64_t b0 = lo; b0 < hi; b0 += 32) {
            const int64_t b = b0 + lane;
            const int64_t id = b < hi ? ptx::ld_dep(ids + b) : -1;
            const bool in = id >= v0 && id < v1;
            if (__ballot_sync(0xffffffffu, in) == 0) continue;
            const int key = in ? static_cast<int>(id - v0) : -1;
            const unsigned same = __match_any_sync(0xffffffffu, key);
            const int rank = __popc(same & ((1u << lane) - 1u));
            const int at = in ? hist[warp][key] + rank : 0;
            __syncwarp();
            if (in && rank == 0) hist[warp][key] += __popc(same);
            __syncwarp();
            if (in && in_range(1411, at, 1, B)) {
                ws.pos[at] = static_cast<int>(b);
                ws.row[at] = static_cast<int>(id);
            }
        }
    }
    if (!accumulate) {
        const int64_t c4 = C >> 2;
        for (int k = warp; k < rows; k += kSortWarps) {
            if (total[k] != 0 || !in_range(1412, v0 + k, 1, V)) continue;
            float *dst = dtable + (v0 + k) * C;
            for (int64_t e = lane; e < c4; e += 32)
                ptx::st_stream_v4(dst + e * 4, make_uint4(0, 0, 0, 0));
        }
    }
}

__device__ __forceinline__ void put8(float *dst, const float (&v)[8], float scale, int accumulate)
{
    float4 *d = reinterpret_cast<float4 *>(dst);
    float4 a = make_float4(v[0] * scale, v[1] * scale, v[2] * scale, v[3] * scale);
    float4 b = make_float4(v[4] * scale, v[5] * scale, v[6] * scale, v[7] * scale);
    if (accumulate) {
        const float4 x = d[0], y = d[1];
        a = make_float4(x.x + a.x, x.y + a.y, x.z + a.z, x.w + a.w);
        b = make_float4(y.x + b.x, y.y + b.y, y.z + b.z, y.w + b.w);
    }
    __stcs(d, a);
    __stcs(d + 1, b);
}

template <int n>
__global__ void __launch_bounds__(256)
embed_sum_kernel(const uint16_t *__restrict__ dX, float scale, int accumulate, int64_t V,
                 int64_t B, int64_t C, GradWs ws, float *__restrict__ dtable)
{
    __shared__ int pos[kMostChunk], row[kMostChunk + 2];  // row: one before and one after too
    const int64_t C8 = C >> 3;
    const int64_t c8 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    ptx::pdl_wait();
    ptx::pdl_trigger();
    const int count = *ws.count, chunk = ws.chunk;
    for (int64_t k = blockIdx.y; k * chunk < count; k += gridDim.y) {
        const int first = static_cast<int>(k * chunk);
        const int len = count - first < chunk ? count - first : chunk;
        __syncthreads();
        for (int x = threadIdx.x; x < chunk + 2; x += blockDim.x) {
            const int p = first + x - 1;
            row[x] = p >= 0 && p < count ? ws.row[p] : -1;
            if (x < len) pos[x] = ws.pos[first + x];
        }
        __syncthreads();
        if (c8 >= C8) continue;
        float acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        // kBatch positions in flight
        constexpr int kBatch = n <= 2 ? 8 : n <= 4 ? 4 : 2;
        uint4 x[kBatch][n];
        const auto load = [&](int p, uint4 (&to)[n]) {
            if (p >= len || !in_range(1421, pos[p], 1, B)) return;
            const uint16_t *src = dX + static_cast<int64_t>(pos[p]) * n * C + c8 * 8;
#pragma unroll
            for (int i = 0; i < n; ++i) to[i] = ptx::ld_stream_v4(src + i * C);
        };
#pragma unroll
        for (int q = 0; q < kBatch; ++q) load(q, x[q]);
        bool begins = row[0] != row[1];  // the current run starts in this chunk
        for (int p0 = 0; p0 < len; p0 += kBatch)
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const int p = p0 + q;
            if (p >= len) break;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                float f[8];
                unpack8(x[q][i], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += f[e];
            }
            load(p + kBatch, x[q]);
            const int v = row[p + 1];
            const bool ends = row[p + 2] != v;
            if (!ends && p + 1 < len) continue;
            if (begins && ends) {
                if (in_range(1422, v, 1, V))
                    put8(dtable + static_cast<int64_t>(v) * C + c8 * 8, acc, scale, accumulate);
            } else if (in_range(1423, 2 * k + 1, 1, 2 * chunks_of(B, ws.chunk))) {
                put8(ws.part + (2 * k + (begins ? 1 : 0)) * C + c8 * 8, acc, 1.f, 0);
            }
            begins = true;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        }
    }
}

__device__ __forceinline__ float4 stream_f4(const float *p)
{
    const uint4 v = ptx::ld_stream_v4(p);
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                       __uint_as_float(v.w));
}

// A warp per cut run and 128 columns.  Most cut runs are two or three pieces, so a
// run is a short chain of loads and what counts is how many run at once; the pieces
// of a long one (a thousand positions are 64) are loaded eight at a time.
constexpr int kJoinWarps = 8;
constexpr int kJoinCols = 128;

__global__ void __launch_bounds__(kJoinWarps * 32)
embed_join_kernel(float scale, int accumulate, int64_t V, int64_t B, int64_t C, GradWs ws,
                  float *__restrict__ dtable)
{
    __shared__ int lasts[kJoinWarps * 32];
    __shared__ unsigned cut[kJoinWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kJoinCols + lane * 4;
    ptx::pdl_wait();
    ptx::pdl_trigger();
    const int count = *ws.count, chunk = ws.chunk;
    // a CTA takes every gridDim.y-th chunk; its threads look for the cut runs among them
    const int64_t chunks = chunks_of(count, chunk);
    for (int64_t k0 = blockIdx.y; k0 < chunks; k0 += static_cast<int64_t>(gridDim.y) * kJoinWarps * 32) {
        const int64_t mine = k0 + static_cast<int64_t>(threadIdx.x) * gridDim.y;
        const int l = (mine + 1) * chunk < count ? ws.last[mine] : -1;
        const unsigned m = __ballot_sync(0xffffffffu, l >= 0);
        lasts[threadIdx.x] = l;
        if (lane == 0) cut[warp] = m;
        __syncthreads();
        int turn = 0;
        for (int x = 0; x < kJoinWarps; ++x)
            for (unsigned left = cut[x]; left != 0; left &= left - 1) {
                if (turn++ % kJoinWarps != warp) continue;
                // the run that starts in chunk k and is cut by its end: its piece there, then
                // one of each chunk up to `last`
                const int at = x * 32 + __ffs(left) - 1;
                const int64_t k = k0 + static_cast<int64_t>(at) * gridDim.y, last = lasts[at];
                const int v = ws.row[(k + 1) * chunk];
                if (c >= C || !in_range(1431, v, 1, V) || !in_range(1432, last, 1, chunks_of(B, ws.chunk))) continue;
                const float *piece = ws.part + (2 * k + 2) * C + c;
                float4 s = stream_f4(ws.part + (2 * k + 1) * C + c);
#pragma unroll 8
                for (int64_t kk = k + 1; kk <= last; ++kk, piece += 2 * C) {
                    const float4 a = stream_f4(piece);
                    s.x += a.x; s.y += a.y; s.z += a.z; s.w += a.w;
                }
                float4 *d = reinterpret_cast<float4 *>(dtable + v * C + c);
                s = make_float4(s.x * scale, s.y * scale, s.z * scale, s.w * scale);
                if (accumulate) {
                    const float4 x4 = *d;
                    s = make_float4(x4.x + s.x, x4.y + s.y, x4.z + s.z, x4.w + s.w);
                }
                __stcs(d, s);
            }
        __syncthreads();
    }
}

int block_threads(int64_t C8)
{
    for (int t : {256, 128, 64, 32})
        if (C8 % t == 0) return t;
    return 128;
}

dim3 col_grid(int64_t rows, int64_t C8, int threads)
{
    return dim3(static_cast<unsigned>((C8 + threads - 1) / threads),
                static_cast<unsigned>(rows < kMaxGridY ? rows : kMaxGridY), 1);
}

}  // namespace

template <typename T>
cudaError_t launch_embed(const T *table, const int64_t *ids, float scale, int64_t V, int64_t B,
                         int n, int64_t C, uint16_t *X, cudaStream_t stream)
{
    const int threads = block_threads(C / 8);
    return launch_pdl(embed_kernel<T>, col_grid(B, C / 8, threads), dim3(threads), 0, stream,
                      table, ids, scale, V, B, n, C, X);
}
template cudaError_t launch_embed<uint16_t>(const uint16_t *, const int64_t *, float, int64_t,
                                            int64_t, int, int64_t, uint16_t *, cudaStream_t);
template cudaError_t launch_embed<float>(const float *, const int64_t *, float, int64_t, int64_t,
                                         int, int64_t, uint16_t *, cudaStream_t);

size_t embed_backward_workspace_bytes(int64_t, int64_t B, int, int64_t C)
{
    GradWs w;
    return carve(w, nullptr, B, C);
}

cudaError_t launch_embed_backward(const uint16_t *dX, const int64_t *ids, float scale,
                                  int accumulate, int64_t V, int64_t B, int n, int64_t C,
                                  float *dtable, void *workspace, int num_sms,
                                  cudaStream_t stream)
{
    static_assert(kMaxRange == kSortThreads, "a thread per row of the range");
    GradWs ws;
    carve(ws, workspace, B, C);
    int64_t range = (V + 2 * num_sms - 1) / (2 * num_sms);  // two CTAs an SM, in one wave
    if (range > kMaxRange) range = kMaxRange;
    cudaError_t e = launch_pdl(embed_sort_kernel,
                               dim3(static_cast<unsigned>((V + range - 1) / range)),
                               dim3(kSortThreads), 0, stream, ids, V, B, C,
                               static_cast<int>(range), accumulate, ws, dtable);
    if (e != cudaSuccess) return e;
    const int threads = block_threads(C / 8);
    const dim3 grid = col_grid(chunks_of(B, ws.chunk), C / 8, threads);
    switch (n) {
#define MHC_CASE(k)                                                                           \
    case k:                                                                                   \
        e = launch_pdl(embed_sum_kernel<k>, grid, dim3(threads), 0, stream, dX, scale,        \
                       accumulate, V, B, C, ws, dtable);                                      \
        break;
        MHC_CASE(1) MHC_CASE(2) MHC_CASE(3) MHC_CASE(4) MHC_CASE(5) MHC_CASE(6) MHC_CASE(7)
        MHC_CASE(8)
#undef MHC_CASE
    default: return cudaErrorInvalidValue;
    }
    if (e != cudaSuccess || B <= ws.chunk) return e;  // one chunk cuts no run
    const int64_t strips = (C + kJoinCols - 1) / kJoinCols;
    const int64_t rows = 16 * num_sms / strips > 1 ? 16 * num_sms / strips : 1;
    const dim3 join(static_cast<unsigned>(strips),
                    static_cast<unsigned>(rows < chunks_of(B, ws.chunk) ? rows : chunks_of(B, ws.chunk)));
    return launch_pdl(embed_join_kernel, join, dim3(kJoinWarps * 32), 0, stream, scale, accumulate,
                      V, B, C, ws, dtable);
}

}  // namespace mhc
