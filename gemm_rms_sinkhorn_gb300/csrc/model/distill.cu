// Distillation from a teacher of which K logits a row are kept: the loss, and the gradient
// of the student's logits z [B][V].
//
// With x = z·inv_tau, q = softmax(x) over the row, p_k the teacher's probabilities
// (model.h's t and t_lse; mhc.h defines them) and p_rest what they leave, 0 unless t_lse
// is given:
//   loss     = Σ_k p_k·(log p_k - log q_k) + p_rest·(log p_rest - log q_rest)
//   dz_j     = w·(M·q_j - p_j)                     j among the kept ids
//   dz_j     = w·q_j·(M - p_rest/q_rest)           else;  w = dloss·inv_tau, M = Σ p_k + p_rest
// q_rest is the sum of q over all that is not kept, summed for itself (1 - Σ q_k would
// cancel), and relative to its own largest value, so it does not underflow where the kept
// logits are far above the rest.
//
// A row is read once and its gradient written once: the blocks of a cluster of up to 8 hold
// a segment each, a thread up to 64 values in registers, and walk the rows.  A thread's
// pieces of the next segment are copied into shared memory meanwhile; only it reads them, so
// nothing else has to wait for them.  Without a gradient nothing has to be held, and a block
// takes several segments of a row one after another; clusters are for few rows then.
//
// Two more warps keep all else away from those.  One takes the K entries, one or two rows
// ahead: it works out the teacher's sums, fetches the student's logits at those of its own
// segments and marks the kept ids of a segment in a bit map, a word a thread; the thread
// overwrites its marked values with -inf before it reads them.  A mark that is there already is
// an id that came before.  The other warp joins a row's sums, over warps and over the cluster
// through distributed shared memory, answers with the factor of the gradient, and then has the
// row before to finish: its loss, and what is due at the kept ids, behind what the row's threads
// wrote there.  Where ids repeat it makes one entry of all of an id first (merge_repeats): p_k is
// their sum.  Each block of a cluster has its own ids' part of the loss; rank 0 adds them up, by
// rank.  dz may be z: a row is written after all of the cluster has summed it up.
//
// Exponentials are exp2((z - m)·c), c = inv_tau·log2 e, m the largest z seen, two values at
// a time.  As one fused multiply-add z·c - m·c they would be off by what m·c rounds away:
// with a vocabulary masked by the type's lowest value m may be that.
//
// Bound by memory, all else is kept behind it: 3.6 instructions a value for the sum and 4.4 for
// the gradient, two exponentials at 32 a clock and SM.  Of the copy rate of 6.78 TB/s: loss of
// 2048 rows of 131072 bf16, K = 64, 81 us, 0.98; with the gradient 4095 rows of 32000, K = 32,
// 84 us, 0.93 (14 rounds of rows for 13.5); 4096 of 131072, K = 128, 348 us, 0.91 (blocks of a
// cluster wait for one another); 500 rows of 50001 fp32 36.8 us, 0.80 (7 rounds for 6.6).  Few
// rows: 5.6 us, the call.  Above K = 256 the entries' warp sets the pace: 4096 rows of 32000
// with the gradient 90 us at K = 128, 97 at 256, 140 at 512, 335 at 1024.  Repeats cost the
// joining warp: loss / with the gradient, one repeat in every row 63 / 97 us at K = 128 (53 / 90
// without), 312 / 343 at 1024 (302 / 335); every id twice 71 / 106 and 589 / 629.
// All figures here and below are of calls back to back over inputs larger than L2.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "check.cuh"
#include "mix.cuh"
#include "model.h"
#include "ptx.cuh"

namespace mhc {
namespace {

constexpr int kMaxWarps = 16;  // that hold a row; two more for the entries and for joining
constexpr int kMaxThreads = kMaxWarps * 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxBits = 64;  // values a thread
constexpr int kMaxItems = 8;  // pieces a thread, but where 8 blocks do not reach
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive_release() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Barriers of the block by number, of `count` threads: one that waits, one that does not.
__device__ __forceinline__ void block_sync(int id, int count)
{
    asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(id), "r"(count) : "memory");
}
__device__ __forceinline__ void block_arrive(int id, int count)
{
    asm volatile("barrier.cta.arrive.aligned %0, %1;" ::"r"(id), "r"(count) : "memory");
}
// The same for one of the barriers `id` and `id` + 1: by numbers known to the compiler, which
// otherwise sets all 16 barriers aside for the block.
__device__ __forceinline__ void block_sync_turn(int id, int turn, int count)
{
    if (turn == 0)
        block_sync(id, count);
    else
        block_sync(id + 1, count);
}
__device__ __forceinline__ void block_arrive_turn(int id, int turn, int count)
{
    if (turn == 0)
        block_arrive(id, count);
    else
        block_arrive(id + 1, count);
}
// 8 bytes to `p`'s place in the shared memory of block `rank` of the cluster.
__device__ __forceinline__ void st_cluster(float2 *p, uint32_t rank, float2 v)
{
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(p)), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1,%2};" ::"r"(at), "f"(v.x), "f"(v.y) : "memory");
}

// ---- the logits' types, by pieces of 16 bytes
template <typename T>
struct Logit;
template <>
struct Logit<uint16_t> {
    static constexpr int kVec = 8;
    static constexpr uint32_t kLowest = 0xFF80FF80u;
    __device__ static uint16_t from(float f) { return static_cast<uint16_t>(pack_bf16_rn(f, 0.f)); }
    __device__ static void pairs(const uint4 &v, uint64_t (&f)[4]) { unpack8_pairs(v, f); }
    __device__ static uint4 pack(const float (&f)[8]) { return pack8(f); }
    // what cp_async4 brought of the 4 bytes that value i of a row lies in
    __device__ static float word(uint32_t w, int i) { return i & 1 ? bf16_hi(w) : bf16_lo(w); }
    static constexpr int kWord = 2;  // values
    __device__ static uint16_t lowest() { return 0xFF80u; }
    // the largest value of `items` pieces; a NaN is passed over (the sum meets it)
    template <int ITEMS>
    __device__ static float largest(const uint4 (&v)[ITEMS])
    {
        uint32_t m = kLowest;
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int p = 0; p < 4; ++p) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[p]));
        }
        return fmaxf(bf16_lo(m), bf16_hi(m));
    }
};
template <>
struct Logit<float> {
    static constexpr int kVec = 4;
    static constexpr uint32_t kLowest = 0xFF800000u;
    __device__ static float from(float f) { return f; }
    __device__ static void pairs(const uint4 &v, uint64_t (&f)[2])
    {
        f[0] = f2_pack(__uint_as_float(v.x), __uint_as_float(v.y));
        f[1] = f2_pack(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    __device__ static uint4 pack(const float (&f)[4])
    {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
    __device__ static float word(uint32_t w, int) { return __uint_as_float(w); }
    static constexpr int kWord = 1;
    __device__ static float lowest() { return -INFINITY; }
    template <int ITEMS>
    __device__ static float largest(const uint4 (&v)[ITEMS])
    {
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(v[j].x), __uint_as_float(v[j].y)),
                               fmaxf(__uint_as_float(v[j].z), __uint_as_float(v[j].w))));
        }
        return m;
    }
};

// A sum of exp2((z - m)·c) with its largest z.  Nothing yet: (-inf, 0).
struct Peak {
    float m, s;
};
// -inf, where nothing or only -inf was seen, as a reference that -inf may be taken from.
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ Peak merge(Peak a, Peak b, float c)
{
    const float m = fmaxf(a.m, b.m), r = reference(m);
    return {m, a.s * exp2_fast((a.m - r) * c) + b.s * exp2_fast((b.m - r) * c)};
}
// Over the lanes of a warp, the same in each of them.  The largest value in one instruction,
// as integers of the same order (v is no NaN).
__device__ __forceinline__ float warp_max(float v)
{
    int i = __float_as_int(v);
    i = __reduce_max_sync(0xffffffffu, i ^ ((i >> 31) & 0x7FFFFFFF));
    return __int_as_float(i ^ ((i >> 31) & 0x7FFFFFFF));
}
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}
__device__ __forceinline__ Peak warp_merge(Peak a, float c)
{
    const float m = warp_max(a.m);
    return {m, warp_sum(a.s * exp2_fast((a.m - reference(m)) * c))};
}
// exp2((z - r)·c) of a pair of values.
__device__ __forceinline__ void exp2_pair(uint64_t z, uint64_t minus_r, uint64_t c, float &lo, float &hi)
{
    f2_unpack(f2_mul(f2_add(z, minus_r), c), lo, hi);
    lo = exp2_fast(lo);
    hi = exp2_fast(hi);
}

// The first n values of a piece: a row's last one, which a vector would overrun.
template <typename T>
__device__ __noinline__ void store_some(T *p, uint4 v, int n)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    constexpr int per = 4 / sizeof(T);
#pragma unroll
    for (int e = 0; e < 4 * per; ++e)
        if (e < n) {
            if constexpr (per == 2)
                p[e] = static_cast<uint16_t>(w[e / 2] >> (e % 2 * 16));
            else
                p[e] = __uint_as_float(w[e]);
        }
}

// An entry's id, where it is not just that: kRepeat, an entry before has it, too (in the block that
// holds the id); kFirst, others have it, too, and its x is being added up.
constexpr int kRepeat = 1 << 30, kFirst = 1 << 29;

// The entries of an id made one: the first gets the x of their sum, log Σ e^(x - shift) + shift, the
// others are absent from here on.  For one warp; `chunks` has bit j where one of entries 32·j.. is a
// repeat.  Sums are added in the order of the entries, by chunks.
//
// A repeat looks for its first among all entries before it, 128 at once.  Where that would be many, two
// tables of Kp places each are laid first, one behind the other: an id's entry is at its place in the
// first unless another has overwritten it, and in that case in the second unless, again, overwritten;
// so few are left to look.  4096 rows of 32000, K = 128, loss, us, looking / with tables: 2 repeats a
// row 62 / 66, 6 64 / 68, 8 67 / 69, 12 79 / 75; K = 1024 6 313 / 318, 16 340 / 330; K = 32 6 54 / 53.
constexpr int kFewRepeats = 6;
__device__ __noinline__ void merge_repeats(float *x, int *ids, uint16_t *table, int Kp, float shift, uint32_t chunks)
{
    const int lane = threadIdx.x & 31;
    const auto repeat = [](int i) { return i >= 0 && (i & kRepeat) != 0; };
    const auto place1 = [&](int id) { return table + __umulhi(static_cast<uint32_t>(id) * 0x9E3779B1u, Kp); };
    const auto place2 = [&](int id) { return table + Kp + __umulhi(static_cast<uint32_t>(id) * 0x85EBCA6Bu, Kp); };
    int repeats = 0;
#pragma unroll 1
    for (uint32_t m = chunks; m != 0; m &= m - 1) {
        const int k = (__ffs(static_cast<int>(m)) - 1) * 32 + lane;
        repeats += __popc(__ballot_sync(0xffffffffu, k < Kp && repeat(ids[k])));
    }
    const bool laid = repeats > kFewRepeats;
    if (laid) {
#pragma unroll 4
        for (int k = lane; k < Kp; k += 32)
            if (ids[k] >= 0 && !repeat(ids[k])) *place1(ids[k]) = static_cast<uint16_t>(k);
        __syncwarp();
#pragma unroll 4
        for (int k = lane; k < Kp; k += 32)
            if (ids[k] >= 0 && !repeat(ids[k]) && *place1(ids[k]) != k) *place2(ids[k]) = static_cast<uint16_t>(k);
        __syncwarp();
    }
    uint32_t firsts = 0;  // as `chunks`
#pragma unroll 1
    for (uint32_t m = chunks; m != 0; m &= m - 1) {
        const int base = (__ffs(static_cast<int>(m)) - 1) * 32, k = base + lane, i = k < Kp ? ids[k] : -1;
        const bool again = repeat(i);
        const int id = i ^ kRepeat;
        int first = -1;
        if (laid && again) {  // a place that nothing was written to holds anything
            const auto right = [&](int f) { return f < Kp && (ids[f] & ~kFirst) == id; };
            first = *place1(id);
            if (!right(first)) first = *place2(id);
            if (!right(first)) first = -1;
        }
        const int end = min(base + 32, Kp);
#pragma unroll 1
        for (uint32_t left = __ballot_sync(0xffffffffu, again && first < 0); left != 0; left &= left - 1) {
            const int from = __ffs(static_cast<int>(left)) - 1, look = __shfl_sync(0xffffffffu, id, from);
            int f = -1;
#pragma unroll 4
            for (int at = lane * 4; at < end; at += 128) {
                const int4 v = *reinterpret_cast<const int4 *>(ids + at);
                if ((v.x & ~kFirst) == look) f = at;
                if ((v.y & ~kFirst) == look) f = at + 1;
                if ((v.z & ~kFirst) == look) f = at + 2;
                if ((v.w & ~kFirst) == look) f = at + 3;
            }
            f = __reduce_max_sync(0xffffffffu, f);
            if (lane == from) first = f;
        }
        const float e = again ? expf(x[k] - shift) : 0.f;
        if (again) ids[k] = -1;
        const uint32_t same = __match_any_sync(0xffffffffu, first >= 0 ? first : -1 - lane);
        float sum = e;
        if (__any_sync(0xffffffffu, (same & (same - 1)) != 0)) {
            sum = 0.f;
#pragma unroll 8
            for (int l = 0; l < 32; ++l) {
                const float more = __shfl_sync(0xffffffffu, e, l);
                if ((same >> l & 1) != 0) sum += more;
            }
        }
        if (first >= 0 && lane == __ffs(static_cast<int>(same)) - 1) {
            const bool added = (ids[first] & kFirst) != 0;
            x[first] = (added ? x[first] : expf(x[first] - shift)) + sum;
            ids[first] |= kFirst;
            firsts |= 1u << (first >> 5);
        }
        __syncwarp();
    }
    firsts = __reduce_or_sync(0xffffffffu, firsts);
#pragma unroll 1
    for (; firsts != 0; firsts &= firsts - 1) {
        const int k = (__ffs(static_cast<int>(firsts)) - 1) * 32 + lane;
        if (k >= Kp || ids[k] < 0 || (ids[k] & kFirst) == 0) continue;
        ids[k] ^= kFirst;
        x[k] = logf(x[k]) + shift;
    }
    __syncwarp();
}

constexpr int kPlaces = 4;  // rows whose entries are held: one to finish, one summed up, two ahead
struct Info {               // of a row's entries
    float kept_m, kept_s;   // the student's peak there, of this block's segments
    float base, unit;       // log p = x - base, p = e^x·unit (t_lse: e^(x - base))
    float mass, w;          // Σ p, dloss·inv_tau
    int some;               // whether entries are present
    uint32_t repeats;       // bit j: one of entries 32·j.. is a repeat (kRepeat)
};
struct Shared {
    float2 rests[2][kMaxCluster][kMaxWarps], kepts[2][kMaxCluster];  // the cluster's peaks
    float2 parts[2][kMaxCluster];  // rank 0: the blocks' parts of a loss, at the end of the last two
    float4 out;                   // the gradient: what to multiply by, the reference, whether there is one
    float2 rest[2][kMaxWarps];    // peaks by warp
    uint2 marks[3][kMaxThreads];  // bit j·VEC + e: value e of the thread's piece j is kept
    Info info[kPlaces];
};
__host__ __device__ constexpr int room_of(int K) { return (K + 15) & ~15; }  // entries
// The block's barriers:
//   kSegment   (without a gradient) a segment's marks are there, and the one before is done
//              with: the row's threads and the entries' warp meet
//   kSummed    a row's sums and entries, and the next row's marks, are there: the joining warp
//              waits
//   kAnswered  the gradient's factor is there: the row's threads wait
//   kJoined    the row is joined and the one before finished: the entries' warp waits
//   kWritten   the last row's gradient is written: the joining warp waits
// kSummed and kJoined are pairs that rows take in turn: who only arrives there may come for
// the next row before all have come for this one, but not for the one after that.
constexpr int kSegment = 1, kSummed = 2, kJoined = 4, kAnswered = 6, kWritten = 7;

// S blocks a row, Q segments of `seg` values a block.
template <typename T, bool GRAD, int ITEMS>
__global__ void __launch_bounds__(kMaxThreads + 64, ITEMS > 8 ? 1 : 2)
distill_kernel(const DistillArgs<T> a, int seg, int S, int segments)
{
    using L = Logit<T>;
    constexpr int VEC = L::kVec;
    static_assert(ITEMS * VEC <= kMaxBits, "a thread's values have a bit each");
    __shared__ Shared sh;
    // pieces [warps][ITEMS][32], a warp's one after another; then the entries.  Lines of 128
    // bytes: 16 bytes past that the loss of 2048 rows of 131072 takes 99 us, not 83.
    extern __shared__ __align__(128) uint4 dyn[];
    constexpr int kWarpPieces = ITEMS * 32;

    const int Q = GRAD ? 1 : segments;
    const int threads = blockDim.x - 64, warps = threads >> 5;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = S > 1 ? cluster_rank() : 0;
    const int lo = static_cast<int>(rank) * Q * seg;
    const unsigned mine_values = max(min(a.V - lo, Q * seg), 0);  // of the row
    const float c = a.inv_tau * kLog2e;
    const int64_t step = gridDim.x / S, first = blockIdx.x / S;
    // [kPlaces][K, to a multiple of 16] each: x = t·inv_tau less the row's largest (t_lse: not
    // less), the word that z lies in, the id (-1: absent, or kRepeat); then a row's entries as they come
    const int Kp = room_of(a.K);
    float *const xs = reinterpret_cast<float *>(dyn + warps * kWarpPieces);
    uint32_t *const words = reinterpret_cast<uint32_t *>(xs + kPlaces * Kp);
    int *const ids = reinterpret_cast<int *>(words + kPlaces * Kp);
    int64_t *const came_ids = reinterpret_cast<int64_t *>(ids + kPlaces * Kp);
    float *const came_ts = reinterpret_cast<float *>(came_ids + Kp);
    uint16_t *const table = reinterpret_cast<uint16_t *>(came_ts + Kp);  // [2][K, to a multiple of 16]: merge_repeats'
    // A row's barrier of the cluster, for the warps that do not wait for the others' sums:
    // they take part a row behind.
    const auto pass = [&](int64_t b) {
        if (S > 1) {
            if (b != first) cluster_wait();
            cluster_arrive_relaxed();
        }
    };
    // Their last part is in the last row's barrier and in the one of the last losses.
    const bool losses = !GRAD || a.loss != nullptr;
    const auto leave = [&] {
        if (S > 1) {
            cluster_wait();
            if (losses) {
                cluster_arrive_relaxed();
                cluster_wait();
            }
        }
    };

    for (int i = tid; i < 3 * kMaxThreads; i += blockDim.x) (&sh.marks[0][0])[i] = make_uint2(0, 0);
    // No early trigger: blocks of the next kernel that wait in the places of these cost more
    // (4096 rows of 131072, back to back: 592 us, 473 without) than their start would save.
    ptx::pdl_wait();
    if (S > 1) {  // every block has started before another writes into it
        cluster_arrive_relaxed();
        cluster_wait();
    }
    __syncthreads();

    if (warp == warps) {  // ---- the entries
        float lse = 0.f, dloss = 0.f;
        // What is given for row b, on its way; a lane reads what it has copied itself.
        const auto read_ahead = [&](int64_t b) {
            if (b < a.B) {
                const int64_t *id = a.ids + b * a.K;
                const float *t = a.t + b * a.K;
#pragma unroll 4
                for (int k = lane; k < a.K; k += 32) {
                    ptx::cp_async8(came_ids + k, id + k);
                    ptx::cp_async4(came_ts + k, t + k);
                }
                if (a.t_lse != nullptr) lse = ptx::ld_dep(a.t_lse + b);
                if constexpr (GRAD) dloss = ptx::ld_dep(a.dloss + b);
            }
            ptx::cp_async_commit();
        };
        // Marks value `at` of a segment; whether it has been marked before.
        const auto mark = [&](uint2 *marks, int at) {
            const int p = at / VEC, bit = p / 32 % ITEMS * VEC + at % VEC;
            uint32_t *w = &marks[p / kWarpPieces * 32 + p % 32].x + (bit >> 5);
            return (atomicOr(w, 1u << (bit & 31)) >> (bit & 31) & 1u) != 0;
        };
        // Whether an entry's id i has come before; `marked`: whether its mark was there.  Of
        // lanes with the same id, which came to mark it in any order, the first one is new.
        const auto repeats = [&](bool in, int i, bool marked) {
            if (!__any_sync(0xffffffffu, marked)) return false;
            const uint32_t same = __match_any_sync(0xffffffffu, in ? i : -1 - lane);
            const uint32_t fresh = __ballot_sync(0xffffffffu, in && !marked);
            return in && ((same & fresh) == 0 || lane != __ffs(static_cast<int>(same)) - 1);
        };
        uint32_t chunks = 0;  // bit j: this lane has found a repeat in entries 32·j.. of the row prepared last
        // Row b into its place, its first segment's kept ids into `marks`; after read_ahead(b).
        const auto prepare = [&](int64_t b, int place, uint2 *marks) {
            if (b >= a.B) {
                ptx::cp_async_commit();
                return;
            }
            float *x = xs + place * Kp;
            uint32_t *word = words + place * Kp;
            int *idk = ids + place * Kp;
            const T *row = a.z + b * a.ld;
            const int count = max(min(a.V - lo, seg), 0);
            float m = -INFINITY;
            bool some = false;
            ptx::cp_async_wait_all();  // read_ahead's
            chunks = 0;
#pragma unroll 4
            for (int base = 0; base < Kp; base += 32) {
                const int k = base + lane;
                const int64_t id = k < a.K ? came_ids[k] : -1;
                const float t = k < a.K ? came_ts[k] : 0.f;
                const bool here = id >= 0 && id < a.V && t != -INFINITY;
                const int i = here ? static_cast<int>(id) : -1;
                if (k < Kp) x[k] = t;
                if (here) {
                    some = true;
                    m = fmaxf(m, t);
                    if (static_cast<unsigned>(i - lo) < mine_values && in_range(1605, i, 1, a.V))
                        ptx::cp_async4(word + k, row + (i & -L::kWord));
                }
                const bool in = i >= lo && i - lo < count, again = repeats(in, i, in && mark(marks, i - lo));
                if (again) chunks |= 1u << (base >> 5);
                if (k < Kp) idk[k] = again ? i | kRepeat : i;
            }
            ptx::cp_async_commit();
            some = __any_sync(0xffffffffu, some);
            uint32_t repeats_of_all = 0;
            if constexpr (GRAD) repeats_of_all = __reduce_or_sync(0xffffffffu, chunks);
            // the difference first: t times inv_tau may overflow where t is the type's lowest value
            m = a.t_lse != nullptr ? 0.f : warp_max(m);
            float s = 0.f;
#pragma unroll 4
            for (int k = lane; k < a.K; k += 32) {
                x[k] = (x[k] - m) * a.inv_tau;
                if (idk[k] >= 0) s += expf(x[k] - lse);
            }
            s = warp_sum(s);
            if (lane == 0) {
                Info &r = sh.info[place];
                r.base = a.t_lse != nullptr ? lse : logf(s);
                r.unit = a.t_lse != nullptr ? 1.f : 1.f / s;
                r.mass = a.t_lse != nullptr ? s : 1.f;
                r.w = dloss * a.inv_tau;
                r.some = some;
                if constexpr (GRAD) r.repeats = repeats_of_all;
            }
            __syncwarp();
        };
        // The peak at the kept ids of this block, each once.
        const auto peak = [&](int place) {
            const uint32_t *word = words + place * Kp;
            const int *idk = ids + place * Kp;
            Peak kept = {-INFINITY, 0.f};
#pragma unroll 4
            for (int k = lane; k < a.K; k += 32)
                if (static_cast<unsigned>(idk[k] - lo) < mine_values)
                    kept.m = fmaxf(kept.m, L::word(word[k], idk[k]));
            kept.m = warp_max(kept.m);
            const float r = reference(kept.m);
#pragma unroll 4
            for (int k = lane; k < a.K; k += 32)
                if (static_cast<unsigned>(idk[k] - lo) < mine_values)
                    kept.s += exp2_fast((L::word(word[k], idk[k]) - r) * c);
            kept.s = warp_sum(kept.s);
            if (lane == 0) {
                sh.info[place].kept_m = kept.m;
                sh.info[place].kept_s = kept.s;
            }
            __syncwarp();
        };
        constexpr int kLead = GRAD ? 2 : 1;  // rows prepared ahead
        read_ahead(first);
        // the first row's marks are all that the others need to begin (500 rows of fp32 38.0 us
        // behind both rows, 37.2 behind one)
#pragma unroll 1
        for (int r = 0; r < kLead; ++r) {
            prepare(first + r * step, r, sh.marks[r]);
            read_ahead(first + (r + 1) * step);
            if (r == 0) __syncthreads();  // the first marks are there
        }
        int turn = 0, place = 0, third = kLead;  // third: of the marks, where the row after the lead has them
        int unit = 0;
        for (int64_t b = first; b < a.B; b += step, turn ^= 1, place = (place + 1) % kPlaces) {
            if constexpr (!GRAD) {
                int *idk = ids + place * Kp;
                for (int q = 1; q <= Q; ++q) {
                    block_sync(kSegment, threads + 32);
                    unit ^= 1;
                    if (q == Q) break;
                    const int from = lo + q * seg, count = max(min(a.V - from, seg), 0);
#pragma unroll 2
                    for (int base = 0; base < Kp; base += 32) {
                        const int k = base + lane, i = k < Kp ? idk[k] : -1;
                        const bool in = i >= from && i - from < count;
                        if (repeats(in, i, in && mark(sh.marks[unit], i - from))) {
                            idk[k] = i | kRepeat;
                            chunks |= 1u << (base >> 5);
                        }
                    }
                    __syncwarp();
                }
                const uint32_t all = __reduce_or_sync(0xffffffffu, chunks);
                if (lane == 0) sh.info[place].repeats = all;
            }
            if constexpr (GRAD)
                ptx::cp_async_wait_but<2>();
            else
                ptx::cp_async_wait_but<1>();
            __syncwarp();
            peak(place);
            block_arrive_turn(kSummed, turn, threads + 64);
            pass(b);
            // A row on: its place is that of a row that has been finished, and its marks that of
            // one that has been summed up, once the row before this one is joined.
            if (b != first) block_sync_turn(kJoined, turn ^ 1, 64);
            prepare(b + kLead * step, (place + kLead) % kPlaces, sh.marks[GRAD ? third : unit]);
            read_ahead(b + (kLead + 1) * step);
            third = third == 2 ? 0 : third + 1;
        }
        if constexpr (!GRAD) block_sync(kSegment, threads + 32);
        block_sync_turn(kJoined, turn ^ 1, 64);
        leave();
        return;
    }

    if (warp > warps) {  // ---- joining
        // What a joined row leaves to do at this block's kept ids: their part of the loss, and the gradient.
        const auto finish = [&](int64_t b, int place, Peak rest, Peak whole) {
            const Info &r = sh.info[place];
            if (r.repeats != 0)
                merge_repeats(xs + place * Kp, ids + place * Kp, table, Kp, a.t_lse != nullptr ? r.base : 0.f, r.repeats);
            const float *x = xs + place * Kp;
            const uint32_t *word = words + place * Kp;
            const int *idk = ids + place * Kp;
            const float base = r.base, unit = r.unit, mass = r.mass, w = r.w, shift = a.t_lse != nullptr ? base : 0.f;
            const bool some = r.some;
            const float p_rest = a.t_lse != nullptr && rest.s != 0.f ? fmaxf(1.f - mass, 0.f) : 0.f;
            const float ln_s = logf(whole.s), factor = w * (mass + p_rest) / whole.s, ref = reference(whole.m);
            float part = 0.f;
#pragma unroll 2
            for (int k = lane; k < a.K; k += 32) {
                const int i = idk[k];
                if (static_cast<unsigned>(i - lo) >= mine_values) continue;
                const float p = expf(x[k] - shift) * unit, z = L::word(word[k], i);
                if (losses && p != 0.f) part += p * (x[k] - base - ((z - whole.m) * a.inv_tau - ln_s));
                if constexpr (GRAD) {
                    if (in_range(1604, i, 1, a.V))
                        a.dz[b * a.ld + i] = L::from(fmaf(exp2_fast((z - ref) * c), factor, -(w * p)));
                }
            }
            if (losses) {
                part = warp_sum(part);
                if (rank == 0 && p_rest > 0.f)
                    part += p_rest * (logf(p_rest) - ((rest.m - whole.m) * a.inv_tau + logf(rest.s) - ln_s));
                // z has no distribution (all -inf, a NaN, +inf), or the teacher's sum is no number
                if (!(whole.s > 0.f) || !(r.mass < INFINITY)) part = NAN;
                if (!some) part = 0.f;
                if (S == 1 && lane == 0) a.loss[b] = part;
            }
            __syncwarp();
            return part;
        };
        // Row b's loss from what the blocks of the cluster have for it, in rank 0.
        const auto add_up = [&](int64_t b, float part) {
            part = warp_sum(lane < S ? part : 0.f);
            if (lane == 0 && in_range(1606, b, 1, a.B)) a.loss[b] = part;
        };
        float part = 0.f;  // of the last finished row
        __syncthreads();
        Peak last_rest = {}, last_whole = {};
        int turn = 0, place = 0;
        for (int64_t b = first; b < a.B; b += step, turn ^= 1, place = (place + 1) % kPlaces) {
            block_sync_turn(kSummed, turn, threads + 64);
            Peak rest = {-INFINITY, 0.f};
            if (lane < warps) rest = {sh.rest[turn][lane].x, sh.rest[turn][lane].y};
            const Info &r = sh.info[place];
            Peak kept = {r.kept_m, r.kept_s};
            if (S > 1) {
                if (lane < warps)
                    for (int i = 0; i < S; ++i) st_cluster(&sh.rests[turn][rank][lane], i, make_float2(rest.m, rest.s));
                if (lane < S) st_cluster(&sh.kepts[turn][rank], lane, make_float2(kept.m, kept.s));
                if (losses && lane == 0) st_cluster(&sh.parts[turn][rank], 0, make_float2(part, 0.f));
                cluster_arrive_release();
                cluster_wait();
                rest = kept = {-INFINITY, 0.f};
                if (lane < S) kept = {sh.kepts[turn][lane].x, sh.kepts[turn][lane].y};
                float2 p[kMaxCluster / 2];
#pragma unroll
                for (int i = 0; i < kMaxCluster / 2; ++i) {  // two blocks' warps at once
                    const int from = 2 * i + lane / kMaxWarps, w = lane % kMaxWarps;
                    p[i] = from < S && w < warps ? sh.rests[turn][from][w] : make_float2(-INFINITY, 0.f);
                    rest.m = fmaxf(rest.m, p[i].x);
                }
#pragma unroll
                for (int i = 0; i < kMaxCluster / 2; ++i)
                    rest.s += p[i].y * exp2_fast((p[i].x - reference(rest.m)) * c);
                kept = warp_merge(kept, c);
            }
            rest = warp_merge(rest, c);
            const Peak whole = merge(rest, kept, c);
            if constexpr (GRAD) {
                if (lane == 0) {
                    const float p_rest = a.t_lse != nullptr && rest.s != 0.f ? fmaxf(1.f - r.mass, 0.f) : 0.f;
                    // q_rest·(M - p_rest/q_rest) = M·q_rest - p_rest, shared out by exp2 over the rest's sum
                    const float q_rest = rest.s == 0.f ? 0.f : rest.s * exp2_fast((rest.m - whole.m) * c) / whole.s;
                    const float scale = rest.s != 0.f ? r.w * ((r.mass + p_rest) * q_rest - p_rest) / rest.s
                                                      : whole.s > 0.f ? 0.f : NAN;
                    sh.out = make_float4(scale, reference(rest.m), r.some ? 1.f : 0.f, 0.f);
                }
                __syncwarp();
                block_arrive(kAnswered, threads + 32);
            }
            if (S > 1 && losses && rank == 0 && b - step > first)
                add_up(b - 2 * step, sh.parts[turn][lane % kMaxCluster].x);
            // everyone's stores of the row before precede this row's sums
            if (b != first) part = finish(b - step, (place + kPlaces - 1) % kPlaces, last_rest, last_whole);
            block_arrive_turn(kJoined, turn, 64);
            last_rest = rest;
            last_whole = whole;
        }
        if constexpr (GRAD) block_sync(kWritten, threads + 32);
        const int64_t last = first + (a.B - 1 - first) / step * step;
        const float end = finish(last, (place + kPlaces - 1) % kPlaces, last_rest, last_whole);
        if (S > 1 && losses) {
            if (lane == 0) st_cluster(&sh.parts[turn][rank], 0, make_float2(part, end));
            cluster_arrive_release();
            cluster_wait();
            if (rank == 0) {
                const float2 p = sh.parts[turn][lane % kMaxCluster];
                if (last != first) add_up(last - step, p.x);
                add_up(last, p.y);
            }
        }
        return;
    }

    // ---- the row
    const uint64_t cc = f2_pack(c, c);
    const int at0 = warp * kWarpPieces + lane;  // this thread's first piece; the next ones 32 on
    uint4 *const mine = dyn + at0;
    // Segment q: how many values it has, how many pieces are left from at0 on, how many of
    // those are whole.
    const auto count_of = [&](int q) { return max(min(a.V - lo - q * seg, seg), 0); };
    const auto fetch = [&](int64_t b, int q) {
        const T *row = a.z + b * a.ld + lo + q * seg + at0 * VEC;
        const int left = (count_of(q) + VEC - 1) / VEC - at0;
#pragma unroll
        for (int j = 0; j < ITEMS; ++j)
            if (j * 32 < left && in_range(1602, lo + q * seg + (at0 + j * 32) * VEC, VEC, a.ld))
                ptx::cp_async16(mine + j * 32, row + j * 32 * VEC);
        ptx::cp_async_commit();
    };
    const auto strike = [&](uint32_t bits, int from) {  // values from + 0..31 that have a bit become -inf
        while (bits != 0) {
            const int v = from + __ffs(static_cast<int>(bits)) - 1;
            bits &= bits - 1;
            reinterpret_cast<T *>(mine + v / VEC * 32)[v % VEC] = L::lowest();
        }
    };
    if (in_range(1601, first, 1, a.B)) fetch(first, 0);
    __syncthreads();
    int turn = 0, place = 0;  // place: of the marks, by rows in threes or by segments in turn
    for (int64_t b = first; b < a.B; b += step, turn ^= 1) {
        Peak rest = {-INFINITY, 0.f};
        uint4 v[ITEMS];
        int count = 0, left = 0;
        bool tail = false;  // whether the row's last piece, one that is not whole, is this thread's
        for (int q = 0; q < Q; ++q) {
            count = count_of(q);
            left = (count + VEC - 1) / VEC - at0;
            if constexpr (!GRAD) block_sync(kSegment, threads + 32);
            uint2 marks = sh.marks[place][tid];
            if ((marks.x | marks.y) != 0) sh.marks[place][tid] = make_uint2(0, 0);
            place = place == (GRAD ? 2 : 1) ? 0 : place + 1;
            // what lies past the end in the last piece is struck out, too
            tail = count % VEC != 0 && left > 0 && left <= kWarpPieces && left % 32 == 1;
            if (tail) {
                constexpr int per = 32 / VEC;
                const int j = left / 32;
                (j < per ? marks.x : marks.y) |= ((1u << VEC) - (1u << (count % VEC))) << (j % per * VEC);
            }
            ptx::cp_async_wait_all();
            if (left <= (ITEMS - 1) * 32) {
#pragma unroll
                for (int j = 0; j < ITEMS; ++j)  // pieces past the end
                    if (j * 32 >= left) mine[j * 32] = make_uint4(L::kLowest, L::kLowest, L::kLowest, L::kLowest);
            }
            strike(marks.x, 0);
            strike(marks.y, 32);
#pragma unroll
            for (int j = 0; j < ITEMS; ++j) v[j] = mine[j * 32];
            Peak p;
            p.m = L::template largest<ITEMS>(v);
            const float r = reference(p.m);
            const uint64_t minus_r = f2_pack(-r, -r);
            uint64_t s = 0;
#pragma unroll
            for (int j = 0; j < ITEMS; ++j) {
                uint64_t f[VEC / 2];
                L::pairs(v[j], f);
#pragma unroll
                for (int e = 0; e < VEC / 2; ++e) {
                    float l, h;
                    exp2_pair(f[e], minus_r, cc, l, h);
                    s = f2_add(s, f2_pack(l, h));
                }
            }
            float l, h;
            f2_unpack(s, l, h);
            p.s = l + h;
            if constexpr (GRAD)
                rest = p;
            else
                rest = merge(rest, p, c);
            // The next segment (with a gradient: below) behind the sum, not as soon as its place is
            // free: 2048 rows of 131072 81 us, 88; 16384 of 8192 58, 63; 4096 of 32000 42, 47.
            if (q + 1 < Q)
                fetch(b, q + 1);
            else if (!GRAD && b + step < a.B)
                fetch(b + step, 0);
        }
        rest = warp_merge(rest, c);
        if (lane == 0) sh.rest[turn][warp] = make_float2(rest.m, rest.s);
        __syncwarp();
        block_arrive_turn(kSummed, turn, threads + 64);
        pass(b);
        if constexpr (GRAD) {
            // The next row here, not as soon as its place is free: less is in flight while other
            // blocks sum up.  4096 rows of 131072 348 us, 366 as soon as may be, 354 behind the
            // answer; 4096 of 50304 135, 145, 142; 500 of 50001 in fp32 37, 38, 40; but 4096 of
            // 32000 in fp32 174, 169, 166.
            if (b + step < a.B) {
                fetch(b + step, 0);
                // With few blocks on an SM and none to wait for, a block's reads and writes go better
                // apart: 4095 rows of 32000 84 us, 91 without; 8192 of 20000 106, 122; in fp32 of 16384
                // 176, 184.  Not so where 8 warps or fewer hold a row (16384 of 8192 102, 99; 4096 of
                // 16000 47, 45) and in clusters (4096 of 50304 140, 135; of 131072 351, 348; but of 32000
                // in fp32 165, 174).
                if (S == 1 && warps > 8) ptx::cp_async_wait_all();
            }
            block_sync(kAnswered, threads + 32);
            const float4 o = sh.out;
            const uint64_t minus_r = f2_pack(-o.y, -o.y), times = f2_pack(o.x, o.x);
            T *out = a.dz + b * a.ld + lo + at0 * VEC;
            const int full = count / VEC - at0;
            if (o.z == 0.f) {  // no entries: zeros, whatever z holds
                for (int j = 0; j < ITEMS; ++j) {
                    if (j * 32 < full)
                        ptx::st_stream_v4(out + j * 32 * VEC, make_uint4(0, 0, 0, 0));
                    else if (tail && j == left / 32)
                        store_some(out + j * 32 * VEC, make_uint4(0, 0, 0, 0), count % VEC);
                }
                continue;
            }
#pragma unroll
            for (int j = 0; j < ITEMS; ++j) {
                uint64_t f[VEC / 2];
                float g[VEC];
                // unpacked again here, not held in registers since the sum
                asm volatile("" : "+r"(v[j].x), "+r"(v[j].y), "+r"(v[j].z), "+r"(v[j].w));
                L::pairs(v[j], f);
#pragma unroll
                for (int e = 0; e < VEC / 2; ++e) {
                    float l, h;
                    exp2_pair(f[e], minus_r, cc, l, h);
                    f2_unpack(f2_mul(f2_pack(l, h), times), g[2 * e], g[2 * e + 1]);
                }
                if (j * 32 < full) {
                    if (in_range(1603, lo + (at0 + j * 32) * VEC, VEC, a.V))
                        ptx::st_stream_v4(out + j * 32 * VEC, L::pack(g));
                } else if (tail && j == left / 32) {
                    store_some(out + j * 32 * VEC, L::pack(g), count % VEC);
                }
            }
        }
    }
    if constexpr (GRAD)
        block_arrive(kWritten, threads + 32);
    else
        block_sync(kSegment, threads + 32);
    leave();
}

// Blocks a row (a power of two up to 8), segments a block, warps that hold a segment and
// pieces a thread.
struct Plan {
    int S, Q, seg, warps, items;
};
constexpr int kPieces = 4096;    // a segment's most, but where a gradient needs all and 8 blocks do not reach
constexpr int kEntryBytes = kPlaces * 12 + 12 + 4;
constexpr int kMinPieces = 256;  // rows are split further only down to this

template <typename T>
Plan plan_of(int64_t B, int V, bool grad, int num_sms)
{
    constexpr int VEC = Logit<T>::kVec;
    const auto seg_of = [&](int parts) { return ((V + parts - 1) / parts + 7) / 8 * 8; };
    const auto segments = [&](int s) { return (seg_of(s) / VEC + kPieces - 1) / kPieces; };
    Plan p;
    p.S = 1;
    if (grad)
        while (p.S < kMaxCluster && segments(p.S) > 1) p.S *= 2;
    // More blocks a row where that takes a fifth off the pieces that one after another go
    // through a block (two an SM): where rows are few, or leave many places empty at the end.
    const auto rounds = [&](int s) { return (B * s + 2 * num_sms - 1) / (2 * num_sms) * (seg_of(s) / VEC); };
    for (int s = p.S * 2; s <= kMaxCluster && seg_of(s) / VEC >= kMinPieces; s *= 2)
        if (rounds(s) * 5 <= rounds(p.S) * 4) p.S = s;
    p.Q = grad ? 1 : segments(p.S);
    p.seg = seg_of(p.S * p.Q);
    // a piece a thread where a block has one segment of one row, for the shortest way through
    const int pieces = p.seg / VEC, each = B * p.S <= num_sms && p.Q == 1 ? 1 : kMaxItems;
    const int most = (pieces + 32 * each - 1) / (32 * each);
    const int warps = most < kMaxWarps ? most : kMaxWarps;
    p.items = 1;
    while (warps * 32 * p.items < pieces) p.items *= 2;
    p.warps = (pieces + 32 * p.items - 1) / (32 * p.items);
    return p;
}

template <typename T, bool GRAD, int ITEMS>
cudaError_t launch_items(const DistillArgs<T> &a, const Plan &p, cudaStream_t stream)
{
    // Clusters that are resident at once: by device, log2 of the cluster, warps, and how much
    // shared memory the entries take (up to 512 two blocks of 16 warps are resident)
    static std::atomic<int> resident[64][4][kMaxWarps + 1][3];
    constexpr int most = kMaxThreads * ITEMS * 16 + room_of(kDistillMaxK) * kEntryBytes;
    constexpr int some[3] = {128, 512, kDistillMaxK};
    int dev = 0, log_s = 0;
    const int many = a.K > some[1] ? 2 : a.K > some[0] ? 1 : 0;
    while (1 << log_s < p.S) ++log_s;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(p.warps * 32 + 64);
    const size_t pieces = static_cast<size_t>(p.warps) * 32 * ITEMS * 16;
    cfg.dynamicSmemBytes = pieces + some[many] * kEntryBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(p.S);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    int clusters = dev < 64 ? resident[dev][log_s][p.warps][many].load(std::memory_order_acquire) : 0;
    if (clusters == 0) {
        if ((e = cudaFuncSetAttribute(distill_kernel<T, GRAD, ITEMS>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, most)) != cudaSuccess)
            return e;
        cfg.gridDim = dim3(static_cast<unsigned>(p.S));
        cfg.numAttrs = 1;
        if ((e = cudaOccupancyMaxActiveClusters(&clusters, distill_kernel<T, GRAD, ITEMS>, &cfg)) != cudaSuccess)
            return e;
        if (clusters < 1) clusters = 1;
        if (dev < 64) resident[dev][log_s][p.warps][many].store(clusters, std::memory_order_release);
    }
    const int64_t rows = a.B < clusters ? a.B : clusters;
    cfg.gridDim = dim3(static_cast<unsigned>(rows * p.S));
    cfg.dynamicSmemBytes = pieces + static_cast<size_t>(room_of(a.K)) * kEntryBytes;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, distill_kernel<T, GRAD, ITEMS>, a, p.seg, p.S, p.Q);
}

template <typename T, bool GRAD>
cudaError_t launch_as(const DistillArgs<T> &a, int num_sms, cudaStream_t stream)
{
    const Plan p = plan_of<T>(a.B, a.V, GRAD, num_sms);
    switch (p.items) {
    case 1: return launch_items<T, GRAD, 1>(a, p, stream);
    case 2: return launch_items<T, GRAD, 2>(a, p, stream);
    case 4: return launch_items<T, GRAD, 4>(a, p, stream);
    case 8: return launch_items<T, GRAD, 8>(a, p, stream);
    default:
        if constexpr (GRAD && Logit<T>::kVec * 16 <= kMaxBits) return launch_items<T, GRAD, 16>(a, p, stream);
        return cudaErrorInvalidValue;
    }
}

}  // namespace

template <typename T>
cudaError_t launch_distill(const DistillArgs<T> &a, int num_sms, cudaStream_t stream)
{
    return a.dz != nullptr ? launch_as<T, true>(a, num_sms, stream) : launch_as<T, false>(a, num_sms, stream);
}
template cudaError_t launch_distill<uint16_t>(const DistillArgs<uint16_t> &, int, cudaStream_t);
template cudaError_t launch_distill<float>(const DistillArgs<float> &, int, cudaStream_t);

}  // namespace mhc
