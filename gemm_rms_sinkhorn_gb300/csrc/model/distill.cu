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
// A row is read once: a cluster of up to 8 blocks holds it in shared memory, each a
// segment.  A block copies its segment in, takes out the kept entries (they are summed
// apart and leave -inf behind), forms the largest value and the sum of the rest, and the
// blocks exchange those through distributed shared memory.  The gradient is then formed
// from the segment and written once; dz may be z.  Every block works out the K entries
// for itself.
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

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait()
{
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 16 bytes at `p`'s place in the shared memory of block `rank` of the cluster.
__device__ __forceinline__ float4 ld_cluster(const float4 *p, uint32_t rank)
{
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(p)), "r"(rank));
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

// ---- the logits' types: 16 bytes as fp32, and back
template <typename T>
struct Logit;
template <>
struct Logit<uint16_t> {
    static constexpr int kVec = 8;
    __device__ static float value(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
    __device__ static uint16_t from(float f) { return static_cast<uint16_t>(pack_bf16_rn(f, 0.f)); }
    __device__ static uint16_t tag(int k) { return static_cast<uint16_t>(k); }
    __device__ static int tag_of(uint16_t v) { return v; }
    __device__ static uint16_t lowest() { return 0xFF80u; }
    __device__ static void unpack(const uint4 &v, float (&f)[8]) { unpack8(v, f); }
    __device__ static uint4 pack(const float (&f)[8]) { return pack8(f); }
    __device__ static uint16_t load(const uint16_t *p) { return static_cast<uint16_t>(ptx::ld_dep(p)); }
};
template <>
struct Logit<float> {
    static constexpr int kVec = 4;
    __device__ static float value(float v) { return v; }
    __device__ static float from(float f) { return f; }
    __device__ static float tag(int k) { return __int_as_float(k); }
    __device__ static int tag_of(float v) { return __float_as_int(v); }
    __device__ static float lowest() { return -INFINITY; }
    __device__ static void unpack(const uint4 &v, float (&f)[4])
    {
        f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
    }
    __device__ static uint4 pack(const float (&f)[4])
    {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
    __device__ static float load(const float *p) { return ptx::ld_dep(p); }
};

// A sum of exp((v - m)·c), c > 0, kept with its largest v.  Nothing yet: (-inf, 0).
struct Peak {
    float m, s;
};
__device__ __forceinline__ Peak merge(Peak a, Peak b, float c2)
{
    const float m = fmaxf(a.m, b.m);
    if (m == -INFINITY) return {m, a.s + b.s};
    return {m, a.s * exp2_fast((a.m - m) * c2) + b.s * exp2_fast((b.m - m) * c2)};
}

struct Shared {
    float4 mine;               // (rest.m, rest.s, top.m, top.s) of this block, read by the cluster
    float4 all[kMaxCluster];
    float a[kWarps], b[kWarps], c[kWarps];
};

// Reductions over the block; every thread gets the result.  Between two that use the
// same array there has to be a barrier after the first one's last read: callers alternate.
__device__ __forceinline__ float block_sum(float v, float *red)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < kWarps ? red[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}
__device__ __forceinline__ float block_max(float v, float *red)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < kWarps ? red[threadIdx.x & 31] : -INFINITY;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

// -inf, where nothing or only -inf was seen, as a reference that -inf may be taken from.
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.f : m; }

template <typename T, bool GRAD>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillArgs<T> a, int seg, int S)
{
    using L = Logit<T>;
    constexpr int VEC = L::kVec;
    __shared__ Shared sh;
    extern __shared__ __align__(16) uint8_t dyn[];
    T *buf = reinterpret_cast<T *>(dyn);                                // [seg]
    float *lp = reinterpret_cast<float *>(dyn + static_cast<size_t>(seg) * sizeof(T));  // log p [K]
    float *zk = lp + a.K;                                               // the student's logit there
    int *idk = reinterpret_cast<int *>(zk + a.K);                       // -1: absent

    const int tid = threadIdx.x;
    const uint32_t rank = S > 1 ? cluster_rank() : 0;
    const int lo = static_cast<int>(rank) * seg;
    const int count = min(a.V - lo, seg) > 0 ? min(a.V - lo, seg) : 0;
    const int chunks = (count + VEC - 1) / VEC;
    const float c2 = a.inv_tau * kLog2e;
    const uint32_t buf_at = ptx::smem_u32(buf);
    bool waiting = false;  // for the cluster to have read `mine`

    ptx::pdl_wait();
    ptx::pdl_trigger();
    for (int64_t b = blockIdx.x / S; b < a.B; b += gridDim.x / S) {
        if (!in_range(1601, b, 1, a.B)) break;
        const T *row = a.z + b * a.ld + lo;
        for (int i = tid; i < chunks; i += kThreads)
            if (in_range(1602, lo + i * VEC, VEC, a.ld)) cp_async16(buf_at + i * 16, row + i * VEC);
        ptx::cp_async_commit();

        // the teacher's entries
        int some = 0;
        float tm = -INFINITY;
        for (int k = tid; k < a.K; k += kThreads) {
            const int64_t id = ptx::ld_dep(a.ids + b * a.K + k);
            const float t = ptx::ld_dep(a.t + b * a.K + k);
            const bool here = id >= 0 && id < a.V && t != -INFINITY;
            idk[k] = here ? static_cast<int>(id) : -1;
            lp[k] = t * a.inv_tau;
            if (!here) continue;
            some = 1;
            tm = fmaxf(tm, t * a.inv_tau);
            if (rank == 0) zk[k] = L::value(L::load(a.z + b * a.ld + id));
        }
        if (!__syncthreads_or(some)) {
            if (rank == 0 && tid == 0 && a.loss != nullptr) a.loss[b] = 0.f;
            if constexpr (GRAD) {
                T *out = a.dz + b * a.ld + lo;
                for (int i = tid; i < count; i += kThreads) out[i] = L::from(0.f);
            }
            ptx::cp_async_wait_all();
            __syncthreads();
            continue;
        }
        float base = 0.f, mass = 0.f;
        if (a.t_lse != nullptr) {
            base = ptx::ld_dep(a.t_lse + b);
            for (int k = tid; k < a.K; k += kThreads) {
                lp[k] -= base;
                if (idk[k] >= 0) mass += expf(lp[k]);
            }
            mass = block_sum(mass, sh.b);
        } else {
            tm = block_max(tm, sh.a);
            float s = 0.f;
            for (int k = tid; k < a.K; k += kThreads) {
                lp[k] -= tm;
                if (idk[k] >= 0) s += expf(lp[k]);
            }
            base = logf(block_sum(s, sh.b));
            for (int k = tid; k < a.K; k += kThreads) lp[k] -= base;
            mass = 1.f;
        }

        // the segment: what is past its end, and the kept entries, become -inf
        ptx::cp_async_wait_all();
        __syncthreads();
        if (tid < chunks * VEC - count) buf[count + tid] = L::lowest();
        for (int k = tid; k < a.K; k += kThreads) {
            const int j = idk[k] - lo;
            if (idk[k] >= 0 && j >= 0 && j < count) zk[k] = L::value(buf[j]);
        }
        __syncthreads();
        for (int k = tid; k < a.K; k += kThreads) {
            const int j = idk[k] - lo;
            if (idk[k] >= 0 && j >= 0 && j < count) buf[j] = L::tag(k);
        }
        __syncthreads();
        int twice = 0;  // whether an id comes more than once
        for (int k = tid; k < a.K; k += kThreads) {
            const int j = idk[k] - lo;
            if (idk[k] >= 0 && j >= 0 && j < count) twice |= L::tag_of(buf[j]) != k;
        }
        twice = __syncthreads_or(twice);
        Peak top = {-INFINITY, 0.f};
        for (int k = tid; k < a.K; k += kThreads) {
            const int j = idk[k] - lo;
            if (idk[k] < 0 || j < 0 || j >= count) continue;
            buf[j] = L::lowest();
            bool first = true;
            if (twice)
                for (int i = 0; i < k; ++i) first = first && idk[i] != idk[k];
            const float one = zk[k] == -INFINITY ? 0.f : zk[k] != zk[k] ? zk[k] : 1.f;
            if (first) top = merge(top, {zk[k], one}, c2);
        }
        __syncthreads();

        // the rest's largest value and sum
        float m = -INFINITY;
        const uint4 *chunk = reinterpret_cast<const uint4 *>(buf);
        for (int i = tid; i < chunks; i += kThreads) {
            float f[VEC];
            L::unpack(chunk[i], f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) m = fmaxf(m, f[e]);
        }
        m = block_max(m, sh.c);
        const float ref = reference(m);
        float s = 0.f;
        for (int i = tid; i < chunks; i += kThreads) {
            float f[VEC];
            L::unpack(chunk[i], f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) s += exp2_fast((f[e] - ref) * c2);
        }
        Peak rest = {m, block_sum(s, sh.a)};
        const float topm = block_max(top.m, sh.b);
        // sum of the kept entries, relative to their largest
        top.s = block_sum(topm == -INFINITY ? top.s : top.s * exp2_fast((top.m - topm) * c2), sh.c);
        top.m = topm;

        if (S > 1) {
            if (waiting) cluster_wait();
            if (tid == 0) sh.mine = make_float4(rest.m, rest.s, top.m, top.s);
            cluster_arrive();
            cluster_wait();
            if (tid < S) sh.all[tid] = ld_cluster(&sh.mine, tid);
            cluster_arrive();
            waiting = true;
            __syncthreads();
            rest = {-INFINITY, 0.f};
            top = {-INFINITY, 0.f};
            for (int r = 0; r < S; ++r) {
                const float4 v = sh.all[r];
                rest = merge(rest, {v.x, v.y}, c2);
                top = merge(top, {v.z, v.w}, c2);
            }
        }
        const Peak whole = merge(rest, top, c2);
        const float ln_s = logf(whole.s);
        const float p_rest = a.t_lse != nullptr && rest.s != 0.f ? fmaxf(1.f - mass, 0.f) : 0.f;

        if (rank == 0 && a.loss != nullptr) {
            float part = 0.f;
            for (int k = tid; k < a.K; k += kThreads) {
                if (idk[k] < 0) continue;
                const float p = expf(lp[k]);
                if (p != 0.f) part += p * (lp[k] - ((zk[k] - whole.m) * a.inv_tau - ln_s));
            }
            part = block_sum(part, sh.a);
            if (tid == 0) {
                if (p_rest > 0.f)
                    part += p_rest * (logf(p_rest) - ((rest.m - whole.m) * a.inv_tau + logf(rest.s) - ln_s));
                a.loss[b] = part;
            }
        }
        if constexpr (GRAD) {
            const float w = ptx::ld_dep(a.dloss + b) * a.inv_tau, all = mass + p_rest;
            // q_rest·(M - p_rest/q_rest) = M·q_rest - p_rest, shared out by exp over the rest's sum
            const float q_rest = rest.s == 0.f ? 0.f : rest.s * exp2_fast((rest.m - whole.m) * c2) / whole.s;
            const float scale = rest.s != 0.f ? w * (all * q_rest - p_rest) / rest.s
                                              : whole.s != 0.f ? 0.f : NAN;
            const float at = reference(rest.m);
            T *out = a.dz + b * a.ld + lo;
            for (int i = tid; i < chunks; i += kThreads) {
                float f[VEC];
                L::unpack(chunk[i], f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) f[e] = exp2_fast((f[e] - at) * c2) * scale;
                if ((i + 1) * VEC <= count) {
                    if (in_range(1603, lo + i * VEC, VEC, a.ld)) ptx::st_stream_v4(out + i * VEC, L::pack(f));
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        if (i * VEC + e < count) out[i * VEC + e] = L::from(f[e]);
                }
            }
            __syncthreads();  // the kept entries' places hold 0 until here
            for (int k = tid; k < a.K; k += kThreads) {
                const int j = idk[k] - lo;
                if (idk[k] < 0 || j < 0 || j >= count) continue;
                float p = expf(lp[k]);
                if (twice) {
                    p = 0.f;
                    for (int i = 0; i < a.K; ++i)
                        if (idk[i] == idk[k]) p += expf(lp[i]);
                }
                const float q = exp2_fast((zk[k] - whole.m) * c2) / whole.s;
                out[j] = L::from(w * (all * q - p));
            }
        }
        __syncthreads();  // the entries and the segment are no longer read
    }
    if (waiting) cluster_wait();
}

// Blocks a row: a segment of at most kSegBytes; and more where rows are so few that SMs
// would be idle.
constexpr int kSegBytes = 72 << 10;
constexpr int kMinSeg = 4096;

template <typename T, bool GRAD>
cudaError_t launch_as(const DistillArgs<T> &a, int num_sms, cudaStream_t stream)
{
    int S = 1;
    const auto seg_of = [&](int s) { return ((a.V + s - 1) / s + 7) / 8 * 8; };
    while (S < kMaxCluster && (static_cast<int64_t>(seg_of(S)) * sizeof(T) > kSegBytes ||
                               (a.B * S < num_sms && seg_of(S) > kMinSeg)))
        S *= 2;
    const int seg = seg_of(S);
    const size_t smem = static_cast<size_t>(seg) * sizeof(T) + static_cast<size_t>(a.K) * 12;
    static std::atomic<uint64_t> done{0};
    constexpr int most = static_cast<int>(kDistillMaxV / kMaxCluster * 4 + kDistillMaxK * 12);
    cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(distill_kernel<T, GRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    });
    if (e != cudaSuccess) return e;
    const int64_t rows = a.B < (int64_t{1} << 24) ? a.B : int64_t{1} << 24;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows * S));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(S);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = S > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, distill_kernel<T, GRAD>, a, seg, S);
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
