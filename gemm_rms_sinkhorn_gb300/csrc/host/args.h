// Argument checks shared by the C ABI's source files (api.cu, train/train_api.cu,
// model/model_api.cu):
// shapes, pointers, overlaps and where the memory lies.  Host code only.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mhc.h"
#include "mhc_internal.h"

namespace mhc {

struct Buf {
    const void *p;
    size_t bytes;
};

inline bool overlaps(const Buf &a, const Buf &b)
{
    if (a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Shape rules shared by every call.  Returns MHC_OK or the error.
inline int check_shape(int64_t B, int n, int64_t C, bool needs_c)
{
    if (B < 0) return MHC_ERR_INVALID;
    if (n < 1 || n > 8) return MHC_ERR_UNSUPPORTED;
    if (needs_c) {
        if (C < 8 || C % 8 != 0) return MHC_ERR_UNSUPPORTED;
        // K = n*C is addressed with 32-bit TMA coordinates and int kernel arguments
        if (static_cast<int64_t>(n) * C > (int64_t{1} << 30)) return MHC_ERR_UNSUPPORTED;
    }
    // token rows are TMA coordinates, 32-bit signed
    if (B >= (int64_t{1} << 31)) return MHC_ERR_UNSUPPORTED;
    return MHC_OK;
}

inline int check_ptrs(const Buf *bufs, int count)
{
    for (int i = 0; i < count; ++i)
        if (bufs[i].p == nullptr) return MHC_ERR_INVALID;
    for (int i = 0; i < count; ++i)
        if (!aligned16(bufs[i].p)) return MHC_ERR_ALIGN;
    return MHC_OK;
}

// Outputs must not overlap inputs or each other.  `alias_ok` names one
// (output, input) pair that may be exactly equal.
inline int check_overlap(const Buf *outs, int n_out, const Buf *ins, int n_in, const void *alias_out,
                  const void *alias_in)
{
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j) {
            if (outs[i].p == alias_out && ins[j].p == alias_in && alias_out == alias_in &&
                outs[i].bytes == ins[j].bytes)
                continue;
            if (overlaps(outs[i], ins[j])) return MHC_ERR_INVALID;
        }
        for (int j = i + 1; j < n_out; ++j)
            if (overlaps(outs[i], outs[j])) return MHC_ERR_INVALID;
    }
    return MHC_OK;
}

// Whether the pointer checks of the device-memory entry points run (on unless a
// test turns them off to time their cost).
inline std::atomic<int> g_memory_checks{1};

// Every buffer must be device memory of the current device (cudaMalloc,
// stream-ordered pools or mapped VMM ranges): a host pointer, managed memory
// or another GPU's memory reached over peer access is MHC_ERR_INVALID, before
// anything is launched.  The kernels' TMA descriptors and stores assume local
// device memory.
inline int check_on_device(const Buf *bufs, int count, const DeviceInfo &info)
{
    if (!g_memory_checks.load(std::memory_order_relaxed)) return MHC_OK;
    for (int i = 0; i < count; ++i) {
        cudaPointerAttributes a{};
        if (cudaPointerGetAttributes(&a, bufs[i].p) != cudaSuccess) {
            cudaGetLastError();  // not sticky; clear it
            return MHC_ERR_INVALID;
        }
        if (a.type != cudaMemoryTypeDevice || a.device != info.device) return MHC_ERR_INVALID;
    }
    return MHC_OK;
}

// Every buffer must be host memory (page-locked or pageable), as the runtime
// records it: device or managed memory is MHC_ERR_INVALID.
inline int check_on_host(const Buf *bufs, int count)
{
    for (int i = 0; i < count; ++i) {
        cudaPointerAttributes a{};
        if (cudaPointerGetAttributes(&a, bufs[i].p) != cudaSuccess) {
            cudaGetLastError();  // not sticky; clear it
            return MHC_ERR_INVALID;
        }
        if (a.type != cudaMemoryTypeHost && a.type != cudaMemoryTypeUnregistered)
            return MHC_ERR_INVALID;
    }
    return MHC_OK;
}

inline int check_device(DeviceInfo *info)
{
    if (current_device_info(info) != cudaSuccess) return MHC_ERR_CUDA;
    if (info->cc_major != 10 || info->cc_minor != 3) return MHC_ERR_UNSUPPORTED;
    return MHC_OK;
}

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? MHC_OK : MHC_ERR_CUDA; }

inline size_t bf16_bytes(int64_t count) { return static_cast<size_t>(count) * 2; }
inline size_t f32_bytes(int64_t count) { return static_cast<size_t>(count) * 4; }

#define MHC_TRY(expr)                   \
    do {                                \
        const int st_ = (expr);         \
        if (st_ != MHC_OK) return st_;  \
    } while (0)

// The checks that follow the shape rules, in the order of the other calls:
// pointers, overlaps, device, memory.  `ws` (may be NULL): the workspace, which
// needs `need(num_sms)` bytes.
template <typename Need>
inline int check_buffers(const Buf *ins, int n_in, Buf *outs, int n_out, const void *alias_out,
                         const void *alias_in, Buf *ws, Need need, DeviceInfo *info)
{
    MHC_TRY(check_ptrs(ins, n_in));
    MHC_TRY(check_ptrs(outs, n_out));
    MHC_TRY(check_overlap(outs, n_out, ins, n_in, alias_out, alias_in));
    MHC_TRY(check_device(info));
    MHC_TRY(check_on_device(ins, n_in, *info));
    MHC_TRY(check_on_device(outs, n_out, *info));
    if (ws != nullptr) {
        const size_t bytes = need(info->num_sms);
        if (ws->p == nullptr || ws->bytes < bytes) return MHC_ERR_WORKSPACE;
        const Buf w = {ws->p, bytes};
        MHC_TRY(check_ptrs(&w, 1));
        MHC_TRY(check_overlap(&w, 1, ins, n_in, nullptr, nullptr));
        MHC_TRY(check_overlap(&w, 1, outs, n_out, nullptr, nullptr));
        MHC_TRY(check_on_device(&w, 1, *info));
    }
    return MHC_OK;
}

inline int check_buffers(const Buf *ins, int n_in, Buf *outs, int n_out, const void *alias_out,
                         const void *alias_in, DeviceInfo *info)
{
    return check_buffers(ins, n_in, outs, n_out, alias_out, alias_in, nullptr,
                         [](int) { return size_t{0}; }, info);
}

inline cudaStream_t cu(mhc_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Gradients of weights that no token touches: zero unless they are added to.
inline int zero_grads(const Buf *outs, int count, int accumulate, mhc_stream_t stream)
{
    if (accumulate) return MHC_OK;
    MHC_TRY(check_ptrs(outs, count));
    DeviceInfo info;
    MHC_TRY(check_device(&info));
    MHC_TRY(check_on_device(outs, count, info));
    for (int i = 0; i < count; ++i)
        if (cudaMemsetAsync(const_cast<void *>(outs[i].p), 0, outs[i].bytes, cu(stream)) !=
            cudaSuccess)
            return MHC_ERR_CUDA;
    return MHC_OK;
}

}  // namespace mhc
