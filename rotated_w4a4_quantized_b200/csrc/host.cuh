// host.cuh -- host-side checks shared by the group-scaled and the cache
// library: device set-up, pointer look-ups and alignment.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <initializer_list>
#include <mutex>

#include "../../include/convrot.h"

namespace host {

// Internal linkage: every library has its own state.  (An inline variable
// would be one object for all libraries of the process, and the set-up of the
// first would pass for that of the others.)
namespace {

constexpr int kMaxDevices = 64;

// `ready` is stored (release) only after every other field is written and
// read (acquire) before any of them; the first set-up on each device runs
// under the lock.  A CUDA call that failed (for want of memory while the
// kernels load, say) is tried again by the next call: only what cannot change,
// success and another kind of device, is kept.
struct DeviceState {
    std::atomic<bool> ready{false};
    convrot_status status = CONVROT_OK;
    int num_sms = 0;
};

DeviceState g_dev[kMaxDevices];
std::mutex g_mu;

// The current device's state; `kernels` opts the library's kernels into
// their shared memory (true when all of them could be).
template <class F>
convrot_status device_setup(int *dev_out, F kernels) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return CONVROT_ERR_CUDA;
    }
    *dev_out = dev;
    DeviceState &st = g_dev[dev];
    if (st.ready.load(std::memory_order_acquire)) return st.status;
    std::lock_guard<std::mutex> lock(g_mu);
    if (st.ready.load(std::memory_order_relaxed)) return st.status;
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        st.status = CONVROT_ERR_CUDA;
    else if (major != 10 || minor != 0)
        st.status = CONVROT_ERR_UNSUPPORTED;
    else
        st.status = kernels() ? CONVROT_OK : CONVROT_ERR_CUDA;
    if (st.status == CONVROT_ERR_CUDA) {
        cudaGetLastError();   // reported here: no later launch finds it
        return st.status;
    }
    st.num_sms = sms;
    st.ready.store(true, std::memory_order_release);
    return st.status;
}

inline bool aligned(unsigned bytes, std::initializer_list<const void *> ptrs) {
    for (const void *p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) return false;
    return true;
}

inline bool aligned16(std::initializer_list<const void *> ptrs) { return aligned(16, ptrs); }

// CONVROT_OK when every non-null pointer is device (or managed) memory of
// device `dev`: run before any launch, so a bad pointer never reaches a
// kernel.
inline convrot_status check_device_ptrs(int dev, std::initializer_list<const void *> ptrs) {
    for (const void *p : ptrs) {
        if (!p) continue;
        cudaPointerAttributes a;
        if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
            cudaGetLastError();   // clear the look-up error (it is not sticky)
            return CONVROT_ERR_NOT_DEVICE;
        }
        if ((a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged) || a.device != dev)
            return CONVROT_ERR_NOT_DEVICE;
    }
    return CONVROT_OK;
}

struct Span {
    const void *p;
    int64_t bytes;
};

// Whether a buffer that a call writes shares bytes with another that it writes
// or reads.
inline bool overlap(std::initializer_list<Span> written, std::initializer_list<Span> read) {
    auto meet = [](const Span &a, const Span &b) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
        return a.p && b.p && a.bytes > 0 && b.bytes > 0 && x < y + static_cast<uint64_t>(b.bytes) && y < x + static_cast<uint64_t>(a.bytes);
    };
    for (const Span *a = written.begin(); a != written.end(); ++a) {
        for (const Span *b = a + 1; b != written.end(); ++b)
            if (meet(*a, *b)) return true;
        for (const Span &b : read)
            if (meet(*a, b)) return true;
    }
    return false;
}

inline size_t round256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// A launch that may start while the previous kernel of the stream finishes
// (programmatic dependent launch); the kernel waits in griddepcontrol.wait.
template <class K, class... A>
convrot_status launch_dependent(K *kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                                A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess) return CONVROT_OK;
    cudaGetLastError();       // as above
    return CONVROT_ERR_CUDA;
}

}  // namespace
}  // namespace host
