// The device set-up and launches of csrc/host.cuh against a fake of the CUDA
// runtime (no GPU): what is kept of a failure, and whether its error is left
// for a later call to find.  Prints "ok", or the line of the first failure.
#include <cuda_runtime.h>

#include <cstdio>

namespace fake {
cudaError_t attribute = cudaSuccess, launch = cudaSuccess, last = cudaSuccess;
int major = 10, attribute_calls = 0;
cudaError_t result(cudaError_t e) {
    if (e != cudaSuccess) last = e;
    return e;
}
cudaError_t GetDevice(int *dev) { return *dev = 3, cudaSuccess; }
cudaError_t DeviceGetAttribute(int *v, cudaDeviceAttr a, int) {
    ++attribute_calls;
    *v = a == cudaDevAttrComputeCapabilityMajor ? major : a == cudaDevAttrComputeCapabilityMinor ? 0 : 148;
    return result(attribute);
}
cudaError_t GetLastError() {
    const cudaError_t e = last;
    last = cudaSuccess;
    return e;
}
template <class K, class... A>
cudaError_t LaunchKernelEx(const cudaLaunchConfig_t *, K *, A...) { return result(launch); }
}  // namespace fake

#define cudaGetDevice fake::GetDevice
#define cudaDeviceGetAttribute fake::DeviceGetAttribute
#define cudaGetLastError fake::GetLastError
#define cudaLaunchKernelEx fake::LaunchKernelEx
#define cudaPointerGetAttributes(a, p) cudaSuccess
#include "../rotated_w4a4_quantized_b200/csrc/host.cuh"

static void kernel(int) {}

#define CHECK(c) \
    if (!(c)) return std::printf("line %d: %s\n", __LINE__, #c), 1

int main() {
    int dev = -1, kernels = 0;
    bool load = false;
    auto setup = [&] {
        return host::device_setup(&dev, [&] {
            ++kernels;
            if (!load) fake::result(cudaErrorMemoryAllocation);
            return load;
        });
    };
    fake::attribute = cudaErrorInitializationError;
    CHECK(setup() == CONVROT_ERR_CUDA && kernels == 0);
    CHECK(fake::last == cudaSuccess);
    fake::attribute = cudaSuccess;
    CHECK(setup() == CONVROT_ERR_CUDA && kernels == 1);   // tried again: now the kernels do not load
    CHECK(fake::last == cudaSuccess);
    load = true;
    CHECK(setup() == CONVROT_OK && kernels == 2 && dev == 3 && host::g_dev[3].num_sms == 148);
    const int calls = fake::attribute_calls;
    CHECK(setup() == CONVROT_OK && kernels == 2 && fake::attribute_calls == calls);   // success is kept
    fake::launch = cudaErrorLaunchOutOfResources;
    CHECK(host::launch_dependent(&kernel, dim3(1), dim3(1), 0, nullptr, 5) == CONVROT_ERR_CUDA);
    CHECK(fake::last == cudaSuccess);
    fake::launch = cudaSuccess;
    CHECK(host::launch_dependent(&kernel, dim3(1), dim3(1), 0, nullptr, 5) == CONVROT_OK);
    // another kind of device is kept too
    host::g_dev[3].ready = false;
    fake::major = 9;
    CHECK(setup() == CONVROT_ERR_UNSUPPORTED);
    const int once = fake::attribute_calls;
    CHECK(setup() == CONVROT_ERR_UNSUPPORTED && fake::attribute_calls == once);
    std::printf("ok\n");
    return 0;
}
