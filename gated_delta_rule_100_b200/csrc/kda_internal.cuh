// kda_internal.cuh -- host helpers of kda_api.cu that other files of the C
// boundary use: the current device's status word, the tensor-map encoder, the
// polls a bounded wait makes, and a device's SM count (all cached).
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace kda {
int host_status_word(uint32_t **out);
int host_encoder(PFN_cuTensorMapEncodeTiled_v12000 *fn);
uint64_t host_wait_polls();
int host_num_sms(int dev);

// Lets a kernel have `bytes` of dynamic shared memory, asking the runtime once a device.
template <class... A>
cudaError_t allow_smem(void (*kernel)(A...), int bytes) {
    // one word a signature would be shared by kernels of the same parameters: keep the kernels
    struct Entry { std::atomic<void *> kernel; std::atomic<unsigned long long> devices; };
    static Entry known[16];
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    for (Entry &x : known) {
        void *k = x.kernel.load();
        if (k == nullptr && !x.kernel.compare_exchange_strong(k, reinterpret_cast<void *>(kernel))) k = x.kernel.load();
        else if (k == nullptr) k = reinterpret_cast<void *>(kernel);
        if (k != reinterpret_cast<void *>(kernel)) continue;
        const unsigned long long bit = 1ull << (dev & 63);
        if (x.devices.load() & bit) return cudaSuccess;
        const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (r == cudaSuccess) x.devices.fetch_or(bit);
        return r;
    }
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}
}  // namespace kda
