// kda_internal.cuh -- host helpers of kda_api.cu that other files of the C
// boundary use: the current device's status word, the tensor-map encoder, the
// polls a bounded wait makes, and a device's SM count (all cached).
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <stdint.h>

namespace kda {
int host_status_word(uint32_t **out);
int host_encoder(PFN_cuTensorMapEncodeTiled_v12000 *fn);
uint64_t host_wait_polls();
int host_num_sms(int dev);
}  // namespace kda
