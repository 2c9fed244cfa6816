// Device helpers of the decoding operators' kernels.
#pragma once

#include "lowbit_device.h"

namespace lowbit {

// dma16 with 4 bytes a lane (at lds_wave_base + 4 * i).
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t rs, void* lds_wave_base, uint32_t voff, int soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)lds_wave_base, 4, voff, soff, 0, 0);
}

}  // namespace lowbit
