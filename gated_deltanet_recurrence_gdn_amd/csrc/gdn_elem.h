// gdn_elem.h -- typed element loads and stores shared by the kernels of the operators
// around the recurrence: every input type is widened exactly to fp32, outputs are fp32
// or bf16 (rounded to nearest even, once).
#pragma once

#include "gdn_common.h"
#include "gdn_launch.h"

namespace gdn {

template <int IO>
__device__ __forceinline__ float load1(const void *p, size_t i) {
    if constexpr (IO == IO_F32) {
        return static_cast<const float *>(p)[i];
    } else if constexpr (IO == IO_BF16) {
        return __uint_as_float((uint32_t) static_cast<const uint16_t *>(p)[i] << 16);
    } else {
        float f[4];
        fp8x4_to_f32(static_cast<const uint8_t *>(p)[i], f);
        return f[0];
    }
}

// Output element of the type that belongs to input type IO.
template <int IO>
__device__ __forceinline__ void store1(void *p, size_t i, float x) {
    if constexpr (IO == IO_F32)
        static_cast<float *>(p)[i] = x;
    else
        static_cast<uint16_t *>(p)[i] = (uint16_t)f32_to_bf16_bits(x);
}

}  // namespace gdn
