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

// The output type that belongs to an input type.
template <int IO>
constexpr int OutIo = IO == IO_F32 ? IO_F32 : IO_BF16;

// Address of element i.
template <int IO>
__device__ __forceinline__ const void *at(const void *p, size_t i) {
    return static_cast<const char *>(p) + i * io_in_bytes(IO);
}
template <int IO>
__device__ __forceinline__ void *at(void *p, size_t i) {
    return static_cast<char *>(p) + i * io_in_bytes(IO);
}

// Outputs leave with the non-temporal hint: no kernel here reads them again, and without it
// they push out what is read (2 x 32,760 tokens of 64 heads turned: 368 us against 389; the
// norm's training step on two clips: 107 against 116, its first pass over x alone 15 against
// 26).  A kernel behind that reads them finds them no slower (a recurrence and the norm of its
// outputs, 6 to 537 MB: 3% less to 10% less time, 3% more at 77 MB).
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
template <typename T>
__device__ __forceinline__ void stream_out(T *p, T x) {
    __builtin_nontemporal_store(x, p);
}

// The same hint for inputs that a call reads once (rows of 32 groups normalised: 201 us against
// 209).  Where a second pass reads them again it costs more than it gives (the norm's training
// step on two clips: 115 us against 107).
template <typename T>
__device__ __forceinline__ T stream_in(const T *p) {
    return __builtin_nontemporal_load(p);
}

// Eight neighbouring elements, as they lie in memory; i counts vectors.  load_once: read by no
// later pass of the call.
template <int IO>
struct Vec;
template <>
struct Vec<IO_F32> {
    float4 r[2];
    __device__ __forceinline__ void load(const void *p, size_t i) {
        r[0] = static_cast<const float4 *>(p)[2 * i];
        r[1] = static_cast<const float4 *>(p)[2 * i + 1];
    }
    __device__ __forceinline__ void load_once(const void *p, size_t i) {
        const f32x4_t a = stream_in(static_cast<const f32x4_t *>(p) + 2 * i), b = stream_in(static_cast<const f32x4_t *>(p) + 2 * i + 1);
        r[0] = make_float4(a[0], a[1], a[2], a[3]);
        r[1] = make_float4(b[0], b[1], b[2], b[3]);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = r[0].x; f[1] = r[0].y; f[2] = r[0].z; f[3] = r[0].w;
        f[4] = r[1].x; f[5] = r[1].y; f[6] = r[1].z; f[7] = r[1].w;
    }
    static __device__ __forceinline__ void store(void *p, size_t i, const float (&f)[8]) {
        const f32x4_t a = {f[0], f[1], f[2], f[3]}, b = {f[4], f[5], f[6], f[7]};
        stream_out(static_cast<f32x4_t *>(p) + 2 * i, a);
        stream_out(static_cast<f32x4_t *>(p) + 2 * i + 1, b);
    }
};
template <>
struct Vec<IO_BF16> {
    uint4 r;
    __device__ __forceinline__ void load(const void *p, size_t i) { r = static_cast<const uint4 *>(p)[i]; }
    __device__ __forceinline__ void load_once(const void *p, size_t i) {
        const u32x4_t v = stream_in(static_cast<const u32x4_t *>(p) + i);
        r = make_uint4(v[0], v[1], v[2], v[3]);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = bf16_lo(r.x); f[1] = bf16_hi(r.x); f[2] = bf16_lo(r.y); f[3] = bf16_hi(r.y);
        f[4] = bf16_lo(r.z); f[5] = bf16_hi(r.z); f[6] = bf16_lo(r.w); f[7] = bf16_hi(r.w);
    }
    static __device__ __forceinline__ void store(void *p, size_t i, const float (&f)[8]) {
        const u32x4_t v = {pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
        stream_out(static_cast<u32x4_t *>(p) + i, v);
    }
};
template <>
struct Vec<IO_FP8> {
    uint2 r;
    __device__ __forceinline__ void load(const void *p, size_t i) { r = static_cast<const uint2 *>(p)[i]; }
    __device__ __forceinline__ void load_once(const void *p, size_t i) {
        const u32x2_t v = stream_in(static_cast<const u32x2_t *>(p) + i);
        r = make_uint2(v[0], v[1]);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        fp8x4_to_f32(r.x, f);
        fp8x4_to_f32(r.y, f + 4);
    }
};
template <int IO>
using OutVec = Vec<OutIo<IO>>;

}  // namespace gdn
