// gdn_rotary.hip -- rotary positions over three axes (include/gdn.h, gdn_rotary).
//
// Bound by HBM: six flops per pair read and written.  Pair j of every head of a token is
// turned by the same angle, so a block takes TOK tokens at a time, forms their cosines and
// sines once (frequency and angle in 64 bits, the angle reduced to a fraction of a turn before
// the fp32 sine) into LDS and turns all heads with them.
//  * pairs (2i, 2i + 1): a lane takes eight neighbouring elements (16 bytes of bf16), four
//    whole pairs.
//  * halves: a lane takes W neighbouring elements of a section's first half and the W of the
//    second half that belong to them; W is the largest of 8, 4, 2, 1 that divides every half.
// A pair is read and written by one lane, so out may be x.
#include "gdn_elem.h"
#include "gdn_layer.h"

#include <algorithm>

namespace gdn {
namespace {

constexpr int THREADS = 256;

// The angle of pair j of token t of batch element b, in turns, less whole turns.
__device__ __forceinline__ float part_turn(const RotaryArgs &a, unsigned b, long long t, int j) {
    int axis = 0;
    if (2 * j >= a.dim[0]) {
        j -= a.dim[0] / 2;
        axis = 1;
        if (2 * j >= a.dim[1]) {
            j -= a.dim[1] / 2;
            axis = 2;
        }
    }
    long long pos;
    if (a.positions) {
        pos = a.positions[b * a.pos_bs + 3 * t + axis];
    } else {
        const long long n = a.first_token + t, area = (long long)a.height * a.width;
        if (((n | area) >> 32) == 0) {  // a 64-bit division is some hundred instructions
            const unsigned m = (unsigned)n;
            pos = axis == 0 ? m / (unsigned)area : axis == 1 ? m / (unsigned)a.width % (unsigned)a.height : m % (unsigned)a.width;
        } else {
            pos = axis == 0 ? n / area : axis == 1 ? n / a.width % a.height : n % a.width;
        }
    }
    const double turns = (double)pos * (exp2(-2.0 * j / a.dim[axis] * a.log2_theta) * 0.15915494309189533577);  // 1 / 2 pi
    return (float)(turns - rint(turns));
}

__device__ __forceinline__ float2 turn(float2 x, float2 cs) {
    return make_float2(x.x * cs.x - x.y * cs.y, x.x * cs.y + x.y * cs.x);
}

// W neighbouring elements from element i on (i a multiple of W; a row starts at 16 bytes).
template <int IO, int W>
__device__ __forceinline__ void load_part(const void *row, size_t i, float (&f)[W]) {
    if constexpr (W == 8) {
        Vec<IO> x;
        x.load(row, i / 8);
        x.get(f);
    } else if constexpr (W == 1) {
        f[0] = load1<IO>(row, i);
    } else if constexpr (IO == IO_F32) {
        typedef float part __attribute__((ext_vector_type(W)));
        const part x = *reinterpret_cast<const part *>(static_cast<const float *>(row) + i);
#pragma unroll
        for (int k = 0; k < W; ++k) f[k] = x[k];
    } else if constexpr (IO == IO_BF16) {
        typedef uint16_t part __attribute__((ext_vector_type(W)));
        const part x = *reinterpret_cast<const part *>(static_cast<const uint16_t *>(row) + i);
#pragma unroll
        for (int k = 0; k < W; ++k) f[k] = __uint_as_float((uint32_t)x[k] << 16);
    } else {
        float g[4];
        uint32_t x = 0;
        __builtin_memcpy(&x, static_cast<const char *>(row) + i, W);
        fp8x4_to_f32(x, g);
#pragma unroll
        for (int k = 0; k < W; ++k) f[k] = g[k];
    }
}
template <int IO, int W>
__device__ __forceinline__ void store_part(void *row, size_t i, const float (&f)[W]) {
    if constexpr (W == 8) {
        OutVec<IO>::store(row, i / 8, f);
    } else if constexpr (W == 1) {
        store1<IO>(row, i, f[0]);
    } else if constexpr (IO == IO_F32) {
        typedef float part __attribute__((ext_vector_type(W)));
        part x;
#pragma unroll
        for (int k = 0; k < W; ++k) x[k] = f[k];
        *reinterpret_cast<part *>(static_cast<float *>(row) + i) = x;
    } else {
        typedef uint32_t part __attribute__((ext_vector_type(W / 2)));
        part x;
#pragma unroll
        for (int k = 0; k < W / 2; ++k) x[k] = pack_bf16x2(f[2 * k], f[2 * k + 1]);
        *reinterpret_cast<part *>(static_cast<uint16_t *>(row) + i) = x;
    }
}

// W = 0: pairs (2i, 2i + 1); else halves, W elements at a time.
template <int IO, int W, int TOK>
__global__ __launch_bounds__(THREADS) void rotary_kernel(RotaryArgs a) {
    __shared__ float2 cs[TOK][ROTARY_MAX_PAIRS];
    const unsigned rows = (unsigned)(a.B * a.T), T = (unsigned)a.T;
    const float sign = a.inverse ? -1.0f : 1.0f;
    for (unsigned row0 = blockIdx.x * TOK; row0 < rows; row0 += gridDim.x * TOK) {
        const int tokens = rows - row0 < TOK ? rows - row0 : TOK;
        for (int e = threadIdx.x; e < tokens * a.pairs; e += THREADS) {
            const int k = TOK == 1 ? 0 : e / a.pairs, j = e - k * a.pairs;
            float s, c;
            sincospif(2.0f * part_turn(a, (row0 + k) / T, (row0 + k) % T, j), &s, &c);
            cs[k][j] = make_float2(c, sign * s);
        }
        __syncthreads();
        for (int k = 0; k < tokens; ++k) {
            const unsigned b = (row0 + k) / T, t = (row0 + k) % T;
            const void *px = at<IO>(a.x, (size_t)b * a.x_bs + (size_t)t * a.x_ts);
            void *po = at<OutIo<IO>>(a.out, (size_t)b * a.out_bs + (size_t)t * a.out_ts);
            if constexpr (W == 0) {
                const int V = a.d / 8;
                for (int e = threadIdx.x; e < a.H * V; e += THREADS) {
                    Vec<IO> x;
                    float f[8];
                    x.load(px, e);
                    x.get(f);
                    const int j0 = e % V * 4;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (j0 + i < a.pairs) {
                            const float2 y = turn(make_float2(f[2 * i], f[2 * i + 1]), cs[k][j0 + i]);
                            f[2 * i] = y.x;
                            f[2 * i + 1] = y.y;
                        }
                    OutVec<IO>::store(po, e, f);
                }
            } else {
                // a head's parts: its pairs, W at a time, then what passes through
                const int P = a.pairs / W, per = P + (a.d - 2 * a.pairs) / W;
                for (int e = threadIdx.x; e < a.H * per; e += THREADS) {
                    const int h = e / per, p = e - h * per, j = p * W;
                    const size_t head = (size_t)h * a.d;
                    float f[W];
                    if (p < P) {
                        // section starts 2 `before` into the head, pair j is its number j - before
                        const int d0 = a.dim[0] / 2, d1 = a.dim[1] / 2;
                        const int before = j < d0 ? 0 : j < d0 + d1 ? d0 : d0 + d1;
                        const int half = j < d0 ? d0 : j < d0 + d1 ? d1 : a.dim[2] / 2;
                        const size_t i0 = head + before + j, i1 = i0 + half;
                        float g[W];
                        load_part<IO, W>(px, i0, f);
                        load_part<IO, W>(px, i1, g);
#pragma unroll
                        for (int i = 0; i < W; ++i) {
                            const float2 z = turn(make_float2(f[i], g[i]), cs[k][j + i]);
                            f[i] = z.x;
                            g[i] = z.y;
                        }
                        store_part<IO, W>(po, i0, f);
                        store_part<IO, W>(po, i1, g);
                    } else {
                        const size_t i = head + 2 * a.pairs + (p - P) * W;
                        load_part<IO, W>(px, i, f);
                        store_part<IO, W>(po, i, f);
                    }
                }
            }
        }
        __syncthreads();  // the angles are read above and written for the next tokens
    }
}

template <int IO, int W>
hipError_t launch(const RotaryArgs &a, hipStream_t s) {
    // Four tokens share a block's passes over the angles and its barriers; one each where that
    // would leave CUs idle (rows below 4 blocks of 4 tokens a CU).
    const long long rows = a.B * a.T;
    if (rows >= 4096)
        rotary_kernel<IO, W, 4><<<dim3((unsigned)std::min<long long>((rows + 3) / 4, 1 << 20)), dim3(THREADS), 0, s>>>(a);
    else
        rotary_kernel<IO, W, 1><<<dim3((unsigned)rows), dim3(THREADS), 0, s>>>(a);
    return hipGetLastError();
}

template <int IO>
hipError_t launch(const RotaryArgs &a, hipStream_t s) {
    if (!a.halves) return launch<IO, 0>(a, s);
    const int all = a.dim[0] / 2 | a.dim[1] / 2 | a.dim[2] / 2;
    return all % 8 == 0 ? launch<IO, 8>(a, s) : all % 4 == 0 ? launch<IO, 4>(a, s) : all % 2 == 0 ? launch<IO, 2>(a, s)
                                                                                        : launch<IO, 1>(a, s);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs &a, hipStream_t s) {
    return a.io == IO_F32 ? launch<IO_F32>(a, s) : a.io == IO_BF16 ? launch<IO_BF16>(a, s) : launch<IO_FP8>(a, s);
}

}  // namespace gdn
