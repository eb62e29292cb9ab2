// gdn_rotary.hip -- rotary positions over three axes (include/gdn.h, gdn_rotary).
//
// Bound by HBM: six flops per pair read and written.  Pair j of every head of a token is
// turned by the same angle, so a block takes TOK tokens at a time, forms their cosines and
// sines once (angle in 64 bits, reduced to a fraction of a turn before the fp32 sine) into
// LDS and turns all heads with them, eight neighbouring elements (16 bytes of bf16) a lane.
//  * pairs (2i, 2i + 1): a vector holds four whole pairs.
//  * halves, sections of whole vectors (every section a multiple of 16): a lane turns vector
//    i of a section's first half with vector i of its second.
//  * other halves: pairs lie anywhere, so a lane takes one pair after another; its two-byte
//    accesses stay within lines that neighbouring lanes use.
// A pair is read and written by one lane, so out may be x.
#include "gdn_elem.h"
#include "gdn_layer.h"

#include <algorithm>

namespace gdn {
namespace {

constexpr int THREADS = 256;
constexpr int TOK = 4;  // tokens whose angles a block forms together

// Position of token t of batch element b on an axis.
__device__ __forceinline__ long long position(const RotaryArgs &a, long long b, long long t, int axis) {
    if (a.positions) return a.positions[b * a.pos_bs + 3 * t + axis];
    const long long n = a.first_token + t;
    return axis == 0 ? n / ((long long)a.height * a.width) : axis == 1 ? n / a.width % a.height : n % a.width;
}

__device__ __forceinline__ float2 turn(float2 x, float2 cs) {
    return make_float2(x.x * cs.x - x.y * cs.y, x.x * cs.y + x.y * cs.x);
}

enum Layout { NEIGHBOURS, WHOLE_HALVES, ANY_HALVES };

template <int IO, int LAYOUT>
__global__ __launch_bounds__(THREADS) void rotary_kernel(RotaryArgs a) {
    __shared__ float2 cs[TOK][ROTARY_MAX_PAIRS];
    const long long rows = a.B * a.T;
    const int V = a.d / 8, turned = 2 * a.pairs;
    const float sign = a.inverse ? -1.0f : 1.0f;
    for (long long row0 = (long long)blockIdx.x * TOK; row0 < rows; row0 += (long long)gridDim.x * TOK) {
        const int tokens = rows - row0 < TOK ? (int)(rows - row0) : TOK;
        for (int e = threadIdx.x; e < tokens * a.pairs; e += THREADS) {
            const int k = e / a.pairs, j = e % a.pairs;
            const int axis = 2 * j < a.dim[0] ? 0 : 2 * j < a.dim[0] + a.dim[1] ? 1 : 2;
            const long long b = (row0 + k) / a.T, t = (row0 + k) % a.T;
            const double turns = (double)position(a, b, t, axis) * a.turns[j];
            float s, c;
            sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
            cs[k][j] = make_float2(c, sign * s);
        }
        __syncthreads();
        for (int k = 0; k < tokens; ++k) {
            const long long b = (row0 + k) / a.T, t = (row0 + k) % a.T;
            const size_t xr = (size_t)b * a.x_bs + (size_t)t * a.x_ts, orow = (size_t)b * a.out_bs + (size_t)t * a.out_ts;
            if constexpr (LAYOUT == NEIGHBOURS) {
                const void *px = at<IO>(a.x, xr);
                void *po = at<OutIo<IO>>(a.out, orow);
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
            } else if constexpr (LAYOUT == WHOLE_HALVES) {
                const void *px = at<IO>(a.x, xr);
                void *po = at<OutIo<IO>>(a.out, orow);
                const int W = a.pairs / 8, rest = V - 2 * W;  // vector pairs, and vectors that pass through
                for (int e = threadIdx.x; e < a.H * W; e += THREADS) {
                    const int h = e / W, j = e % W * 8;
                    const int axis = 2 * j < a.dim[0] ? 0 : 2 * j < a.dim[0] + a.dim[1] ? 1 : 2;
                    const int before = axis == 0 ? 0 : axis == 1 ? a.dim[0] : a.dim[0] + a.dim[1];
                    // section start + place in its half, in vectors
                    const int v0 = h * V + (before + j - before / 2) / 8, v1 = v0 + a.dim[axis] / 16;
                    Vec<IO> x, y;
                    float f[8], g[8];
                    x.load(px, v0);
                    y.load(px, v1);
                    x.get(f);
                    y.get(g);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 z = turn(make_float2(f[i], g[i]), cs[k][j + i]);
                        f[i] = z.x;
                        g[i] = z.y;
                    }
                    OutVec<IO>::store(po, v0, f);
                    OutVec<IO>::store(po, v1, g);
                }
                for (int e = threadIdx.x; e < a.H * rest; e += THREADS) {
                    const int v = e / rest * V + 2 * W + e % rest;
                    Vec<IO> x;
                    float f[8];
                    x.load(px, v);
                    x.get(f);
                    OutVec<IO>::store(po, v, f);
                }
            } else {
                const int rest = a.d - turned, per = a.pairs + rest;
                for (int e = threadIdx.x; e < a.H * per; e += THREADS) {
                    const int h = e / per, j = e % per;
                    if (j < a.pairs) {
                        const int axis = 2 * j < a.dim[0] ? 0 : 2 * j < a.dim[0] + a.dim[1] ? 1 : 2;
                        const int before = axis == 0 ? 0 : axis == 1 ? a.dim[0] : a.dim[0] + a.dim[1];
                        const size_t i0 = (size_t)h * a.d + before + j - before / 2, i1 = i0 + a.dim[axis] / 2;
                        const float2 z = turn(make_float2(load1<IO>(a.x, xr + i0), load1<IO>(a.x, xr + i1)), cs[k][j]);
                        store1<IO>(a.out, orow + i0, z.x);
                        store1<IO>(a.out, orow + i1, z.y);
                    } else {
                        const size_t i = (size_t)h * a.d + turned + j - a.pairs;
                        store1<IO>(a.out, orow + i, load1<IO>(a.x, xr + i));
                    }
                }
            }
        }
        __syncthreads();  // the angles are read above and written for the next tokens
    }
}

template <int IO>
hipError_t launch(const RotaryArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)std::min<long long>((a.B * a.T + TOK - 1) / TOK, 1 << 20)), block(THREADS);
    const bool whole = a.dim[0] % 16 == 0 && a.dim[1] % 16 == 0 && a.dim[2] % 16 == 0;
    if (!a.halves)
        rotary_kernel<IO, NEIGHBOURS><<<grid, block, 0, s>>>(a);
    else if (whole)
        rotary_kernel<IO, WHOLE_HALVES><<<grid, block, 0, s>>>(a);
    else
        rotary_kernel<IO, ANY_HALVES><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs &a, hipStream_t s) {
    return a.io == IO_F32 ? launch<IO_F32>(a, s) : a.io == IO_BF16 ? launch<IO_BF16>(a, s) : launch<IO_FP8>(a, s);
}

}  // namespace gdn
