// gdn_rotary.hip -- rotary positions over three axes (include/gdn.h, gdn_rotary).
//
// Bound by HBM: six flops per pair read and written.  Pair j of every head of a token is
// turned by the same angle, so a block takes TOK tokens at a time, forms their cosines and
// sines once (frequency and angle in 64 bits, the angle reduced to a fraction of a turn before
// the fp32 sine) into LDS and turns all heads with them.  The frequencies are formed once a
// block; blocks stay for many tokens.
//  * pairs (2i, 2i + 1): a lane takes eight neighbouring elements (16 bytes of bf16), four
//    whole pairs.
//  * halves that are multiples of W elements, W * size >= 8 bytes: a lane takes W neighbouring
//    elements of a section's first half and the W of the second half that belong to them.
//  * other halves: whole heads are staged in LDS in 16-byte vectors; a lane forms eight
//    neighbouring outputs and finds their partners there (2 x 11,267 tokens of 26 heads of 64,
//    halves of 2, 4 and 3, bf16: 52 us, floor 29; two-byte accesses to memory instead: 116 us).
//    Bound by vector instructions, 46 an element and 93% of the time: each output finds its
//    section, its partner and its angle on its own.
// out may be x: a pair is read and written by one lane, and heads are staged whole before any
// of them is written.
// Measured: 2 x 32,760 tokens of 64 heads of 128 in packed rows, bf16: 358 us, 6.0 TB/s read
// and written (a copy of 1 GB: 5.1 TB/s); 8 tokens of 40 heads: 4.3 us, the latency of one block;
// 1,560 tokens of 40 heads, FP8: 7.4 us, floor 4.7 (a short call waits for the frequencies, the
// places and the angles, a barrier behind each, before its first load of x).
#include "gdn_elem.h"
#include "gdn_layer.h"

#include <algorithm>

namespace gdn {
namespace {

constexpr int THREADS = 256;
constexpr int ROTARY_BLOCKS = 1 << 14;

// Axis of pair j, and its number in the axis' section.
__device__ __forceinline__ int axis_of(const RotaryArgs &a, int &j) {
    if (2 * j < a.dim[0]) return 0;
    j -= a.dim[0] / 2;
    if (2 * j < a.dim[1]) return 1;
    j -= a.dim[1] / 2;
    return 2;
}

// Turns of pair j per unit of position.
__device__ __forceinline__ double frequency(const RotaryArgs &a, int j) {
    const int axis = axis_of(a, j);
    return exp2(-2.0 * j / a.dim[axis] * a.log2_theta) * 0.15915494309189533577;  // 1 / 2 pi
}

// Position of token t of batch element b on an axis: a 32-bit number.
__device__ __forceinline__ int position(const RotaryArgs &a, unsigned b, long long t, int axis) {
    if (a.positions) return a.positions[b * a.pos_bs + 3 * t + axis];
    const long long n = a.first_token + t, area = (long long)a.height * a.width;
    if (((n | area) >> 32) == 0) {  // a 64-bit division is some hundred instructions
        const unsigned m = (unsigned)n;
        return axis == 0 ? m / (unsigned)area : axis == 1 ? m / (unsigned)a.width % (unsigned)a.height : m % (unsigned)a.width;
    }
    return (int)(axis == 0 ? n / area : axis == 1 ? n / a.width % a.height : n % a.width);
}

__device__ __forceinline__ float2 turn(float2 x, float2 cs) {
    return make_float2(x.x * cs.x - x.y * cs.y, x.x * cs.y + x.y * cs.x);
}

// W neighbouring elements from element i on (i a multiple of W; a row starts at 16 bytes):
// eight of any type, or at least 8 bytes.
template <int IO, int W>
__device__ __forceinline__ void load_part(const void *row, size_t i, float (&f)[W]) {
    if constexpr (W == 8) {
        Vec<IO> x;
        x.load_once(row, i / 8);
        x.get(f);
    } else if constexpr (IO == IO_F32) {
        typedef float part __attribute__((ext_vector_type(W)));
        const part x = *reinterpret_cast<const part *>(static_cast<const float *>(row) + i);
#pragma unroll
        for (int k = 0; k < W; ++k) f[k] = x[k];
    } else {
        static_assert(IO == IO_BF16 && W == 4, "half a vector");
        const uint2 x = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(row) + i);
        f[0] = bf16_lo(x.x);
        f[1] = bf16_hi(x.x);
        f[2] = bf16_lo(x.y);
        f[3] = bf16_hi(x.y);
    }
}
template <int IO, int W>
__device__ __forceinline__ void store_part(void *row, size_t i, const float (&f)[W]) {
    if constexpr (W == 8) {
        OutVec<IO>::store(row, i / 8, f);
    } else if constexpr (IO == IO_F32) {
        typedef float part __attribute__((ext_vector_type(W)));
        part x;
#pragma unroll
        for (int k = 0; k < W; ++k) x[k] = f[k];
        stream_out(reinterpret_cast<part *>(static_cast<float *>(row) + i), x);
    } else {
        const u32x2_t x = {pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])};
        stream_out(reinterpret_cast<u32x2_t *>(static_cast<uint16_t *>(row) + i), x);
    }
}

// What a block does with its tokens: pairs (2i, 2i + 1), halves by W > 0 elements, or halves
// through LDS.
constexpr int NEIGHBOURS = 0, STAGED = -1;
constexpr int STAGE_BYTES = 16 * 1024;  // of staged elements, in their own type

template <int IO, int W, int TOK>
__global__ __launch_bounds__(THREADS) void rotary_kernel(RotaryArgs a) {
    __shared__ double freq[ROTARY_MAX_PAIRS];
    __shared__ float2 cs[TOK][ROTARY_MAX_PAIRS];
    __shared__ int pos[TOK][3];
    __shared__ const void *from[TOK];  // x and out of the tokens
    __shared__ void *to[TOK];
    __shared__ __align__(16) char stage[W == STAGED ? STAGE_BYTES : 16];
    const unsigned rows = (unsigned)(a.B * a.T), T = (unsigned)a.T;
    const float sign = a.inverse ? -1.0f : 1.0f;
    for (int j = threadIdx.x; j < a.pairs; j += THREADS) freq[j] = frequency(a, j);
    __syncthreads();
    for (unsigned row0 = blockIdx.x * TOK; row0 < rows; row0 += gridDim.x * TOK) {
        const unsigned tokens = rows - row0 < TOK ? rows - row0 : TOK;
        if (threadIdx.x < 4 * tokens) {
            const unsigned k = threadIdx.x / 4, what = threadIdx.x % 4, b = (row0 + k) / T, t = (row0 + k) % T;
            if (what < 3) {
                pos[k][what] = position(a, b, t, what);
            } else {
                from[k] = at<IO>(a.x, (size_t)b * a.x_bs + (size_t)t * a.x_ts);
                to[k] = at<OutIo<IO>>(a.out, (size_t)b * a.out_bs + (size_t)t * a.out_ts);
            }
        }
        __syncthreads();
        for (unsigned e = threadIdx.x; e < tokens * a.pairs; e += THREADS) {
            const unsigned k = TOK == 1 ? 0 : e / a.pairs, j = e - k * a.pairs;
            int i = j;
            const double turns = (double)pos[k][axis_of(a, i)] * freq[j];
            float s, c;
            sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
            cs[k][j] = make_float2(c, sign * s);
        }
        __syncthreads();
        if constexpr (W == NEIGHBOURS) {
            // vector v of token k, number c of its head; divisions only before the loop
            const unsigned V = a.d / 8, HV = a.H * V, step = THREADS % V;
            unsigned k = TOK == 1 ? 0 : threadIdx.x / HV, v = threadIdx.x - k * HV, c = threadIdx.x % V;
            if (TOK == 1 && v >= HV) k = 1;
            while (k < tokens) {
                Vec<IO> x;
                float f[8];
                x.load_once(from[k], v);
                x.get(f);
                const int j0 = c * 4;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (j0 + i < a.pairs) {
                        const float2 y = turn(make_float2(f[2 * i], f[2 * i + 1]), cs[k][j0 + i]);
                        f[2 * i] = y.x;
                        f[2 * i + 1] = y.y;
                    }
                OutVec<IO>::store(to[k], v, f);
                for (v += THREADS; v >= HV && k < tokens; v -= HV) ++k;
                c += step;
                if (c >= V) c -= V;
            }
        } else if constexpr (W > 0) {
            // a head's parts: its pairs, W at a time, then what passes through
            const unsigned P = a.pairs / W, per = P + (a.d - 2 * a.pairs) / W, HP = a.H * per;
            const int d0 = a.dim[0] / 2, d1 = a.dim[1] / 2;
            for (unsigned e = threadIdx.x; e < tokens * HP; e += THREADS) {
                const unsigned k = TOK == 1 ? 0 : e / HP, hp = e - k * HP, h = hp / per, p = hp - h * per;
                const int j = p * W;
                const size_t head = (size_t)h * a.d;
                float f[W];
                if (p < P) {
                    // section starts 2 `before` into the head, pair j is its number j - before
                    const int before = j < d0 ? 0 : j < d0 + d1 ? d0 : d0 + d1;
                    const int half = j < d0 ? d0 : j < d0 + d1 ? d1 : a.dim[2] / 2;
                    const size_t i0 = head + before + j, i1 = i0 + half;
                    float g[W];
                    load_part<IO, W>(from[k], i0, f);
                    load_part<IO, W>(from[k], i1, g);
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        const float2 z = turn(make_float2(f[i], g[i]), cs[k][j + i]);
                        f[i] = z.x;
                        g[i] = z.y;
                    }
                    store_part<IO, W>(to[k], i0, f);
                    store_part<IO, W>(to[k], i1, g);
                } else {
                    const size_t i = head + 2 * a.pairs + (p - P) * W;
                    load_part<IO, W>(from[k], i, f);
                    store_part<IO, W>(to[k], i, f);
                }
            }
        } else {
            // (token, head) number u of the block's tokens x H, as many at a time as fit in LDS
            const unsigned V = a.d / 8, units = tokens * a.H, fit = STAGE_BYTES / (a.d * io_in_bytes(IO));
            const int d0 = a.dim[0] / 2, d1 = a.dim[1] / 2, d2 = a.dim[2] / 2;
            for (unsigned u0 = 0; u0 < units; u0 += fit) {
                const unsigned n = units - u0 < fit ? units - u0 : fit;
                for (unsigned e = threadIdx.x; e < n * V; e += THREADS) {
                    const unsigned u = e / V, k = TOK == 1 ? 0 : (u0 + u) / a.H, h = u0 + u - k * a.H;
                    Vec<IO> x;
                    x.load_once(from[k], h * V + (e - u * V));
                    reinterpret_cast<Vec<IO> *>(stage)[e] = x;
                }
                __syncthreads();
                for (unsigned e = threadIdx.x; e < n * V; e += THREADS) {
                    const unsigned u = e / V, k = TOK == 1 ? 0 : (u0 + u) / a.H, h = u0 + u - k * a.H, v = e - u * V;
                    float f[8];
                    reinterpret_cast<const Vec<IO> *>(stage)[e].get(f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        // element c of the head: pair before + (place in its half)
                        const int c = v * 8 + i;
                        if (c < 2 * a.pairs) {
                            const int before = c < 2 * d0 ? 0 : c < 2 * (d0 + d1) ? d0 : d0 + d1;
                            const int half = c < 2 * d0 ? d0 : c < 2 * (d0 + d1) ? d1 : d2;
                            const int in = c - 2 * before;
                            const bool second = in >= half;
                            const float other = load1<IO>(stage, (size_t)u * a.d + c + (second ? -half : half));
                            const float2 w = cs[k][before + in - (second ? half : 0)];
                            f[i] = second ? other * w.y + f[i] * w.x : f[i] * w.x - other * w.y;
                        }
                    }
                    OutVec<IO>::store(to[k], h * V + v, f);
                }
                __syncthreads();
            }
        }
        __syncthreads();  // the angles are read above and written for the next tokens
    }
}

template <int IO, int W>
hipError_t launch(const RotaryArgs &a, hipStream_t s) {
    // Four tokens share a block's passes over the angles and its barriers where a token alone
    // would leave threads idle (6,240 tokens of 4 heads of 128: 7.6 us, one token at a time
    // 10.8).  One token at a time for wide rows (2 x 32,760 of 64 heads: fours are 7% slower) and
    // where fours would leave CUs idle (1,560 of 40 heads: 8.2 us, by fours 11.3).
    const long long rows = a.B * a.T;
    if (rows >= 4096 && a.H * (long long)a.d < 8 * 4 * THREADS)
        rotary_kernel<IO, W, 4><<<dim3((unsigned)std::min<long long>((rows + 3) / 4, ROTARY_BLOCKS)), dim3(THREADS), 0, s>>>(a);
    else
        rotary_kernel<IO, W, 1><<<dim3((unsigned)std::min<long long>(rows, 4 * ROTARY_BLOCKS)), dim3(THREADS), 0, s>>>(a);
    return hipGetLastError();
}

template <int IO>
hipError_t launch(const RotaryArgs &a, hipStream_t s) {
    if (!a.halves) return launch<IO, NEIGHBOURS>(a, s);
    const int all = a.dim[0] / 2 | a.dim[1] / 2 | a.dim[2] / 2;
    if (all % 8 == 0) return launch<IO, 8>(a, s);
    if constexpr (IO != IO_FP8)
        if (all % 4 == 0) return launch<IO, 4>(a, s);
    if constexpr (IO == IO_F32)
        if (all % 2 == 0) return launch<IO, 2>(a, s);
    return launch<IO, STAGED>(a, s);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs &a, hipStream_t s) {
    return a.io == IO_F32 ? launch<IO_F32>(a, s) : a.io == IO_BF16 ? launch<IO_BF16>(a, s) : launch<IO_FP8>(a, s);
}

}  // namespace gdn
