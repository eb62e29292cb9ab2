// gdn_rms_norm.hip -- the root-mean-square norm with the residual's addition, its 8-bit output
// and its gradient; rows quantised to 8 bits without a norm.
//
//     h = x + r (rounded to the type that holds it),   y = h w / sqrt(mean(h^2) + eps)
//     8 bits: s = max|y| / 127,  q = the nearest of -127 .. 127 to y / s (ties to even)
//     dh = dsum + rstd (w dy - hhat mean(w dy hhat)),  dw = sum over rows of dy hhat,  hhat = h rstd
//
// A wave or a block of four has a row in registers: every input is read once.  Bound by HBM (65,520
// x 4,096 bf16 with the residual to 8 bits: 320-356 us, 5.3-5.9 TB/s; to bf16 358, 6.0), and for few rows by
// the latency of a row's sums.
#include "gdn_elem.h"
#include "gdn_layer.h"

#include <algorithm>

namespace gdn {

namespace {

constexpr int WAVES = 4;  // rows of a block at a time

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int o = 32; o; o /= 2) x += __shfl_xor(x, o);
    return x;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
#pragma unroll
    for (int o = 32; o; o /= 2) x = max(x, (uint32_t)__shfl_xor((int)x, o));
    return x;
}
__device__ __forceinline__ double wave_max(double x) {
#pragma unroll
    for (int o = 32; o; o /= 2) x = fmax(x, __shfl_xor(x, o));
    return x;
}

// The whole number next to 127 p / top, of the two beside `middle`; ties to the even one.  p and top have 48 bits at
// most, so 127 p and middle top do not fit 64, and their quotient does not tell which side of the middle it is on
// (it may be as near as 2^-55 of it).  Their difference does: both products in two parts, which cancel without a rounding.
__device__ __forceinline__ float nearest_level(double p, double top, float middle) {
#pragma clang fp contract(off)  // the products below are rounded ones
    const double x = 127.0 * p, y = middle * top;
    const double d = (x - y) + (fma(127.0, p, -x) - fma((double)middle, top, -y));
    return d == 0.0 ? rintf(middle) : d > 0.0 ? middle + 0.5f : middle - 0.5f;
}

enum RmsOut : int { RMS_SAME = 0, RMS_EIGHT = 1 };

// A row's value over all of its waves: of one wave as it is, of four through LDS.
template <int ROWW, typename T, typename F>
__device__ __forceinline__ T row_join(T x, T *part, F join) {
    if constexpr (ROWW > 1) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
        __syncthreads();
        x = part[0];
#pragma unroll
        for (int w = 1; w < ROWW; ++w) x = join(x, part[w]);
    }
    return x;
}

// V vectors of eight a lane, ROWW waves a row: C <= 512 V ROWW.  With four waves a row the weights
// are asked for with the row; a wave alone reads them again where they are used.
template <int IO, int V, int OUT, int ROWW>
__global__ void __launch_bounds__(64 * WAVES) rms_forward_kernel(const RmsArgs a) {
    static_assert(ROWW == 1 || ROWW == WAVES, "a wave or a block a row");
    __shared__ float part_f[WAVES];
    __shared__ uint32_t part_u[WAVES];
    __shared__ double part_d[WAVES];
    constexpr int LANES = 64 * ROWW;
    const int lane = threadIdx.x % LANES;
    const long long row = ROWW == 1 ? (long long)blockIdx.x * WAVES + (threadIdx.x >> 6)
                                    : (long long)blockIdx.y * gridDim.x + blockIdx.x;
    if (row >= a.N) return;
    const int n8 = a.C / 8;
    const size_t base = (size_t)row * n8;
    Vec<IO> x[V], r[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (lane + LANES * i < n8) x[i].load_once(a.x, base + lane + LANES * i);
    if (a.residual) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + LANES * i < n8) r[i].load_once(a.residual, base + lane + LANES * i);
    }
    Vec<IO_F32> wv[ROWW > 1 ? V : 1];
    if (ROWW > 1 && a.weight) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + LANES * i < n8) wv[i].load(a.weight, lane + LANES * i);
    }
    const auto weights = [&](int i, float (&w)[8]) {  // of vector i, if there are any
        if constexpr (ROWW > 1) {
            wv[i].get(w);
        } else {
            Vec<IO_F32> v;
            v.load(a.weight, lane + LANES * i);
            v.get(w);
        }
    };
    float h[V][8];
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (lane + LANES * i < n8) {
            x[i].get(h[i]);
            if (a.residual) {
                float f[8];
                r[i].get(f);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[i][e] += f[e];
                // the norm is of what the stream holds: one rounding, the one that is stored
                if constexpr (IO == IO_BF16) {
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const uint32_t p = pack_bf16x2(h[i][e], h[i][e + 1]);
                        h[i][e] = bf16_lo(p);
                        h[i][e + 1] = bf16_hi(p);
                    }
                }
                if (a.sum) OutVec<IO>::store(a.sum, base + lane + LANES * i, h[i]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sq += h[i][e] * h[i][e];
        }
    }
    float rstd = 1.0f;
    if (a.norm) {
        sq = row_join<ROWW>(wave_sum(sq), part_f, [](float p, float q) { return p + q; });
        rstd = 1.0f / sqrtf(sq / (float)a.C + a.eps);
        if (a.rstd_out && lane == 0) a.rstd_out[row] = rstd;
    }
    if constexpr (OUT == RMS_SAME) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + LANES * i < n8) {
                float w[8], y[8];
                if (a.weight) weights(i, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y[e] = h[i][e] * rstd;
                    if (a.weight) y[e] *= w[e];
                }
                OutVec<IO>::store(a.out, base + lane + LANES * i, y);
            }
    } else {
        // A row's factor rstd changes its scale, not its levels: they are those of h w.  The
        // product is rounded in 32 bits; where its level is next to the middle of two, and for
        // the largest, it is taken exactly (64 bits hold it), and the level with it.
        uint32_t big = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + LANES * i < n8) {
                float w[8];
                if (a.weight) weights(i, w);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    big = max(big, __float_as_uint(a.weight ? h[i][e] * w[e] : h[i][e]) & 0x7fffffffu);
            }
        big = row_join<ROWW>(wave_max(big), part_u, [](uint32_t p, uint32_t q) { return max(p, q); });
        const float top = __uint_as_float(big);
        // rows of (nearly) zeros: scale 0; rows that are not finite: NaN, as the bits compare
        const bool finite = big < 0x7f800000u && rstd > 0.0f && rstd < __builtin_inff(), some = top >= 0x1p-100f;
        double exact = top;  // without weights, the values are exact
        if (finite && some && a.weight) {  // the same for all of a row's lanes
            exact = 0.0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane + LANES * i < n8) {
                    float w[8];
                    weights(i, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (fabsf(h[i][e] * w[e]) == top) exact = fmax(exact, fabs((double)h[i][e] * (double)w[e]));
                }
            exact = row_join<ROWW>(wave_max(exact), part_d, [](double p, double q) { return fmax(p, q); });
        }
        if (lane == 0) a.scale[row] = !finite ? __builtin_nanf("") : some ? top * rstd / 127.0f : 0.0f;
        const float inv = finite && some ? 127.0f / top : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + LANES * i < n8) {
                float w[8];
                if (a.weight) weights(i, w);
                uint32_t b[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    int q = 0;
                    if (finite && some) {
                        const float level = (a.weight ? h[i][e] * w[e] : h[i][e]) * inv;
                        float k = rintf(level);
                        if (fabsf(level - k) > 0.499f)  // level is off by less than 1e-4
                            k = nearest_level((double)h[i][e] * (a.weight ? (double)w[e] : 1.0), exact, floorf(level) + 0.5f);
                        q = (int)k;
                    }
                    b[e / 4] |= (uint32_t)(q & 0xff) << (8 * (e % 4));
                }
                const u32x2_t v = {b[0], b[1]};
                stream_out(reinterpret_cast<u32x2_t *>(a.out8) + base + lane + LANES * i, v);
            }
    }
}

// Gradient: a wave (or block) walks rows and keeps its share of dweight in registers; the waves of
// a block that have the same channels are joined in LDS, the blocks' rows by the kernel below,
// always in the same order.
template <int IO, int V, int ROWW>
__global__ void __launch_bounds__(64 * WAVES) rms_backward_kernel(const RmsArgs a, float *partial) {
    constexpr int LANES = 64 * ROWW, ROWS = WAVES / ROWW;
    __shared__ float part[ROWW == 1 ? 512 * V : 1];
    __shared__ float part_f[2][WAVES];
    const int lane = threadIdx.x % LANES, wave = threadIdx.x >> 6;
    const int n8 = a.C / 8;
    float dw[V][8], w[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dw[i][e] = 0.0f;
            w[i][e] = 1.0f;
        }
        if (a.weight && lane + LANES * i < n8) {
            Vec<IO_F32> v;
            v.load(a.weight, lane + LANES * i);
            v.get(w[i]);
        }
    }
    int turn = 0;
    for (long long row = (long long)blockIdx.x * ROWS + (ROWW == 1 ? wave : 0); row < a.N; row += (long long)gridDim.x * ROWS) {
        const size_t base = (size_t)row * n8;
        Vec<IO> x[V], dy[V], ds[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + LANES * i < n8) {
                x[i].load_once(a.x, base + lane + LANES * i);
                dy[i].load_once(a.dout, base + lane + LANES * i);
                if (a.dsum) ds[i].load_once(a.dsum, base + lane + LANES * i);
            }
        const float rstd = a.rstd[row];
        float along = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + LANES * i < n8) {
                float f[8], d[8];
                x[i].get(f);
                dy[i].get(d);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float t = d[e] * (f[e] * rstd);
                    dw[i][e] += t;
                    along += t * w[i][e];
                }
            }
        // (one barrier a row: the next row's parts go to the other four places)
        along = row_join<ROWW>(wave_sum(along), part_f[turn], [](float p, float q) { return p + q; }) / (float)a.C;
        turn ^= 1;
        if (a.dx) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane + LANES * i < n8) {
                    float f[8], d[8], s[8];
                    x[i].get(f);
                    dy[i].get(d);
                    if (a.dsum) ds[i].get(s);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float y = rstd * (d[e] * w[i][e] - f[e] * rstd * along);
                        if (a.dsum) y += s[e];
                        f[e] = y;
                    }
                    OutVec<IO>::store(a.dx, base + lane + LANES * i, f);
                }
        }
    }
    if (!partial) return;
    if constexpr (ROWW > 1) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + LANES * i < n8) {
                float *p = partial + (size_t)blockIdx.x * a.C + 8 * (lane + LANES * i);
                *reinterpret_cast<f32x4_t *>(p) = f32x4_t{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
                *reinterpret_cast<f32x4_t *>(p + 4) = f32x4_t{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
            }
    } else {
        for (int k = 0; k < WAVES; ++k) {
            if (wave == k) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (lane + LANES * i < n8) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float *p = part + (lane + LANES * i) * 8 + e;
                            *p = k ? *p + dw[i][e] : dw[i][e];
                        }
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < a.C; c += 64 * WAVES) partial[(size_t)blockIdx.x * a.C + c] = part[c];
    }
}

// dweight[c] = sum over the blocks' rows: 32 columns a block, 32 threads a column (eight took 20 us
// for 512 rows of 2,560, one read after another; twice the rows 4.7 so).
__global__ void __launch_bounds__(1024) rms_weight_kernel(const float *partial, float *dweight, int rows, int C) {
    __shared__ float part[32][33];
    const int l = threadIdx.x & 31, c = blockIdx.x * 32 + l, k = threadIdx.x >> 5;
    float s = 0.0f;
    if (c < C) {
#pragma unroll 4
        for (int r = k; r < rows; r += 32) s += partial[(size_t)r * C + c];
    }
    part[k][l] = s;
    __syncthreads();
    for (int o = 16; o; o /= 2) {
        if (k < o) part[k][l] += part[k + o][l];
        __syncthreads();
    }
    if (k == 0 && c < C) dweight[c] = part[0][l];
}

// A block a row from C = 1,025 on: 65,520 x 4,096 bf16 to 8 bits 356 us against 399 for a wave a row,
// 8 x 2,560 5.6 against 10; below, a wave: 30,000 x 1,024 48 us against 63, 65,000 x 320 51 against 102.
bool block_a_row(int C) { return C > 1024; }

// Blocks of the gradient: enough to fill the device, few enough that their rows of dweight are
// little beside the data (32,760 x 2,560 bf16: four a CU 125 us, two 164, eight 131; 65,520 x 4,096: two
// 362, four 385).
int backward_blocks(int C, long long N, int ncu) {
    const long long rows = block_a_row(C) ? N : (N + WAVES - 1) / WAVES;
    return (int)std::max(1LL, std::min<long long>(rows, (C >= 4096 ? 2LL : 4LL) * ncu));
}

template <int IO, int V, int ROWW>
hipError_t forward_launch(const RmsArgs &a, hipStream_t stream) {
    // a grid's axis holds fewer than 2^32 threads: 2^24 rows of a block each are just too many for one
    const unsigned half = ROWW > 1 && a.N > (1LL << 23) ? 2 : 1;
    const dim3 grid((unsigned)(ROWW == 1 ? (a.N + WAVES - 1) / WAVES : (a.N + half - 1) / half), half), block(64 * WAVES);
    if (a.out8) hipLaunchKernelGGL((rms_forward_kernel<IO, V, RMS_EIGHT, ROWW>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((rms_forward_kernel<IO, V, RMS_SAME, ROWW>), grid, block, 0, stream, a);
    return hipGetLastError();
}
template <int IO, int V, int ROWW>
hipError_t backward_launch(const RmsArgs &a, hipStream_t stream) {
    const int blocks = backward_blocks(a.C, a.N, a.ncu);
    float *partial = a.dweight ? static_cast<float *>(a.work) : nullptr;
    hipLaunchKernelGGL((rms_backward_kernel<IO, V, ROWW>), dim3(blocks), dim3(64 * WAVES), 0, stream, a, partial);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !partial) return e;
    hipLaunchKernelGGL(rms_weight_kernel, dim3((a.C + 31) / 32), dim3(1024), 0, stream, partial, a.dweight, blocks, a.C);
    return hipGetLastError();
}

#define GDN_RMS_SIZES(FN)                                 \
    if (!block_a_row(a.C))                                \
        return a.C <= 512 ? FN<IO, 1, 1>(a, stream) : FN<IO, 2, 1>(a, stream); \
    if (a.C <= 2048) return FN<IO, 1, WAVES>(a, stream);  \
    if (a.C <= 4096) return FN<IO, 2, WAVES>(a, stream);  \
    return FN<IO, 4, WAVES>(a, stream);
template <int IO>
hipError_t forward_sizes(const RmsArgs &a, hipStream_t stream) { GDN_RMS_SIZES(forward_launch) }
template <int IO>
hipError_t backward_sizes(const RmsArgs &a, hipStream_t stream) { GDN_RMS_SIZES(backward_launch) }
#undef GDN_RMS_SIZES

__global__ void __launch_bounds__(256) rms_zero_kernel(float *p, int n) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = 0.0f;
}

}  // namespace

size_t rms_work_bytes(int C, long long max_N, int ncu) {
    return (size_t)backward_blocks(C, max_N, ncu) * C * sizeof(float);
}

hipError_t launch_rms_forward(const RmsArgs &a, hipStream_t stream) {
    if (a.N == 0) return hipSuccess;
    return a.io == IO_F32 ? forward_sizes<IO_F32>(a, stream) : forward_sizes<IO_BF16>(a, stream);
}

hipError_t launch_rms_backward(const RmsArgs &a, hipStream_t stream) {
    if (a.N == 0) {
        if (!a.dweight) return hipSuccess;
        hipLaunchKernelGGL(rms_zero_kernel, dim3((a.C + 255) / 256), dim3(256), 0, stream, a.dweight, a.C);
        return hipGetLastError();
    }
    return a.io == IO_F32 ? backward_sizes<IO_F32>(a, stream) : backward_sizes<IO_BF16>(a, stream);
}

}  // namespace gdn
