// gdn_group_norm.hip -- group norm with an activation, channels last, and its gradient
// (include/gdn.h, gdn_group_norm_forward / gdn_group_norm_backward).
//
// All forms are bound by HBM, the small ones by the latency of their steps.  A thread holds
// eight neighbouring channels (a 16-byte vector in bf16) and a fixed place in the row, so that
// weight and bias stay in registers; V = C / 8 threads make a row, and a block has
// R = threads / V rows at once.  Three forms by the size of a sample:
//  * rows (S = 1, D = C / G channels of a group a multiple of 8 up to 512): a group is D / 8
//    lanes of a wave, or the power of two above with the rest idle; its sums are exchanges
//    between lanes and the row is read once.
//  * resident (small samples): a block has a sample, or a piece of it of whole groups where
//    samples are few, in registers for the forward pass, and joins its groups through LDS; one
//    launch.
//  * split (larger samples): a sample is cut into stretches of rows.  One launch forms each
//    stretch's sums, a small one joins them, one applies them, taking the stretches in the
//    opposite order so that what the first left in the caches is read from there.
// Squares are always taken around a mean, or a value of the set itself, and partial results
// (count, mean, squares around it) are joined by
//     mean = sum n_i mean_i / n,   squares = sum squares_i + sum n_i (mean_i - mean)^2,
// so that means far from zero cost no precision.  Everything is fp32 until the last rounding.
// Measured (a copy of 1 GB: 5.1 TB/s): rows, 65,520 x 4096 in 32 groups, SiLU, bf16: 201 us,
// 5.3 TB/s (its gradient 350 us, 4.6 TB/s; joined through LDS instead: 585 us forward); split,
// 2 x 32,760 x 512 forward 44 us and gradient 66 us with both passes over x and dout; resident,
// 3 x 77 x 320 fp32: 6 us forward and 11 us with the gradient's two launches, 8 pieces a sample
// (whole samples: 9 and 16 us).
#include "gdn_elem.h"
#include "gdn_layer.h"

#include <algorithm>
#include <numeric>

namespace gdn {
namespace {

constexpr int RES_K = 4;        // rows of a thread in the resident form
constexpr int ROWS_U = 4;       // rows a thread of the other forms has in flight
constexpr int BATCH = 1024;     // samples of one round of the split form (bounds the workspace)
// Stretches times groups of a sample that each block may join for itself: saves a launch (20 x
// 1,798 x 256, 52 stretches of 16 groups: 19.9 us against 21.8).
constexpr int JOIN_HERE = 2048;

// 1 / (1 + e^-z) with the hardware's exponential and reciprocal (an ulp each; the IEEE
// forms would make the pass bound by the vector units).
__device__ __forceinline__ float sigmoid_fast(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * LOG2E_F));
}
template <bool SILU>
__device__ __forceinline__ float act(float z) {
    return SILU ? z * sigmoid_fast(z) : z;
}
// dy act'(z)
template <bool SILU>
__device__ __forceinline__ float act_grad(float dy, float z) {
    if (!SILU) return dy;
    const float q = sigmoid_fast(z);
    return dy * (q * fmaf(z, 1.0f - q, 1.0f));
}

// Sum over aligned groups of L lanes (a power of two up to 64), in each of them.
__device__ __forceinline__ float lanes_sum(float x, int L) {
    if (L > 1) x += dpp_mov<0xB1>(x);
    if (L > 2) x += dpp_mov<0x4E>(x);
    if (L > 4) x += dpp_mov<0x141>(x);
    if (L > 8) x += dpp_mov<0x140>(x);
    if (L > 16) x += __shfl_xor(x, 16);
    if (L > 32) x += __shfl_xor(x, 32);
    return x;
}

__device__ __forceinline__ void channel8(float (&f)[8], const float *p, int col, float none) {
    if (p) {
        const float4 a = reinterpret_cast<const float4 *>(p)[2 * col], b = reinterpret_cast<const float4 *>(p)[2 * col + 1];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = none;
    }
}

// eps is a normal number, which the hardware's reciprocal square root (an ulp) needs.
__device__ __forceinline__ float inv_std(float var, float eps) { return __builtin_amdgcn_rsqf(var + eps); }

// ---- rows ---------------------------------------------------------------------------

// A thread's place: group by group, L lanes each (P = V / G of them used), a row after another.
struct Place {
    int row, col;
    bool on;  // idle lanes repeat the first vector of their group
    __device__ __forceinline__ Place(const GroupNormArgs &a, int V, int R, int L) {
        const int P = V / a.G, width = a.G * L, at = threadIdx.x % width, i = at % L;
        row = threadIdx.x / width;
        col = at / L * P + (i < P ? i : 0);
        on = row < R && i < P;
    }
};

template <int IO, bool SILU>
__global__ __launch_bounds__(512) void rows_forward_kernel(GroupNormArgs a, int V, int R, int L) {
    const Place p(a, V, R, L);
    const int row = p.row, col = p.col, P = V / a.G;
    const bool on = p.on;
    float w[8], b[8];
    channel8(w, a.weight, col, 1.0f);
    channel8(b, a.bias, col, 0.0f);
    const float inv = 1.0f / (float)(8 * P);
    const long long step = (long long)gridDim.x * R;
    for (long long n0 = (long long)blockIdx.x * R; n0 < a.N; n0 += ROWS_U * step) {
        Vec<IO> x[ROWS_U];
#pragma unroll
        for (int u = 0; u < ROWS_U; ++u) {
            const long long n = n0 + u * step + row;
            if (row < R && n < a.N) x[u].load_once(a.x, (size_t)n * V + col);
        }
#pragma unroll
        for (int u = 0; u < ROWS_U; ++u) {
            const long long n = n0 + u * step + row;
            float f[8], s = 0.0f, q = 0.0f;
            x[u].get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) s += f[i];
            const float mean = lanes_sum(on ? s : 0.0f, L) * inv;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[i] -= mean;
                q = fmaf(f[i], f[i], q);
            }
            const float rstd = inv_std(lanes_sum(on ? q : 0.0f, L) * inv, a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = act<SILU>(fmaf(f[i] * rstd, w[i], b[i]));
            if (on && n < a.N) {
                OutVec<IO>::store(a.out, (size_t)n * V + col, f);
                if (a.stats_out && col % P == 0)
                    reinterpret_cast<float2 *>(a.stats_out)[(size_t)n * a.G + col / P] = make_float2(mean, rstd);
            }
        }
    }
}

// Eight floats at the vector `i` of an LDS row.
__device__ __forceinline__ void put8(float *lds, int i, const float (&f)[8]) {
    reinterpret_cast<float4 *>(lds)[2 * i] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(lds)[2 * i + 1] = make_float4(f[4], f[5], f[6], f[7]);
}

// Sums of a block's rows for each of its C channels: part[0 .. C) gets s1, part[stride ..
// stride + C) s2.  Many rows are first summed by P threads a channel to P rows, the square root
// of R as far as the block has threads for them (204 rows of 40 channels: 2 us less; 89 rows:
// 0.3 us more, for the barrier).
__device__ __forceinline__ void block_channels(const float (&s1)[8], const float (&s2)[8], float *lds, float *part, int stride,
                                               int C, int row, int col, int R) {
    int P = 1;
    while (R > 128 && P * P < R && (P + 1) * C <= (int)blockDim.x) ++P;
    for (int k = 0; k < 2; ++k) {
        if (row < R) put8(lds + row * C, col, k ? s2 : s1);
        __syncthreads();
        if (P > 1) {
            if ((int)threadIdx.x < P * C) {
                float s = 0.0f;
#pragma unroll 4
                for (int i = threadIdx.x; i < R * C; i += P * C) s += lds[i];
                lds[threadIdx.x] = s;  // row threadIdx.x / C, which this thread alone reads
            }
            __syncthreads();
        }
        const int rows = P > 1 ? P : R;
        for (int c = threadIdx.x; c < C; c += blockDim.x) {
            float s = lds[c];
            for (int r = 1; r < rows; ++r) s += lds[r * C + c];
            part[(size_t)k * stride + c] = s;
        }
        __syncthreads();
    }
}

template <int IO, bool SILU>
__global__ __launch_bounds__(512) void rows_backward_kernel(GroupNormArgs a, int V, int R, int L, float *part) {
    extern __shared__ float lds[];
    const Place p(a, V, R, L);
    const int row = p.row, col = p.col, P = V / a.G;
    const bool on = p.on;
    float w[8], b[8], sw[8] = {}, sb[8] = {};
    channel8(w, a.weight, col, 1.0f);
    channel8(b, a.bias, col, 0.0f);
    const float inv = 1.0f / (float)(8 * P);
    constexpr int U = ROWS_U / 2;
    const long long step = (long long)gridDim.x * R;
    for (long long n0 = (long long)blockIdx.x * R; n0 < a.N; n0 += U * step) {
        Vec<IO> x[U];
        OutVec<IO> y[U];
        float2 st[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long n = n0 + u * step + row;
            if (row < R && n < a.N) {
                x[u].load_once(a.x, (size_t)n * V + col);
                y[u].load_once(a.dout, (size_t)n * V + col);
                st[u] = reinterpret_cast<const float2 *>(a.stats)[(size_t)n * a.G + col / P];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long n = n0 + u * step + row;
            const bool in = on && n < a.N;
            float f[8], t[8], s1 = 0.0f, s2 = 0.0f;
            x[u].get(f);
            y[u].get(t);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[i] = (f[i] - st[u].x) * st[u].y;
                const float dz = act_grad<SILU>(t[i], fmaf(f[i], w[i], b[i]));
                if (in) {
                    sb[i] += dz;
                    sw[i] = fmaf(dz, f[i], sw[i]);
                }
                t[i] = dz * w[i];
                s1 += t[i];
                s2 = fmaf(t[i], f[i], s2);
            }
            const float m1 = lanes_sum(on ? s1 : 0.0f, L) * inv, m2 = lanes_sum(on ? s2 : 0.0f, L) * inv;
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = st[u].y * (t[i] - m1 - f[i] * m2);
            if (in && a.dx) OutVec<IO>::store(a.dx, (size_t)n * V + col, t);
        }
    }
    if (part) block_channels(sb, sw, lds, part + (size_t)blockIdx.x * 2 * a.C, a.C, a.C, on ? row : R, col, R);
}

// ---- joining a block's threads by group ---------------------------------------------

// How many rows thread row r of R has of n: rows r, r + R, ...
struct Share {
    int each, extra;
    __device__ __forceinline__ Share(int n, int R) : each(n / R), extra(n % R) {}
    __device__ __forceinline__ float operator()(int r) const { return (float)(each + (r < extra)); }
};

// A thread's eight channels are first joined among themselves, as far as they are of one
// group: `unit` channels, the largest of 8, 4, 2, 1 that divides D.  LDS then holds R rows of
// C / unit entries (and R more for the second value).
__device__ __forceinline__ int unit_of(int D) { return D % 8 == 0 ? 8 : D % 4 == 0 ? 4 : D % 2 == 0 ? 2 : 1; }

template <int U>
__device__ __forceinline__ void put_moments_by(float *lds, int R, int K, int row, int col, float count, const float (&mean)[8],
                                               const float (&sq)[8]) {
#pragma unroll
    for (int e = 0; e < 8 / U; ++e) {
        float m = 0.0f, q = 0.0f;
#pragma unroll
        for (int i = 0; i < U; ++i) m += mean[e * U + i];
        m *= 1.0f / U;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const float d = mean[e * U + i] - m;
            q += fmaf(count * d, d, sq[e * U + i]);
        }
        lds[row * K + col * (8 / U) + e] = m;
        lds[(R + row) * K + col * (8 / U) + e] = q;
    }
}
__device__ __forceinline__ void put_moments(float *lds, int R, int C, int unit, int row, int col, float count,
                                            const float (&mean)[8], const float (&sq)[8]) {
    if (unit == 8)
        put_moments_by<8>(lds, R, C / 8, row, col, count, mean, sq);
    else if (unit == 4)
        put_moments_by<4>(lds, R, C / 4, row, col, count, mean, sq);
    else if (unit == 2)
        put_moments_by<2>(lds, R, C / 2, row, col, count, mean, sq);
    else
        put_moments_by<1>(lds, R, C, row, col, count, mean, sq);
}
template <int U>
__device__ __forceinline__ void put_sums_by(float *lds, int R, int K, int row, int col, const float (&s1)[8], const float (&s2)[8]) {
#pragma unroll
    for (int e = 0; e < 8 / U; ++e) {
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            a += s1[e * U + i];
            b += s2[e * U + i];
        }
        lds[row * K + col * (8 / U) + e] = a;
        lds[(R + row) * K + col * (8 / U) + e] = b;
    }
}
__device__ __forceinline__ void put_sums(float *lds, int R, int C, int unit, int row, int col, const float (&s1)[8],
                                         const float (&s2)[8]) {
    if (unit == 8)
        put_sums_by<8>(lds, R, C / 8, row, col, s1, s2);
    else if (unit == 4)
        put_sums_by<4>(lds, R, C / 4, row, col, s1, s2);
    else if (unit == 2)
        put_sums_by<2>(lds, R, C / 2, row, col, s1, s2);
    else
        put_sums_by<1>(lds, R, C, row, col, s1, s2);
}

// The whole block calls f(g, lane, L) for every group, L lanes of one wave for each (a power
// of two up to 64, as many as a group has items if that is less); g >= G marks lanes that
// only take part in the exchanges.
template <typename F>
__device__ __forceinline__ void each_group(int G, int items, F f) {
    int L = 1;
    while (L < 64 && L < items) L *= 2;
    const int per = blockDim.x / L;
    for (int g0 = 0; g0 < G; g0 += per) f(g0 + (int)threadIdx.x / L, (int)threadIdx.x % L, L);
}
// i / n for 0 <= i < 2^16 with inv = 1 / n: the quotient's distance from a whole number is at
// least 1 / 2n, its error below 2^-6 of that.
__device__ __forceinline__ int quotient(int i, float inv) { return (int)(((float)i + 0.5f) * inv); }

// What put_moments left: done(g, mean, squares) in one lane of each group of `rows` rows.
template <typename Done>
__device__ __forceinline__ void join_groups(const float *lds, int R, int C, int D, int unit, const Share &share, float rows,
                                            Done done) {
    const int K = C / unit, Du = D / unit, G = C / D, items = R * Du;
    const float *mean = lds, *sq = lds + R * K;
    const float inv = 1.0f / (float)Du, all = 1.0f / (rows * (float)Du);
    each_group(G, items, [&](int g, int lane, int L) {
        const int at = (g < G ? g : 0) * Du;
        float s = 0.0f, q = 0.0f;
        for (int i = lane; i < items; i += L) {
            const int r = quotient(i, inv);
            s = fmaf(share(r), mean[r * K + at + i - r * Du], s);
        }
        const float m = lanes_sum(s, L) * all;
        for (int i = lane; i < items; i += L) {
            const int r = quotient(i, inv), k = r * K + at + i - r * Du;
            const float d = mean[k] - m;
            q += fmaf(share(r) * (float)unit * d, d, sq[k]);
        }
        q = lanes_sum(q, L);
        if (g < G && lane == 0) done(g, m, q);
    });
}

// What put_sums left: done(g, sum1, sum2) in one lane of each group.
template <typename Done>
__device__ __forceinline__ void sum_groups(const float *lds, int R, int C, int D, int unit, Done done) {
    const int K = C / unit, Du = D / unit, G = C / D, items = R * Du;
    const float inv = 1.0f / (float)Du;
    each_group(G, items, [&](int g, int lane, int L) {
        const int at = (g < G ? g : 0) * Du;
        float s1 = 0.0f, s2 = 0.0f;
        for (int i = lane; i < items; i += L) {
            const int r = quotient(i, inv), k = r * K + at + i - r * Du;
            s1 += lds[k];
            s2 += lds[R * K + k];
        }
        s1 = lanes_sum(s1, L);
        s2 = lanes_sum(s2, L);
        if (g < G && lane == 0) done(g, s1, s2);
    });
}

// ---- resident -----------------------------------------------------------------------

// The call as piece p sees it, C channels in G groups.
template <int IO>
__device__ __forceinline__ void to_piece(GroupNormArgs &a, int p, int C, int G) {
    const size_t c = (size_t)p * C;
    a.x = at<IO>(a.x, c);
    if (a.weight) a.weight += c;
    if (a.bias) a.bias += c;
    if (a.out) a.out = at<OutIo<IO>>(a.out, c);
    if (a.dout) a.dout = at<OutIo<IO>>(a.dout, c);
    if (a.dx) a.dx = at<OutIo<IO>>(a.dx, c);
    if (a.stats) a.stats += 2 * p * G;
    if (a.stats_out) a.stats_out += 2 * p * G;
}

// A block takes a piece of V vectors (whole groups; piece blockIdx.y) of samples blockIdx.x,
// + gridDim.x, ...; thread (row, col) has rows row + k R.  LDS: 2 R C floats for joining (C, G:
// the piece's channels and groups), then 2 G for the groups' results.
template <int IO, bool SILU>
__global__ __launch_bounds__(1024) void resident_forward_kernel(GroupNormArgs a, int V, int R) {
    extern __shared__ float lds[];
    const int row = threadIdx.x / V, col = threadIdx.x % V, C = 8 * V, D = a.C / a.G, S = (int)a.S;
    const int width = a.C / 8;
    to_piece<IO>(a, blockIdx.y, C, C / D);
    const bool on = row < R;
    float2 *group = reinterpret_cast<float2 *>(lds + 2 * R * C);
    const Share share(S, R);
    const int unit = unit_of(D);
    for (long long n = blockIdx.x; n < a.N; n += gridDim.x) {
        Vec<IO> x[RES_K];
        const size_t base = (size_t)n * S * width + col;
#pragma unroll
        for (int k = 0; k < RES_K; ++k)
            if (on && row + k * R < S) x[k].load(a.x, base + (size_t)(row + k * R) * width);
        if (on) {
            float mean[8] = {}, sq[8] = {};
            const float inv = row < S ? 1.0f / share(row) : 0.0f;
#pragma unroll
            for (int k = 0; k < RES_K; ++k)
                if (row + k * R < S) {
                    float f[8];
                    x[k].get(f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) mean[i] += f[i];
                }
#pragma unroll
            for (int i = 0; i < 8; ++i) mean[i] *= inv;
#pragma unroll
            for (int k = 0; k < RES_K; ++k)
                if (row + k * R < S) {
                    float f[8];
                    x[k].get(f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) sq[i] = fmaf(f[i] - mean[i], f[i] - mean[i], sq[i]);
                }
            put_moments(lds, R, C, unit, row, col, share(row), mean, sq);
        }
        __syncthreads();
        join_groups(lds, R, C, D, unit, share, (float)S, [&](int g, float mean, float sq) {
            const float2 st = make_float2(mean, inv_std(sq / ((float)S * D), a.eps));
            group[g] = st;
            if (a.stats_out) reinterpret_cast<float2 *>(a.stats_out)[(size_t)n * a.G + g] = st;
        });
        __syncthreads();
        if (on) {
            float w[8], b[8];
            channel8(w, a.weight, col, 1.0f);
            channel8(b, a.bias, col, 0.0f);
            float2 st[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) st[i] = group[(8 * col + i) / D];
#pragma unroll
            for (int k = 0; k < RES_K; ++k)
                if (row + k * R < S) {
                    float f[8];
                    x[k].get(f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = act<SILU>(fmaf((f[i] - st[i].x) * st[i].y, w[i], b[i]));
                    OutVec<IO>::store(a.out, base + (size_t)(row + k * R) * width, f);
                }
        }
        __syncthreads();  // the next sample writes what is read above
    }
}

// The gradient reads a sample twice, the second time from the caches: x and dout in registers
// beside the sums would spill.
template <int IO, bool SILU>
__global__ __launch_bounds__(1024) void resident_backward_kernel(GroupNormArgs a, int V, int R, float *part) {
    extern __shared__ float lds[];
    const int row = threadIdx.x / V, col = threadIdx.x % V, C = 8 * V, D = a.C / a.G, S = (int)a.S;
    const int width = a.C / 8;
    to_piece<IO>(a, blockIdx.y, C, C / D);
    const bool on = row < R;
    const int unit = unit_of(D);
    float2 *group = reinterpret_cast<float2 *>(lds + 2 * R * C);
    const float inv = 1.0f / ((float)S * D);
    float w[8], b[8], sw[8] = {}, sb[8] = {};
    if (on) {
        channel8(w, a.weight, col, 1.0f);
        channel8(b, a.bias, col, 0.0f);
    }
    for (long long n = blockIdx.x; n < a.N; n += gridDim.x) {
        const size_t base = (size_t)n * S * width + col;
        float2 st[8];
        if (on) {
#pragma unroll
            for (int i = 0; i < 8; ++i) st[i] = reinterpret_cast<const float2 *>(a.stats)[(size_t)n * a.G + (8 * col + i) / D];
            float s1[8] = {}, s2[8] = {};
#pragma unroll 2
            for (int r = row; r < S; r += R) {
                Vec<IO> x;
                OutVec<IO> y;
                float f[8], t[8];
                x.load(a.x, base + (size_t)r * width);
                y.load(a.dout, base + (size_t)r * width);
                x.get(f);
                y.get(t);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float xh = (f[i] - st[i].x) * st[i].y, dz = act_grad<SILU>(t[i], fmaf(xh, w[i], b[i]));
                    s1[i] += dz;
                    s2[i] = fmaf(dz, xh, s2[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sb[i] += s1[i];
                sw[i] += s2[i];
                s1[i] *= w[i];
                s2[i] *= w[i];
            }
            put_sums(lds, R, C, unit, row, col, s1, s2);
        }
        __syncthreads();
        sum_groups(lds, R, C, D, unit, [&](int g, float s1, float s2) { group[g] = make_float2(s1 * inv, s2 * inv); });
        __syncthreads();
        if (on && a.dx) {
            float2 m[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] = group[(8 * col + i) / D];
#pragma unroll 2
            for (int r = row; r < S; r += R) {
                Vec<IO> x;
                OutVec<IO> y;
                float f[8], t[8];
                x.load(a.x, base + (size_t)r * width);
                y.load(a.dout, base + (size_t)r * width);
                x.get(f);
                y.get(t);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float xh = (f[i] - st[i].x) * st[i].y, dz = act_grad<SILU>(t[i], fmaf(xh, w[i], b[i]));
                    t[i] = st[i].y * (dz * w[i] - m[i].x - xh * m[i].y);
                }
                OutVec<IO>::store(a.dx, base + (size_t)r * width, t);
            }
        }
        __syncthreads();  // the next sample writes what is read above
    }
    if (part) block_channels(sb, sw, lds, part + (size_t)blockIdx.x * 2 * a.C + blockIdx.y * C, a.C, C, row, col, R);
}

// ---- split --------------------------------------------------------------------------

// Stretch j of a sample: rows [j len, min((j + 1) len, S)).
struct Split {
    int count;       // stretches of a sample
    long long len;   // rows of a stretch
};

// Mean and squares of one stretch and group: part[(n count + j) G + g].  grid: count, samples.
// A thread takes its rows ROWS_U at a time, the next ones' loads issued before these are used.
// Up to PIVOT_ROWS rows it sums the distances d from the first of them, p, and their squares:
// p is in the set, so the squares around the set's mean are at least (p - mean)^2, and
// sum d^2 - (sum d)^2 / n loses at most a factor n + 1 <= 33 of the last place.  Four
// operations an element, where squares around running means take ten.
constexpr int PIVOT_ROWS = 32;
template <int IO>
__global__ __launch_bounds__(1024) void split_stats_kernel(GroupNormArgs a, int V, int R, Split sp, long long n0, float2 *part) {
    extern __shared__ float lds[];
    const int row = threadIdx.x / V, col = threadIdx.x % V, C = a.C, D = C / a.G, unit = unit_of(D);
    const long long j = blockIdx.x, n = n0 + blockIdx.y, lo = j * sp.len;
    const int rows = (int)(lo + sp.len < a.S ? sp.len : a.S - lo);
    const Share share(rows, R);
    if (row < R) {
        float mean[8] = {}, sq[8] = {}, p[8] = {}, s[8] = {}, q[8] = {};
        const size_t base = ((size_t)n * a.S + lo) * V + col;
        const int mine = row < rows ? (int)share(row) : 0;  // rows of this thread
        Vec<IO> next[ROWS_U];
        auto load = [&](int k) {  // number k of this thread's rows on; past the end the last again
#pragma unroll
            for (int u = 0; u < ROWS_U; ++u) {
                const int r = row + (k + u < mine ? k + u : mine - 1) * R;
                next[u].load(a.x, base + (size_t)r * V);
            }
        };
        auto join = [&](int before, int now) {  // `now` rows in p, s, q to `before` rows in mean, sq
            const float k = (float)now, each = 1.0f / k, frac = k / (float)(before + now), weight = (float)before * frac;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = s[i] * each, m = p[i] + d, far = m - mean[i];
                sq[i] += fmaf(far * far, weight, fmaxf(fmaf(-s[i], d, q[i]), 0.0f));
                mean[i] = fmaf(far, frac, mean[i]);
                s[i] = q[i] = 0.0f;
            }
        };
        if (mine > 0) load(0);
        int k = 0, from = 0;
        for (; k < mine; k += ROWS_U) {
            float f[ROWS_U][8];
#pragma unroll
            for (int u = 0; u < ROWS_U; ++u) next[u].get(f[u]);
            if (k + ROWS_U < mine) load(k + ROWS_U);
            if (k - from == PIVOT_ROWS) {
                join(from, PIVOT_ROWS);
                from = k;
            }
            if (k == from)
#pragma unroll
                for (int i = 0; i < 8; ++i) p[i] = f[0][i];
#pragma unroll
            for (int u = 0; u < ROWS_U; ++u)
                if (k + u < mine)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float d = f[u][i] - p[i];
                        s[i] += d;
                        q[i] = fmaf(d, d, q[i]);
                    }
        }
        if (mine > 0) join(from, mine - from);
        put_moments(lds, R, C, unit, row, col, (float)mine, mean, sq);
    }
    __syncthreads();
    join_groups(lds, R, C, D, unit, share, (float)rows, [&](int g, float mean, float sq) {
        part[((size_t)blockIdx.y * sp.count + j) * a.G + g] = make_float2(mean, sq);
    });
}

// Sum over the block's 256 threads, in each of them.
__device__ __forceinline__ float block_sum(float x, float (&lds)[4]) {
    x = lanes_sum(x, 64);
    __syncthreads();
    if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = x;
    __syncthreads();
    return lds[0] + lds[1] + lds[2] + lds[3];
}

// Joins a sample's stretches, a block per group and sample: mean, 1 / std.
__global__ __launch_bounds__(256) void split_stats_join_kernel(GroupNormArgs a, Split sp, const float2 *part, float2 *stats) {
    __shared__ float lds[4];
    const int g = blockIdx.x, n = blockIdx.y;
    const float2 *p = part + (size_t)n * sp.count * a.G + g;
    const float D = (float)(a.C / a.G), total = (float)a.S * D, full = (float)sp.len * D;
    const float last = (float)(a.S - (sp.count - 1) * sp.len) * D;
    float s = 0.0f, q = 0.0f;
#pragma unroll 4
    for (int j = threadIdx.x; j < sp.count; j += 256) s = fmaf((j + 1 < sp.count ? full : last) / total, p[(size_t)j * a.G].x, s);
    const float mean = block_sum(s, lds);
#pragma unroll 4
    for (int j = threadIdx.x; j < sp.count; j += 256) {
        const float2 v = p[(size_t)j * a.G];
        q += fmaf((j + 1 < sp.count ? full : last) * (v.x - mean), v.x - mean, v.y);
    }
    q = block_sum(q, lds);
    if (threadIdx.x == 0) stats[(size_t)n * a.G + g] = make_float2(mean, inv_std(q / total, a.eps));
}

// `part`: the stretches are joined here (few of them: each block does so for its sample), the
// first block of a sample writing stats_out; else stats holds the results.
template <int IO, bool SILU>
__global__ __launch_bounds__(1024) void split_apply_kernel(GroupNormArgs a, int V, int R, Split sp, long long n0,
                                                           const float2 *stats, const float2 *part) {
    extern __shared__ float lds[];
    const int row = threadIdx.x / V, col = threadIdx.x % V, D = a.C / a.G;
    const int ny = gridDim.y - 1 - blockIdx.y;
    const long long j = sp.count - 1 - (int)blockIdx.x, n = n0 + ny;
    const long long lo = j * sp.len, hi = lo + sp.len < a.S ? lo + sp.len : a.S;
    stats += (size_t)ny * a.G;
    if (part) {
        float2 *group = reinterpret_cast<float2 *>(lds);
        const float2 *p = part + (size_t)ny * sp.count * a.G;
        const float total = (float)a.S * (float)D, full = (float)sp.len * (float)D;
        const float last = (float)(a.S - (sp.count - 1) * sp.len) * (float)D;
        each_group(a.G, sp.count, [&](int g, int lane, int L) {
            const bool in = g < a.G;
            float s = 0.0f, q = 0.0f;
            for (int k = lane; in && k < sp.count; k += L) s = fmaf((k + 1 < sp.count ? full : last) / total, p[k * a.G + g].x, s);
            const float m = lanes_sum(s, L);
            for (int k = lane; in && k < sp.count; k += L) {
                const float2 v = p[k * a.G + g];
                q += fmaf((k + 1 < sp.count ? full : last) * (v.x - m), v.x - m, v.y);
            }
            q = lanes_sum(q, L);
            if (in && lane == 0) {
                const float2 st = make_float2(m, inv_std(q / total, a.eps));
                group[g] = st;
                if (a.stats_out && blockIdx.x == 0) reinterpret_cast<float2 *>(a.stats_out)[(size_t)n * a.G + g] = st;
            }
        });
        __syncthreads();
        stats = group;
    }
    if (row >= R) return;
    float mean[8], scale[8], b[8];
    channel8(scale, a.weight, col, 1.0f);
    channel8(b, a.bias, col, 0.0f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 st = stats[(8 * col + i) / D];
        mean[i] = st.x;
        scale[i] *= st.y;
    }
    const size_t base = (size_t)n * a.S * V + col;
    for (long long r = lo + row; r < hi; r += ROWS_U * R) {
        Vec<IO> x[ROWS_U];
#pragma unroll
        for (int u = 0; u < ROWS_U; ++u)
            if (r + u * R < hi) x[u].load(a.x, base + (size_t)(r + u * R) * V);
#pragma unroll
        for (int u = 0; u < ROWS_U; ++u)
            if (r + u * R < hi) {
                float f[8];
                x[u].get(f);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = act<SILU>(fmaf(f[i] - mean[i], scale[i], b[i]));
                OutVec<IO>::store(a.out, base + (size_t)(r + u * R) * V, f);
            }
    }
}

// Per channel sums of dz and dz xhat over one stretch: part[(n count + j)][0 .. C) and
// [C .. 2C).  grid: count, samples.
template <int IO, bool SILU>
__global__ __launch_bounds__(1024) void split_sums_kernel(GroupNormArgs a, int V, int R, Split sp, long long n0, float *part) {
    extern __shared__ float lds[];
    const int row = threadIdx.x / V, col = threadIdx.x % V, D = a.C / a.G;
    const long long j = blockIdx.x, n = n0 + blockIdx.y;
    const long long lo = j * sp.len, hi = lo + sp.len < a.S ? lo + sp.len : a.S;
    float s1[8] = {}, s2[8] = {};
    if (row < R) {
        float w[8], b[8];
        float2 st[8];
        channel8(w, a.weight, col, 1.0f);
        channel8(b, a.bias, col, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) st[i] = reinterpret_cast<const float2 *>(a.stats)[(size_t)n * a.G + (8 * col + i) / D];
        const size_t base = (size_t)n * a.S * V + col;
        constexpr int U = ROWS_U / 2;
        for (long long r = lo + row; r < hi; r += U * R) {
            Vec<IO> x[U];
            OutVec<IO> y[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r + u * R < hi) {
                    x[u].load(a.x, base + (size_t)(r + u * R) * V);
                    y[u].load(a.dout, base + (size_t)(r + u * R) * V);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r + u * R < hi) {
                    float f[8], t[8];
                    x[u].get(f);
                    y[u].get(t);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float xh = (f[i] - st[i].x) * st[i].y, dz = act_grad<SILU>(t[i], fmaf(xh, w[i], b[i]));
                        s1[i] += dz;
                        s2[i] = fmaf(dz, xh, s2[i]);
                    }
                }
        }
    }
    block_channels(s1, s2, lds, part + ((size_t)blockIdx.y * sp.count + blockIdx.x) * 2 * a.C, a.C, a.C, row, col, R);
}

template <int IO, bool SILU>
__global__ __launch_bounds__(1024) void split_dx_kernel(GroupNormArgs a, int V, int R, Split sp, long long n0,
                                                        const float *chan) {
    extern __shared__ float lds[];
    const int row = threadIdx.x / V, col = threadIdx.x % V, C = a.C, D = C / a.G;
    const int ny = gridDim.y - 1 - blockIdx.y;
    const long long j = sp.count - 1 - (int)blockIdx.x, n = n0 + ny;
    const long long lo = j * sp.len, hi = lo + sp.len < a.S ? lo + sp.len : a.S;
    // the means of w dz and w dz xhat over each group, from the sums per channel
    float2 *group = reinterpret_cast<float2 *>(lds + 2 * C);
    const float inv = 1.0f / ((float)a.S * D);
    for (int c = threadIdx.x; c < 2 * C; c += blockDim.x)
        lds[c] = chan[(size_t)ny * 2 * C + c] * (a.weight ? a.weight[c < C ? c : c - C] : 1.0f);
    __syncthreads();
    sum_groups(lds, 1, C, D, 1, [&](int g, float s1, float s2) { group[g] = make_float2(s1 * inv, s2 * inv); });
    __syncthreads();
    if (row >= R) return;
    float w[8], b[8];
    float2 st[8], m[8];
    channel8(w, a.weight, col, 1.0f);
    channel8(b, a.bias, col, 0.0f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        st[i] = reinterpret_cast<const float2 *>(a.stats)[(size_t)n * a.G + (8 * col + i) / D];
        m[i] = group[(8 * col + i) / D];
    }
    const size_t base = (size_t)n * a.S * V + col;
    constexpr int U = ROWS_U / 2;
    for (long long r = lo + row; r < hi; r += U * R) {
        Vec<IO> x[U];
        OutVec<IO> y[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (r + u * R < hi) {
                x[u].load(a.x, base + (size_t)(r + u * R) * V);
                y[u].load(a.dout, base + (size_t)(r + u * R) * V);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (r + u * R < hi) {
                float f[8], t[8];
                x[u].get(f);
                y[u].get(t);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float xh = (f[i] - st[i].x) * st[i].y, dz = act_grad<SILU>(t[i], fmaf(xh, w[i], b[i]));
                    t[i] = st[i].y * (dz * w[i] - m[i].x - xh * m[i].y);
                }
                OutVec<IO>::store(a.dx, base + (size_t)(r + u * R) * V, t);
            }
    }
}

// Sums of the rows of part [samples][rows][2][C] per channel.  Block row y < samples: the rows
// of sample y, to chan[y][2][C].  The last block row (`whole`): all rows, to dbias and dweight
// (either may be nullptr), added to what is there if `add`.  A block has 32 of the 2 C columns
// by 32 rows of threads.
__global__ __launch_bounds__(1024) void channels_kernel(const float *part, int samples, int rows, int C, float *chan, bool whole,
                                                        float *dbias, float *dweight, bool add) {
    __shared__ float lds[32][33];
    const int tc = threadIdx.x % 32, tr = threadIdx.x / 32, k = blockIdx.x * 32 + tc, y = blockIdx.y;
    const bool all = whole && y + 1 == (int)gridDim.y;
    const size_t lo = all ? 0 : (size_t)y * rows, hi = all ? (size_t)samples * rows : lo + rows;
    float s = 0.0f;
    if (k < 2 * C)
#pragma unroll 8
        for (size_t r = lo + tr; r < hi; r += 32) s += part[r * 2 * C + k];
    lds[tr][tc] = s;
    __syncthreads();
    // column tr, its 32 partial sums across half a wave
    s = lds[tc][tr];
    for (int l = 16; l > 0; l /= 2) s += __shfl_xor(s, l);
    const int c = blockIdx.x * 32 + tr;
    if (tc == 0 && c < 2 * C) {
        if (!all) {
            chan[(size_t)y * 2 * C + c] = s;
        } else if (float *to = c < C ? dbias : dweight) {
            to += c < C ? c : c - C;
            *to = (add ? *to : 0.0f) + s;
        }
    }
}

// ---- host ---------------------------------------------------------------------------

// Threads and rows of a block: whole waves that hold at least one row.
struct Layout {
    int V, R, threads;
};
Layout layout(int C, int at_least) {
    Layout l;
    l.V = C / 8;
    l.threads = std::max(at_least, (l.V + 63) / 64 * 64);
    l.R = l.threads / l.V;
    return l;
}

// Lanes of a group in the rows form: the power of two from D / 8 on; 0 where the form does not
// apply.
int rows_lanes(const GroupNormArgs &a) {
    const int D = a.C / a.G, P = D / 8;
    if (a.S != 1 || D % 8 || P > 64) return 0;
    int L = 1;
    while (L < P) L *= 2;
    return a.G * L <= 512 ? L : 0;
}
Layout rows_layout(const GroupNormArgs &a, int L) {
    Layout l;
    l.V = a.C / 8;
    l.threads = std::max(256, (a.G * L + 63) / 64 * 64);
    l.R = l.threads / (a.G * L);
    return l;
}

// Pieces of a sample in the resident form, which takes blocks of their own: whole groups and
// vectors, as many as even parts of at least PIECE vectors (128 bytes of fp32) allow while
// samples alone leave CUs idle.
constexpr int PIECE = 4, WIDE = 128;
int pieces(const GroupNormArgs &a) {
    const int V = a.C / 8, D = a.C / a.G, parts = V / (D / std::gcd(D, 8));  // of whole groups and vectors
    int p = (int)std::min<long long>({parts, V / PIECE, a.ncu / std::max<long long>(a.N, 1)});
    while (p > 1 && parts % p) --p;
    return std::max(p, 1);
}

// At most RES_K rows of a thread.  What fits is faster here than split even if a sample is
// alone in one piece, and faster in pieces (3 x 77 x 320 fp32, forward and backward: 17 us in 8
// pieces, 25 whole; 8 x 200 x 1280 in 32 pieces 27 us, split 39; forward only, 1 x 800 x 512 in
// 16 pieces 9.6 us, split 12.3).  The gradient's two passes of few blocks take longer than the
// split form's many: beyond whole samples that fit and half a row a thread it wants most CUs
// busy, or rows so wide that a split block has one or two at a time (3 x 400 x 320: in pieces
// 18 us, split 14; 8 x 400 x 1280: 20 us, split 29; 2 x 77 x 4096: 14 us, split 23).
bool resident_form(const GroupNormArgs &a, int p, bool gradient) {
    const int V = a.C / 8;
    if (a.S > RES_K * (1024 / (V / p))) return false;
    return !gradient || a.S <= RES_K * (1024 / V) || a.S * (V / p) <= 512 || V >= WIDE ||
           4 * p * a.N >= 3LL * a.ncu;
}

// Threads of the resident form for rows of V vectors: few for small samples, RES_K vectors each
// for large ones.
Layout resident_layout(const GroupNormArgs &a, int V) {
    const long long vectors = a.S * V;
    long long t = std::max<long long>(64, std::min<long long>(1024, (vectors + 63) / 64 * 64));
    Layout l = layout(8 * V, (int)t);
    while ((long long)l.R * RES_K < a.S) l = layout(8 * V, l.threads + 64);  // a row's width may not divide
    return l;
}

// Blocks of about 16 waves a CU in all.
int blocks_for(int ncu, int threads) { return std::max(1, 16 * ncu * 64 / threads); }

Split split_for(const GroupNormArgs &a, const Layout &l, long long samples) {
    const long long want = std::max<long long>(1, (blocks_for(a.ncu, l.threads) + samples - 1) / samples);
    const long long least = (long long)l.R * ROWS_U;  // rows of a round: stretches are whole rounds
    Split s;
    s.len = (std::max(least, (a.S + want - 1) / want) + least - 1) / least * least;
    s.count = (int)((a.S + s.len - 1) / s.len);
    return s;
}

// Wide rows with many groups need more dynamic LDS than a launch gets unasked.
hipError_t allow_lds(const void *kernel, size_t bytes) {
    return bytes <= 64 * 1024 ? hipSuccess
                              : hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

size_t aligned(size_t n) { return (n + 255) / 256 * 256; }
constexpr int MAX_NCU = 512;  // sizes the workspace; gfx950 devices have 256

// The workspace: partial sums (the rows of blocks or stretches), then sums per sample and
// channel, then results per sample and group.
struct Work {
    float *part, *chan;
    float2 *group;
};
size_t part_bytes(int C, long long samples) {
    const int threads = std::max(64, (C / 8 + 63) / 64 * 64);
    return aligned(((size_t)blocks_for(MAX_NCU, threads) + samples) * 2 * C * sizeof(float));
}
Work work_of(const GroupNormArgs &a) {
    const long long samples = std::min<long long>(a.max_N, BATCH);
    Work w;
    w.part = static_cast<float *>(a.work);
    w.chan = reinterpret_cast<float *>(static_cast<char *>(a.work) + part_bytes(a.C, samples));
    w.group = reinterpret_cast<float2 *>(reinterpret_cast<char *>(w.chan) + aligned((size_t)samples * 2 * a.C * sizeof(float)));
    return w;
}

template <int IO, bool SILU>
hipError_t forward(const GroupNormArgs &a, hipStream_t s) {
    if (const int L = rows_lanes(a)) {
        const Layout l = rows_layout(a, L);
        // 24 waves a CU, where 16 to 20 fit at once: at 65,520 x 4096 in bf16 16 waves are 9%
        // slower, 64 or 128 waves 5 to 7%
        const long long blocks = std::min<long long>((a.N + l.R - 1) / l.R, blocks_for(a.ncu, l.threads) * 3 / 2);
        rows_forward_kernel<IO, SILU><<<dim3((unsigned)blocks), dim3(l.threads), 0, s>>>(a, l.V, l.R, L);
        return hipGetLastError();
    }
    if (const int p = pieces(a); resident_form(a, p, false)) {
        const Layout l = resident_layout(a, a.C / 8 / p);
        const size_t lds = (2 * (size_t)l.R * 8 * l.V + 2 * (a.G / p)) * sizeof(float);
        const long long blocks = std::min<long long>(a.N, 1 << 20);
        const hipError_t e = allow_lds(reinterpret_cast<const void *>(&resident_forward_kernel<IO, SILU>), lds);
        if (e != hipSuccess) return e;
        resident_forward_kernel<IO, SILU><<<dim3((unsigned)blocks, p), dim3(l.threads), lds, s>>>(a, l.V, l.R);
        return hipGetLastError();
    }
    const Layout l = layout(a.C, 256);
    const size_t lds = 2 * (size_t)l.R * a.C * sizeof(float);
    const Work w = work_of(a);
    for (long long n0 = 0; n0 < a.N; n0 += BATCH) {
        const int samples = (int)std::min<long long>(BATCH, a.N - n0);
        const Split sp = split_for(a, l, samples);
        const dim3 grid(sp.count, samples), block(l.threads);
        float2 *stats = a.stats_out ? reinterpret_cast<float2 *>(a.stats_out) + n0 * a.G : w.group;
        split_stats_kernel<IO><<<grid, block, lds, s>>>(a, l.V, l.R, sp, n0, reinterpret_cast<float2 *>(w.part));
        const float2 *part = reinterpret_cast<const float2 *>(w.part);
        if (sp.count * a.G <= JOIN_HERE) {
            split_apply_kernel<IO, SILU><<<grid, block, a.G * sizeof(float2), s>>>(a, l.V, l.R, sp, n0, stats, part);
        } else {
            split_stats_join_kernel<<<dim3(a.G, samples), dim3(256), 0, s>>>(a, sp, part, stats);
            split_apply_kernel<IO, SILU><<<grid, block, 0, s>>>(a, l.V, l.R, sp, n0, stats, nullptr);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// dbias and dweight from `rows` rows of sums.
hipError_t channels(const GroupNormArgs &a, const float *part, int rows, hipStream_t s) {
    channels_kernel<<<dim3((2 * a.C + 31) / 32), dim3(1024), 0, s>>>(part, 1, rows, a.C, nullptr, true, a.dbias, a.dweight, false);
    return hipGetLastError();
}

template <int IO, bool SILU>
hipError_t backward(const GroupNormArgs &a, hipStream_t s) {
    const bool wanted = a.dweight || a.dbias;
    const Work w = work_of(a);
    if (a.N * a.S == 0) return wanted ? channels(a, w.part, 0, s) : hipSuccess;
    if (const int L = rows_lanes(a)) {
        const Layout l = rows_layout(a, L);
        const int blocks = (int)std::min<long long>((a.N + l.R - 1) / l.R, blocks_for(a.ncu, l.threads));
        rows_backward_kernel<IO, SILU><<<dim3(blocks), dim3(l.threads), (size_t)l.R * a.C * sizeof(float), s>>>(
            a, l.V, l.R, L, wanted ? w.part : nullptr);
        return wanted ? channels(a, w.part, blocks, s) : hipGetLastError();
    }
    if (const int p = pieces(a); resident_form(a, p, true)) {
        const Layout l = resident_layout(a, a.C / 8 / p);
        const size_t lds = (2 * (size_t)l.R * 8 * l.V + 2 * (a.G / p)) * sizeof(float);
        const int blocks = (int)std::min<long long>(a.N, blocks_for(a.ncu, l.threads));
        const hipError_t e = allow_lds(reinterpret_cast<const void *>(&resident_backward_kernel<IO, SILU>), lds);
        if (e != hipSuccess) return e;
        resident_backward_kernel<IO, SILU><<<dim3(blocks, p), dim3(l.threads), lds, s>>>(a, l.V, l.R, wanted ? w.part : nullptr);
        return wanted ? channels(a, w.part, blocks, s) : hipGetLastError();
    }
    const Layout l = layout(a.C, 256);
    const size_t lds = (size_t)l.R * a.C * sizeof(float);
    const size_t dx_lds = (2 * (size_t)a.C + 2 * a.G) * sizeof(float);
    if (const hipError_t e = allow_lds(reinterpret_cast<const void *>(&split_dx_kernel<IO, SILU>), dx_lds)) return e;
    for (long long n0 = 0; n0 < a.N; n0 += BATCH) {
        const int samples = (int)std::min<long long>(BATCH, a.N - n0);
        const Split sp = split_for(a, l, samples);
        const dim3 grid(sp.count, samples), block(l.threads);
        split_sums_kernel<IO, SILU><<<grid, block, lds, s>>>(a, l.V, l.R, sp, n0, w.part);
        channels_kernel<<<dim3((2 * a.C + 31) / 32, samples + wanted), dim3(1024), 0, s>>>(
            w.part, samples, sp.count, a.C, w.chan, wanted, a.dbias, a.dweight, n0 > 0);
        if (a.dx) split_dx_kernel<IO, SILU><<<grid, block, dx_lds, s>>>(a, l.V, l.R, sp, n0, w.chan);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

#define GROUP_NORM_DISPATCH(f)                                                                      \
    if (a.io == IO_F32) return a.silu ? f<IO_F32, true>(a, s) : f<IO_F32, false>(a, s);             \
    if (a.io == IO_BF16) return a.silu ? f<IO_BF16, true>(a, s) : f<IO_BF16, false>(a, s);          \
    return a.silu ? f<IO_FP8, true>(a, s) : f<IO_FP8, false>(a, s);

}  // namespace

size_t group_norm_work_bytes(int C, int G, long long max_N) {
    const long long samples = std::min<long long>(max_N, BATCH);
    return part_bytes(C, samples) + aligned((size_t)samples * 2 * C * sizeof(float)) + aligned((size_t)samples * G * sizeof(float2));
}

hipError_t launch_group_norm_forward(const GroupNormArgs &a, hipStream_t s) { GROUP_NORM_DISPATCH(forward) }
hipError_t launch_group_norm_backward(const GroupNormArgs &a, hipStream_t s) { GROUP_NORM_DISPATCH(backward) }

}  // namespace gdn
