// gdn_group_norm.hip -- group norm with an activation, channels last, and its gradient
// (include/gdn.h, gdn_group_norm_forward / gdn_group_norm_backward).
//
// All forms are bound by HBM.  A thread holds eight neighbouring channels (a 16-byte vector
// in bf16) and a fixed place in the row, so that weight and bias stay in registers; V = C / 8
// threads make a row, and a block has R = threads / V rows at once.  Three forms by the size
// of a sample:
//  * rows (S = 1, D = C / G channels of a group, D / 8 a power of two up to 64): a group is
//    D / 8 lanes of a wave; its sums are exchanges between lanes and the row is read once.
//  * resident (samples of up to RES_K vectors for each of 1024 threads): a block holds a
//    sample in registers and joins its groups through LDS; one read, one launch.
//  * split (larger samples): a sample is cut into stretches of rows.  One launch forms each
//    stretch's sums, a small one joins them, one applies them, taking the stretches in the
//    opposite order so that what the first left in the caches is read from there.
// Squares are always taken around a mean: a thread's few rows around their own, and partial
// results (count, mean, squares around it) are joined by
//     mean = sum n_i mean_i / n,   squares = sum squares_i + sum n_i (mean_i - mean)^2,
// so that means far from zero cost no precision.  Everything is fp32 until the last rounding.
#include "gdn_elem.h"
#include "gdn_layer.h"

#include <algorithm>

namespace gdn {
namespace {

constexpr int RES_K = 4;        // vectors of a thread in the resident form
constexpr int ROWS_U = 4;       // rows a thread of the other forms has in flight
constexpr int BATCH = 1024;     // samples of one round of the split form (bounds the workspace)

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

__device__ __forceinline__ float inv_std(float var, float eps) { return 1.0f / sqrtf(var + eps); }

// ---- rows ---------------------------------------------------------------------------

template <int IO, bool SILU>
__global__ __launch_bounds__(512) void rows_forward_kernel(GroupNormArgs a, int V, int R) {
    const int row = threadIdx.x / V, col = threadIdx.x % V, P = a.C / a.G / 8;
    const bool on = row < R;
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
            if (on && n < a.N) x[u].load(a.x, (size_t)n * V + col);
        }
#pragma unroll
        for (int u = 0; u < ROWS_U; ++u) {
            const long long n = n0 + u * step + row;
            float f[8], s = 0.0f, q = 0.0f;
            x[u].get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) s += f[i];
            const float mean = lanes_sum(s, P) * inv;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[i] -= mean;
                q = fmaf(f[i], f[i], q);
            }
            const float rstd = inv_std(lanes_sum(q, P) * inv, a.eps);
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

// Sums of a block's rows per channel: part[blockIdx.x][0 .. C) gets s1, [C .. 2C) s2.
__device__ __forceinline__ void block_channels(const float (&s1)[8], const float (&s2)[8], float *lds, float *part, int C,
                                               int row, int col, int R) {
    for (int k = 0; k < 2; ++k) {
        if (row < R)
#pragma unroll
            for (int i = 0; i < 8; ++i) lds[row * C + 8 * col + i] = k ? s2[i] : s1[i];
        __syncthreads();
        for (int c = threadIdx.x; c < C; c += blockDim.x) {
            float s = lds[c];
            for (int r = 1; r < R; ++r) s += lds[r * C + c];
            part[(size_t)blockIdx.x * 2 * C + k * C + c] = s;
        }
        __syncthreads();
    }
}

template <int IO, bool SILU>
__global__ __launch_bounds__(512) void rows_backward_kernel(GroupNormArgs a, int V, int R, float *part) {
    extern __shared__ float lds[];
    const int row = threadIdx.x / V, col = threadIdx.x % V, P = a.C / a.G / 8;
    const bool on = row < R;
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
            if (on && n < a.N) {
                x[u].load(a.x, (size_t)n * V + col);
                y[u].load(a.dout, (size_t)n * V + col);
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
            const float m1 = lanes_sum(s1, P) * inv, m2 = lanes_sum(s2, P) * inv;
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = st[u].y * (t[i] - m1 - f[i] * m2);
            if (in && a.dx) OutVec<IO>::store(a.dx, (size_t)n * V + col, t);
        }
    }
    if (part) block_channels(sb, sw, lds, part, a.C, row, col, R);
}

// ---- joining a block's threads by group ---------------------------------------------

// lds: R rows of C means, then R rows of C squares around them, of cnt(row) values each.  For
// every group g calls done(g, count, mean, squares) (count: of `rows` rows) in one lane.  Several groups share a wave
// where they are small.
template <typename Count, typename Done>
__device__ __forceinline__ void join_groups(const float *lds, int R, int C, int D, int rows, Count cnt, Done done) {
    const float *mean = lds, *sq = lds + R * C;
    const int items = R * D, G = C / D;
    int L = 1;
    while (L < 64 && L < items) L *= 2;
    const int lane = threadIdx.x % L, per = blockDim.x / L;
    const float total = (float)rows * (float)D;
    for (int g0 = 0; g0 < G; g0 += per) {  // every lane of a wave stays for the exchanges
        const int g = g0 + (int)threadIdx.x / L;
        const int at = (g < G ? g : 0) * D;
        float s = 0.0f, q = 0.0f;
        for (int i = lane; i < items; i += L) s = fmaf(cnt(i / D), mean[i / D * C + at + i % D], s);
        const float m = lanes_sum(s, L) / total;
        for (int i = lane; i < items; i += L) {
            const int k = i / D * C + at + i % D;
            const float d = mean[k] - m;
            q += fmaf(cnt(i / D) * d, d, sq[k]);
        }
        q = lanes_sum(q, L);
        if (g < G && lane == 0) done(g, total, m, q);
    }
}

// ---- resident -----------------------------------------------------------------------

// A block takes samples blockIdx.x, + gridDim.x, ...; thread (row, col) has rows row + k R.
// LDS: 2 R C floats for joining, then 2 G for the groups' results.
template <int IO, bool SILU>
__global__ __launch_bounds__(1024) void resident_forward_kernel(GroupNormArgs a, int V, int R) {
    extern __shared__ float lds[];
    const int row = threadIdx.x / V, col = threadIdx.x % V, C = a.C, D = C / a.G, S = (int)a.S;
    const bool on = row < R;
    float2 *group = reinterpret_cast<float2 *>(lds + 2 * R * C);
    auto cnt = [&](int r) { return (float)(r < S ? (S - r + R - 1) / R : 0); };
    for (long long n = blockIdx.x; n < a.N; n += gridDim.x) {
        Vec<IO> x[RES_K];
        const size_t base = (size_t)n * S * V + col;
#pragma unroll
        for (int k = 0; k < RES_K; ++k)
            if (on && row + k * R < S) x[k].load(a.x, base + (size_t)(row + k * R) * V);
        if (on) {
            float mean[8] = {}, sq[8] = {};
            const float inv = row < S ? 1.0f / cnt(row) : 0.0f;
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
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                lds[row * C + 8 * col + i] = mean[i];
                lds[(R + row) * C + 8 * col + i] = sq[i];
            }
        }
        __syncthreads();
        join_groups(lds, R, C, D, S, cnt, [&](int g, float total, float mean, float sq) {
            const float2 st = make_float2(mean, inv_std(sq / total, a.eps));
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
                    OutVec<IO>::store(a.out, base + (size_t)(row + k * R) * V, f);
                }
        }
        __syncthreads();  // the next sample writes what is read above
    }
}

// Sums over the rows and over a group's channels of two per-channel values: lds holds R rows
// of C first values, then R rows of second ones; done(g, sum1, sum2) in one lane each.
template <typename Done>
__device__ __forceinline__ void sum_groups(const float *lds, int R, int C, int D, Done done) {
    const int items = R * D, G = C / D;
    int L = 1;
    while (L < 64 && L < items) L *= 2;
    const int lane = threadIdx.x % L, per = blockDim.x / L;
    for (int g0 = 0; g0 < G; g0 += per) {
        const int g = g0 + (int)threadIdx.x / L;
        const int at = (g < G ? g : 0) * D;
        float s1 = 0.0f, s2 = 0.0f;
        for (int i = lane; i < items; i += L) {
            s1 += lds[i / D * C + at + i % D];
            s2 += lds[(R + i / D) * C + at + i % D];
        }
        s1 = lanes_sum(s1, L);
        s2 = lanes_sum(s2, L);
        if (g < G && lane == 0) done(g, s1, s2);
    }
}

template <int IO, bool SILU>
__global__ __launch_bounds__(1024) void resident_backward_kernel(GroupNormArgs a, int V, int R, float *part) {
    extern __shared__ float lds[];
    const int row = threadIdx.x / V, col = threadIdx.x % V, C = a.C, D = C / a.G, S = (int)a.S;
    const bool on = row < R;
    float2 *group = reinterpret_cast<float2 *>(lds + 2 * R * C);
    const float inv = 1.0f / ((float)S * D);
    float w[8], b[8], sw[8] = {}, sb[8] = {};
    if (on) {
        channel8(w, a.weight, col, 1.0f);
        channel8(b, a.bias, col, 0.0f);
    }
    for (long long n = blockIdx.x; n < a.N; n += gridDim.x) {
        Vec<IO> x[RES_K];
        OutVec<IO> y[RES_K];
        const size_t base = (size_t)n * S * V + col;
        float2 st[8];
        if (on) {
#pragma unroll
            for (int k = 0; k < RES_K; ++k)
                if (row + k * R < S) {
                    x[k].load(a.x, base + (size_t)(row + k * R) * V);
                    y[k].load(a.dout, base + (size_t)(row + k * R) * V);
                }
#pragma unroll
            for (int i = 0; i < 8; ++i) st[i] = reinterpret_cast<const float2 *>(a.stats)[(size_t)n * a.G + (8 * col + i) / D];
            float s1[8] = {}, s2[8] = {};
#pragma unroll
            for (int k = 0; k < RES_K; ++k)
                if (row + k * R < S) {
                    float f[8], t[8];
                    x[k].get(f);
                    y[k].get(t);
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
                lds[row * C + 8 * col + i] = s1[i] * w[i];
                lds[(R + row) * C + 8 * col + i] = s2[i] * w[i];
            }
        }
        __syncthreads();
        sum_groups(lds, R, C, D, [&](int g, float s1, float s2) { group[g] = make_float2(s1 * inv, s2 * inv); });
        __syncthreads();
        if (on && a.dx)
#pragma unroll
            for (int k = 0; k < RES_K; ++k)
                if (row + k * R < S) {
                    float f[8], t[8];
                    x[k].get(f);
                    y[k].get(t);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 m = group[(8 * col + i) / D];
                        const float xh = (f[i] - st[i].x) * st[i].y, dz = act_grad<SILU>(t[i], fmaf(xh, w[i], b[i]));
                        t[i] = st[i].y * (dz * w[i] - m.x - xh * m.y);
                    }
                    OutVec<IO>::store(a.dx, base + (size_t)(row + k * R) * V, t);
                }
        __syncthreads();
    }
    if (part) block_channels(sb, sw, lds, part, C, row, col, R);
}

// ---- split --------------------------------------------------------------------------

// Stretch j of a sample: rows [j len, min((j + 1) len, S)).
struct Split {
    int count;       // stretches of a sample
    long long len;   // rows of a stretch
};

// Mean and squares of one stretch and group: part[(n count + j) G + g].  grid: count, samples.
template <int IO>
__global__ __launch_bounds__(1024) void split_stats_kernel(GroupNormArgs a, int V, int R, Split sp, long long n0, float2 *part) {
    extern __shared__ float lds[];
    const int row = threadIdx.x / V, col = threadIdx.x % V, C = a.C;
    const long long j = blockIdx.x, n = n0 + blockIdx.y;
    const long long lo = j * sp.len, hi = lo + sp.len < a.S ? lo + sp.len : a.S;
    if (row < R) {
        float mean[8] = {}, sq[8] = {}, have = 0.0f;
        const size_t base = (size_t)n * a.S * V + col;
        long long r = lo + row;
        // chunks of ROWS_U rows: around their own mean, then joined to those before
        for (; r + (ROWS_U - 1) * R < hi; r += ROWS_U * R) {
            Vec<IO> x[ROWS_U];
#pragma unroll
            for (int u = 0; u < ROWS_U; ++u) x[u].load(a.x, base + (size_t)(r + u * R) * V);
            float f[ROWS_U][8];
#pragma unroll
            for (int u = 0; u < ROWS_U; ++u) x[u].get(f[u]);
            const float share = (float)ROWS_U / (have + ROWS_U), weight = have * share;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float m = 0.0f, q = 0.0f;
#pragma unroll
                for (int u = 0; u < ROWS_U; ++u) m += f[u][i];
                m *= 1.0f / ROWS_U;
#pragma unroll
                for (int u = 0; u < ROWS_U; ++u) q = fmaf(f[u][i] - m, f[u][i] - m, q);
                const float d = m - mean[i];
                mean[i] = fmaf(d, share, mean[i]);
                sq[i] += fmaf(d * d, weight, q);
            }
            have += ROWS_U;
        }
        for (; r < hi; r += R) {
            Vec<IO> x;
            float f[8];
            x.load(a.x, base + (size_t)r * V);
            x.get(f);
            const float share = 1.0f / (have + 1.0f), weight = have * share;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = f[i] - mean[i];
                mean[i] = fmaf(d, share, mean[i]);
                sq[i] = fmaf(d * d, weight, sq[i]);
            }
            have += 1.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lds[row * C + 8 * col + i] = mean[i];
            lds[(R + row) * C + 8 * col + i] = sq[i];
        }
    }
    __syncthreads();
    const int rows = (int)(hi - lo);
    join_groups(lds, R, C, C / a.G, rows, [&](int r) { return (float)(r < rows ? (rows - r + R - 1) / R : 0); },
                [&](int g, float, float mean, float sq) {
                    part[((size_t)blockIdx.y * sp.count + j) * a.G + g] = make_float2(mean, sq);
                });
}

// Joins a sample's stretches, a wave per sample and group: mean, 1 / std.
__global__ __launch_bounds__(256) void split_stats_join_kernel(GroupNormArgs a, Split sp, int samples,
                                                               const float2 *part, float2 *stats) {
    const int lane = threadIdx.x % 64, D = a.C / a.G;
    const long long id = (long long)blockIdx.x * 4 + threadIdx.x / 64;
    if (id >= (long long)samples * a.G) return;
    const int n = (int)(id / a.G), g = (int)(id % a.G);
    const float2 *p = part + (size_t)n * sp.count * a.G + g;
    const float total = (float)a.S * D;
    auto cnt = [&](int j) { return (float)D * (float)(j + 1 < sp.count ? sp.len : a.S - j * sp.len); };
    float s = 0.0f, q = 0.0f;
    for (int j = lane; j < sp.count; j += 64) s = fmaf(cnt(j) / total, p[(size_t)j * a.G].x, s);
    const float mean = lanes_sum(s, 64);
    for (int j = lane; j < sp.count; j += 64) {
        const float2 v = p[(size_t)j * a.G];
        q += fmaf(cnt(j) * (v.x - mean), v.x - mean, v.y);
    }
    q = lanes_sum(q, 64);
    if (lane == 0) stats[(size_t)n * a.G + g] = make_float2(mean, inv_std(q / total, a.eps));
}

template <int IO, bool SILU>
__global__ __launch_bounds__(1024) void split_apply_kernel(GroupNormArgs a, int V, int R, Split sp, long long n0,
                                                           const float2 *stats) {
    const int row = threadIdx.x / V, col = threadIdx.x % V, D = a.C / a.G;
    if (row >= R) return;
    const int ny = gridDim.y - 1 - blockIdx.y;
    const long long j = sp.count - 1 - (int)blockIdx.x, n = n0 + ny;
    const long long lo = j * sp.len, hi = lo + sp.len < a.S ? lo + sp.len : a.S;
    float mean[8], scale[8], b[8];
    channel8(scale, a.weight, col, 1.0f);
    channel8(b, a.bias, col, 0.0f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 st = stats[(size_t)ny * a.G + (8 * col + i) / D];
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
    block_channels(s1, s2, lds, part + (size_t)blockIdx.y * sp.count * 2 * a.C, a.C, row, col, R);
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
    sum_groups(lds, 1, C, D, [&](int g, float s1, float s2) { group[g] = make_float2(s1 * inv, s2 * inv); });
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

// Sums of the `rows` rows of part[blockIdx.y][rows][2][C] per channel: to[blockIdx.y][0 .. C)
// first values and more[blockIdx.y][0 .. C) second ones (either may be nullptr), added to what
// is there if `add`.  A block has 32 of the 2 C columns by 32 rows of threads.
__global__ __launch_bounds__(1024) void channels_kernel(const float *part, int rows, int C, size_t pitch, float *first,
                                                        float *second, int add) {
    __shared__ float lds[32][33];
    const int tc = threadIdx.x % 32, tr = threadIdx.x / 32, k = blockIdx.x * 32 + tc;
    part += (size_t)blockIdx.y * rows * 2 * C;
    float s = 0.0f;
    if (k < 2 * C)
        for (int r = tr; r < rows; r += 32) s += part[(size_t)r * 2 * C + k];
    lds[tr][tc] = s;
    __syncthreads();
    // column tr, its 32 partial sums across half a wave
    s = lds[tc][tr];
    for (int l = 16; l > 0; l /= 2) s += __shfl_xor(s, l);
    const int c = blockIdx.x * 32 + tr;
    if (tc == 0 && c < 2 * C) {
        float *to = c < C ? first : second;
        if (to) {
            to += blockIdx.y * pitch + (c < C ? c : c - C);
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

bool rows_form(const GroupNormArgs &a) {
    const int D = a.C / a.G, P = D / 8;
    return a.S == 1 && D % 8 == 0 && (P & (P - 1)) == 0 && P <= 64 && a.C / 8 <= 512;
}
bool resident_form(const GroupNormArgs &a) { return a.S <= RES_K * (1024 / (a.C / 8)); }

// Threads of the resident form: few for small samples, RES_K vectors each for large ones.
Layout resident_layout(const GroupNormArgs &a) {
    const long long vectors = a.S * (a.C / 8);
    long long t = std::max<long long>(64, std::min<long long>(1024, (vectors + 63) / 64 * 64));
    Layout l = layout(a.C, (int)t);
    while ((long long)l.R * RES_K < a.S) l = layout(a.C, l.threads + 64);  // a row's width may not divide
    return l;
}

// Blocks of about 16 waves a CU in all.
int blocks_for(int ncu, int threads) { return std::max(1, 16 * ncu * 64 / threads); }

Split split_for(const GroupNormArgs &a, const Layout &l, long long samples) {
    const long long want = std::max<long long>(1, (blocks_for(a.ncu, l.threads) + samples - 1) / samples);
    const long long least = (long long)l.R * ROWS_U;  // rows worth a block
    Split s;
    s.len = std::max(least, (a.S + want - 1) / want);
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
    if (rows_form(a)) {
        const Layout l = layout(a.C, 256);
        const long long blocks = std::min<long long>((a.N + l.R - 1) / l.R, blocks_for(a.ncu, l.threads));
        rows_forward_kernel<IO, SILU><<<dim3((unsigned)blocks), dim3(l.threads), 0, s>>>(a, l.V, l.R);
        return hipGetLastError();
    }
    if (resident_form(a)) {
        const Layout l = resident_layout(a);
        const size_t lds = (2 * (size_t)l.R * a.C + 2 * a.G) * sizeof(float);
        const long long blocks = std::min<long long>(a.N, 1 << 20);
        const hipError_t e = allow_lds(reinterpret_cast<const void *>(&resident_forward_kernel<IO, SILU>), lds);
        if (e != hipSuccess) return e;
        resident_forward_kernel<IO, SILU><<<dim3((unsigned)blocks), dim3(l.threads), lds, s>>>(a, l.V, l.R);
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
        split_stats_join_kernel<<<dim3((unsigned)(((long long)samples * a.G + 3) / 4)), dim3(256), 0, s>>>(
            a, sp, samples, reinterpret_cast<const float2 *>(w.part), stats);
        split_apply_kernel<IO, SILU><<<grid, block, 0, s>>>(a, l.V, l.R, sp, n0, stats);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// dbias and dweight from `rows` rows of sums.
hipError_t channels(const GroupNormArgs &a, const float *part, int rows, bool add, hipStream_t s) {
    channels_kernel<<<dim3((2 * a.C + 31) / 32), dim3(1024), 0, s>>>(part, rows, a.C, 0, a.dbias, a.dweight, add);
    return hipGetLastError();
}

template <int IO, bool SILU>
hipError_t backward(const GroupNormArgs &a, hipStream_t s) {
    const bool wanted = a.dweight || a.dbias;
    const Work w = work_of(a);
    if (a.N * a.S == 0) return wanted ? channels(a, w.part, 0, false, s) : hipSuccess;
    if (rows_form(a)) {
        const Layout l = layout(a.C, 256);
        const int blocks = (int)std::min<long long>((a.N + l.R - 1) / l.R, blocks_for(a.ncu, l.threads));
        rows_backward_kernel<IO, SILU><<<dim3(blocks), dim3(l.threads), (size_t)l.R * a.C * sizeof(float), s>>>(
            a, l.V, l.R, wanted ? w.part : nullptr);
        return wanted ? channels(a, w.part, blocks, false, s) : hipGetLastError();
    }
    if (resident_form(a)) {
        const Layout l = resident_layout(a);
        const size_t lds = (2 * (size_t)l.R * a.C + 2 * a.G) * sizeof(float);
        const int blocks = (int)std::min<long long>(a.N, blocks_for(a.ncu, l.threads));
        const hipError_t e = allow_lds(reinterpret_cast<const void *>(&resident_backward_kernel<IO, SILU>), lds);
        if (e != hipSuccess) return e;
        resident_backward_kernel<IO, SILU><<<dim3(blocks), dim3(l.threads), lds, s>>>(a, l.V, l.R, wanted ? w.part : nullptr);
        return wanted ? channels(a, w.part, blocks, false, s) : hipGetLastError();
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
        channels_kernel<<<dim3((2 * a.C + 31) / 32, samples), dim3(1024), 0, s>>>(w.part, sp.count, a.C, 2 * (size_t)a.C, w.chan,
                                                                                 w.chan + a.C, 0);
        if (a.dx) split_dx_kernel<IO, SILU><<<grid, block, dx_lds, s>>>(a, l.V, l.R, sp, n0, w.chan);
        hipError_t e = hipGetLastError();
        if (e == hipSuccess && wanted) e = channels(a, w.chan, samples, n0 > 0, s);
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
