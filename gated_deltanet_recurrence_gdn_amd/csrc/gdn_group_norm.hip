// gdn_group_norm.hip -- group norm with an activation, channels last, and its gradient
// (include/gdn.h, gdn_group_norm_forward / gdn_group_norm_backward).
//
// One block per sample and group: mean, then the squares around it, then the outputs.
#include "gdn_elem.h"
#include "gdn_layer.h"

#include <algorithm>

namespace gdn {
namespace {

constexpr int THREADS = 256;

__device__ float block_sum(float x, float *lds) {
    lds[threadIdx.x] = x;
    __syncthreads();
    for (int k = THREADS / 2; k > 0; k /= 2) {
        if ((int)threadIdx.x < k) lds[threadIdx.x] += lds[threadIdx.x + k];
        __syncthreads();
    }
    const float r = lds[0];
    __syncthreads();
    return r;
}

template <int IO>
__global__ __launch_bounds__(THREADS) void group_norm_kernel(GroupNormArgs a) {
    __shared__ float lds[THREADS];
    for (long long ng = blockIdx.x; ng < a.N * a.G; ng += gridDim.x) {
    const long long n = ng / a.G;
    const int g = ng % a.G, D = a.C / a.G;
    const long long m = a.S * D;
    const size_t base = (size_t)n * a.S * a.C + (size_t)g * D;
    float s = 0.0f;
    for (long long e = threadIdx.x; e < m; e += THREADS) s += load1<IO>(a.x, base + e / D * a.C + e % D);
    const float mean = block_sum(s, lds) / (float)m;
    s = 0.0f;
    for (long long e = threadIdx.x; e < m; e += THREADS) {
        const float d = load1<IO>(a.x, base + e / D * a.C + e % D) - mean;
        s = fmaf(d, d, s);
    }
    const float rstd = 1.0f / sqrtf(block_sum(s, lds) / (float)m + a.eps);
    if (a.stats_out && threadIdx.x == 0) {
        a.stats_out[2 * ng] = mean;
        a.stats_out[2 * ng + 1] = rstd;
    }
    for (long long e = threadIdx.x; e < m; e += THREADS) {
        const int c = g * D + (int)(e % D);
        const size_t at = base + e / D * a.C + e % D;
        float z = (load1<IO>(a.x, at) - mean) * rstd;
        if (a.weight) z *= a.weight[c];
        if (a.bias) z += a.bias[c];
        store1<IO>(a.out, at, a.silu ? z * sigmoid_f32(z) : z);
    }
    }
}

// xhat and dz = dy act'(z) of one element.
template <int IO>
__device__ __forceinline__ void grad_terms(const GroupNormArgs &a, size_t at, int c, float mean, float rstd, float *xhat,
                                           float *dz) {
    *xhat = (load1<IO>(a.x, at) - mean) * rstd;
    *dz = load1<IO == IO_F32 ? IO_F32 : IO_BF16>(a.dout, at);
    if (a.silu) {
        const float z = *xhat * (a.weight ? a.weight[c] : 1.0f) + (a.bias ? a.bias[c] : 0.0f);
        const float q = sigmoid_f32(z);
        *dz *= q * (1.0f + z * (1.0f - q));
    }
}

template <int IO>
__global__ __launch_bounds__(THREADS) void group_norm_dx_kernel(GroupNormArgs a) {
    __shared__ float lds[THREADS];
    for (long long ng = blockIdx.x; ng < a.N * a.G; ng += gridDim.x) {
    const long long n = ng / a.G;
    const int g = ng % a.G, D = a.C / a.G;
    const long long m = a.S * D;
    const size_t base = (size_t)n * a.S * a.C + (size_t)g * D;
    const float mean = a.stats[2 * ng], rstd = a.stats[2 * ng + 1];
    float s1 = 0.0f, s2 = 0.0f, xhat, dz;
    for (long long e = threadIdx.x; e < m; e += THREADS) {
        const int c = g * D + (int)(e % D);
        grad_terms<IO>(a, base + e / D * a.C + e % D, c, mean, rstd, &xhat, &dz);
        const float u = a.weight ? dz * a.weight[c] : dz;
        s1 += u;
        s2 = fmaf(u, xhat, s2);
    }
    const float m1 = block_sum(s1, lds) / (float)m, m2 = block_sum(s2, lds) / (float)m;
    for (long long e = threadIdx.x; e < m; e += THREADS) {
        const int c = g * D + (int)(e % D);
        const size_t at = base + e / D * a.C + e % D;
        grad_terms<IO>(a, at, c, mean, rstd, &xhat, &dz);
        const float u = a.weight ? dz * a.weight[c] : dz;
        store1<IO>(a.dx, at, rstd * (u - m1 - xhat * m2));
    }
    }
}

template <int IO>
__global__ __launch_bounds__(THREADS) void group_norm_dw_kernel(GroupNormArgs a) {
    __shared__ float lds[THREADS];
    const int c = blockIdx.x, g = c / (a.C / a.G);
    float s1 = 0.0f, s2 = 0.0f, xhat, dz;
    for (long long r = threadIdx.x; r < a.N * a.S; r += THREADS) {
        const size_t st = 2 * ((size_t)(r / a.S) * a.G + g);
        grad_terms<IO>(a, (size_t)r * a.C + c, c, a.stats[st], a.stats[st + 1], &xhat, &dz);
        s1 += dz;
        s2 = fmaf(dz, xhat, s2);
    }
    s1 = block_sum(s1, lds);
    s2 = block_sum(s2, lds);
    if (threadIdx.x == 0) {
        if (a.dbias) a.dbias[c] = s1;
        if (a.dweight) a.dweight[c] = s2;
    }
}

template <int IO>
hipError_t forward(const GroupNormArgs &a, hipStream_t s) {
    group_norm_kernel<IO><<<dim3((unsigned)std::min(a.N * a.G, 1LL << 20)), dim3(THREADS), 0, s>>>(a);
    return hipGetLastError();
}

template <int IO>
hipError_t backward(const GroupNormArgs &a, hipStream_t s) {
    if (a.dx && a.N * a.S > 0) group_norm_dx_kernel<IO><<<dim3((unsigned)std::min(a.N * a.G, 1LL << 20)), dim3(THREADS), 0, s>>>(a);
    if (a.dweight || a.dbias) group_norm_dw_kernel<IO><<<dim3(a.C), dim3(THREADS), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

size_t group_norm_work_bytes(int, int, long long) { return 0; }

hipError_t launch_group_norm_forward(const GroupNormArgs &a, hipStream_t s) {
    return a.io == IO_F32 ? forward<IO_F32>(a, s) : a.io == IO_BF16 ? forward<IO_BF16>(a, s) : forward<IO_FP8>(a, s);
}

hipError_t launch_group_norm_backward(const GroupNormArgs &a, hipStream_t s) {
    return a.io == IO_F32 ? backward<IO_F32>(a, s) : a.io == IO_BF16 ? backward<IO_BF16>(a, s) : backward<IO_FP8>(a, s);
}

}  // namespace gdn
