// gdn_glr.hip -- the diagonal gated linear recurrence h_t = a_t h_{t-1} + b_t v_t and its
// gradient (include/gdn.h, gdn_glr_forward / gdn_glr_backward).
//
// One thread per channel walks the tokens; a block holds one head, so that gates per
// head sum their gradients over the block.
#include "gdn_elem.h"
#include "gdn_layer.h"

namespace gdn {
namespace {

// Token walked as number i (0 = first in walking order).
__device__ __forceinline__ long long token(const GlrArgs &a, long long i) { return a.reverse ? a.T - 1 - i : i; }

template <int IO>
__global__ void glr_forward_kernel(GlrArgs a) {
    const int h = blockIdx.x, b = blockIdx.y, c = threadIdx.x;
    const size_t st = ((size_t)b * a.H + h) * a.d + c;
    float s = a.state_in ? a.state_in[st] : 0.0f;
    const long long tiles = (a.T + GLR_TILE - 1) / GLR_TILE;
    for (long long i = 0; i < a.T; ++i) {
        const size_t row = ((size_t)b * a.T + token(a, i)) * a.H + h;
        const size_t gate = a.gate_dim == 1 ? row : row * a.d + c;
        if (a.saved_out && i % GLR_TILE == 0)
            a.saved_out[(((size_t)b * tiles + i / GLR_TILE) * a.H + h) * a.d + c] = s;
        float x = load1<IO>(a.v, row * a.d + c);
        if (a.beta) x *= a.beta[gate];
        s = fmaf(a.decay[gate], s, x);
        store1<IO>(a.out, row * a.d + c, s);
    }
    if (a.state_out) a.state_out[st] = s;
}

// Sum over the block's d threads, in every thread.
__device__ float block_sum(float x, float *lds) {
    const int c = threadIdx.x;
    lds[c] = x;
    __syncthreads();
    for (int k = blockDim.x / 2; k > 0; k /= 2) {
        if (c < k) lds[c] += lds[c + k];
        __syncthreads();
    }
    const float r = lds[0];
    __syncthreads();
    return r;
}

template <int IO>
__global__ void glr_backward_kernel(GlrArgs a) {
    constexpr int HALF = GLR_TILE / 2;
    __shared__ float hist[HALF][128];  // the states before the tokens of half a tile
    __shared__ float lds[128];
    const int h = blockIdx.x, b = blockIdx.y, c = threadIdx.x;
    const size_t st = ((size_t)b * a.H + h) * a.d + c;
    float g = a.dstate_out ? a.dstate_out[st] : 0.0f;
    const long long tiles = (a.T + GLR_TILE - 1) / GLR_TILE, halves = (a.T + HALF - 1) / HALF;
    for (long long k = halves - 1; k >= 0; --k) {
        const long long tile = k / 2, i0 = k * HALF, i1 = i0 + HALF < a.T ? i0 + HALF : a.T;
        float s = a.saved[(((size_t)b * tiles + tile) * a.H + h) * a.d + c];
        for (long long i = tile * GLR_TILE; i < i1; ++i) {
            if (i >= i0) hist[i - i0][c] = s;
            const size_t row = ((size_t)b * a.T + token(a, i)) * a.H + h;
            const size_t gate = a.gate_dim == 1 ? row : row * a.d + c;
            float x = load1<IO>(a.v, row * a.d + c);
            if (a.beta) x *= a.beta[gate];
            s = fmaf(a.decay[gate], s, x);
        }
        for (long long i = i1 - 1; i >= i0; --i) {
            const size_t row = ((size_t)b * a.T + token(a, i)) * a.H + h;
            const size_t gate = a.gate_dim == 1 ? row : row * a.d + c;
            // dout has the output's type: fp32 or bf16
            g += load1<IO == IO_F32 ? IO_F32 : IO_BF16>(a.dout, row * a.d + c);
            float da = g * hist[i - i0][c], db = g * load1<IO>(a.v, row * a.d + c);
            if (a.dv) store1<IO>(a.dv, row * a.d + c, a.beta ? a.beta[gate] * g : g);
            if (a.gate_dim == 1) {
                if (a.ddecay) da = block_sum(da, lds);
                if (a.dbeta) db = block_sum(db, lds);
            }
            if (a.gate_dim != 1 || c == 0) {
                if (a.ddecay) a.ddecay[gate] = da;
                if (a.dbeta) a.dbeta[gate] = db;
            }
            g *= a.decay[gate];
        }
    }
    if (a.dstate_in) a.dstate_in[st] = g;
}

}  // namespace

size_t glr_work_bytes(int, int, int, long long) { return 0; }

hipError_t launch_glr_forward(const GlrArgs &a, hipStream_t s) {
    const dim3 grid(a.H, a.B), block(a.d);
    if (a.io == IO_F32)
        glr_forward_kernel<IO_F32><<<grid, block, 0, s>>>(a);
    else if (a.io == IO_BF16)
        glr_forward_kernel<IO_BF16><<<grid, block, 0, s>>>(a);
    else
        glr_forward_kernel<IO_FP8><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_glr_backward(const GlrArgs &a, hipStream_t s) {
    const dim3 grid(a.H, a.B), block(a.d);
    if (a.io == IO_F32)
        glr_backward_kernel<IO_F32><<<grid, block, 0, s>>>(a);
    else if (a.io == IO_BF16)
        glr_backward_kernel<IO_BF16><<<grid, block, 0, s>>>(a);
    else
        glr_backward_kernel<IO_FP8><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace gdn
