// gdn_rotary.hip -- rotary positions over three axes (include/gdn.h, gdn_rotary).
//
// Pair j of every head of a token is turned by the same angle, so a block takes one
// token, forms its cosines and sines once (angle in 64 bits, reduced to a fraction of a
// turn before the fp32 sine) and turns all heads with them.
#include "gdn_elem.h"
#include "gdn_layer.h"

#include <algorithm>

namespace gdn {
namespace {

template <int IO>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a) {
    __shared__ float cs[ROTARY_MAX_PAIRS], sn[ROTARY_MAX_PAIRS];
    __shared__ int first[ROTARY_MAX_PAIRS], second[ROTARY_MAX_PAIRS];
    for (long long row = blockIdx.x; row < a.B * a.T; row += gridDim.x) {
    const long long b = row / a.T, t = row % a.T;
    for (int j = threadIdx.x; j < a.pairs; j += blockDim.x) {
        int i = j, base = 0, axis = 0;
        while (i >= a.dim[axis] / 2) {
            i -= a.dim[axis] / 2;
            base += a.dim[axis++];
        }
        long long pos;
        if (a.positions) {
            pos = a.positions[b * a.pos_bs + 3 * t + axis];
        } else {
            const long long n = a.first_token + t;
            pos = axis == 0 ? n / ((long long)a.height * a.width) : axis == 1 ? n / a.width % a.height : n % a.width;
        }
        const double turn = (double)pos * a.turns[j];
        sincospif(2.0f * (float)(turn - rint(turn)), &sn[j], &cs[j]);
        if (a.inverse) sn[j] = -sn[j];
        first[j] = base + (a.halves ? i : 2 * i);
        second[j] = a.halves ? first[j] + a.dim[axis] / 2 : first[j] + 1;
    }
    __syncthreads();
    const size_t xr = (size_t)b * a.x_bs + (size_t)t * a.x_ts, orow = (size_t)b * a.out_bs + (size_t)t * a.out_ts;
    for (int e = threadIdx.x; e < a.H * a.pairs; e += blockDim.x) {
        const int h = e / a.pairs, j = e % a.pairs;
        const size_t o = (size_t)h * a.d;
        const float x = load1<IO>(a.x, xr + o + first[j]), y = load1<IO>(a.x, xr + o + second[j]);
        store1<IO>(a.out, orow + o + first[j], x * cs[j] - y * sn[j]);
        store1<IO>(a.out, orow + o + second[j], x * sn[j] + y * cs[j]);
    }
    const int rest = a.d - 2 * a.pairs;
    for (int e = threadIdx.x; e < a.H * rest; e += blockDim.x) {
        const size_t o = (size_t)(e / rest) * a.d + 2 * a.pairs + e % rest;
        store1<IO>(a.out, orow + o, load1<IO>(a.x, xr + o));
    }
    __syncthreads();  // the tables are read above and written by the next token
    }
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)std::min((long long)a.B * a.T, 1LL << 20)), block(256);
    if (a.io == IO_F32)
        rotary_kernel<IO_F32><<<grid, block, 0, s>>>(a);
    else if (a.io == IO_BF16)
        rotary_kernel<IO_BF16><<<grid, block, 0, s>>>(a);
    else
        rotary_kernel<IO_FP8><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace gdn
