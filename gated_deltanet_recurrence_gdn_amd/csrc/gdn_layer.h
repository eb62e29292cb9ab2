// gdn_layer.h -- internal interface between the C-ABI layer and the kernels of the
// operators around the recurrence.  Not installed; callers use include/gdn.h.
#pragma once

#include "gdn_launch.h"

namespace gdn {

constexpr int ROTARY_MAX_PAIRS = 256;  // d <= 512

// One rotary call.  Pairs are numbered through the sections, 0 .. pairs-1.
struct RotaryArgs {
    const void *x;
    void *out;
    long long x_ts, x_bs, out_ts, out_bs;  // elements between tokens / batch elements
    const int *positions;                  // nullptr: raster grid
    long long pos_bs;
    long long first_token;
    int height, width;
    int B, H, d;
    long long T;
    int io;                                // IoType of x
    int halves, inverse;
    int dim[3];                            // section sizes
    int pairs;
    double log2_theta;
};
hipError_t launch_rotary(const RotaryArgs &a, hipStream_t stream);

constexpr int GLR_TILE = 64;   // tokens between saved states

// One call of the diagonal recurrence or of its gradient.
struct GlrArgs {
    const void *v;
    const float *beta, *decay;   // beta may be nullptr (1)
    const float *state_in;       // forward
    float *state_out;
    float *saved_out;            // forward: written if not nullptr
    const float *saved;          // backward
    void *out;
    const void *dout;            // backward
    const float *dstate_out;
    void *dv;
    float *dbeta, *ddecay, *dstate_in;
    int B, H, d;
    long long T;
    int io;
    int gate_dim;                // 1 or d
    int reverse;
    void *work;
    int ncu;
};
size_t glr_work_bytes(int B, int H, int d, long long max_T);
hipError_t launch_glr_forward(const GlrArgs &a, hipStream_t stream);
hipError_t launch_glr_backward(const GlrArgs &a, hipStream_t stream);

// One call of group norm or of its gradient.
struct GroupNormArgs {
    const void *x;
    const float *weight, *bias;
    void *out;
    float *stats_out;            // forward: written if not nullptr
    const float *stats;          // backward
    const void *dout;
    void *dx;
    float *dweight, *dbias;
    long long N, S, max_N;
    int C, G;
    int io;
    int silu;
    float eps;
    void *work;
    int ncu;
};
size_t group_norm_work_bytes(int C, int G, long long max_N);
hipError_t launch_group_norm_forward(const GroupNormArgs &a, hipStream_t stream);
hipError_t launch_group_norm_backward(const GroupNormArgs &a, hipStream_t stream);

}  // namespace gdn
