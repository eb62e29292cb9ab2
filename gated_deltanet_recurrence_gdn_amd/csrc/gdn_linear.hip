// gdn_linear.hip -- linear attention with a decay: the single-token kernel, the joining of
// segments, the decay's gradient, and the launches around the sweeps (gdn_linear_sweep.h).
//
// A sweep is sequential over a pair's tokens, so a call of few (batch, head) pairs is cut into
// segments: one sweep forms every segment's state from zero (reads the row tensors once), a
// join turns these into the segments' start states, and the sweep with outputs then runs all
// segments at once.  The state is linear in its start, so the cut changes rounding only.
#include "gdn_elem.h"
#include "gdn_layer.h"

#include <algorithm>

namespace gdn {

namespace {

// ---- one token (or few): state rows in registers ------------------------------------

// Calls of up to this many tokens: a pair's state is read and written once, its tokens follow one another (the sweep's
// time is the same up to a chunk).  8 x 20 heads, d = 128, step against sweep: bf16 one token 5.3 us against 10.1, four
// 7.6 against 10.0, eight 10.9 against 10.5; fp32 eight 10.4 against 23.4.  4 heads, d = 64: bf16 four 4.5 against 5.3,
// fp32 eight 6.4 against 9.3.
constexpr int step_tokens(int io) { return io == IO_F32 ? 8 : 4; }
constexpr int STEP_ROWS = 4;     // state rows of a lane

struct LinStep {
    LinRows q, k, v;
    LinOut out;
    const float *decay;
    long long g_ts, g_bs;
    const float *state_in;
    float *state_out;
    int H, dk, dv, T;
    float scale;
};

// Four elements and one as they lie in memory; converted where they are used, so that reading them ahead
// waits for nothing.
template <int IO>
struct Raw;
template <>
struct Raw<IO_F32> {
    typedef float4 Four;
    typedef float One;
    static __device__ __forceinline__ float4 four(const Four &w) { return w; }
    static __device__ __forceinline__ float one(One w) { return w; }
};
template <>
struct Raw<IO_BF16> {
    typedef uint2 Four;
    typedef uint16_t One;
    static __device__ __forceinline__ float4 four(const Four &w) {
        return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
    }
    static __device__ __forceinline__ float one(One w) { return __uint_as_float((uint32_t)w << 16); }
};
template <>
struct Raw<IO_FP8> {
    typedef uint32_t Four;
    typedef uint8_t One;
    static __device__ __forceinline__ float4 four(Four w) {
        float f[4];
        fp8x4_to_f32(w, f);
        return make_float4(f[0], f[1], f[2], f[3]);
    }
    static __device__ __forceinline__ float one(One w) {
        float f[4];
        fp8x4_to_f32(w, f);
        return f[0];
    }
};

// LK lanes hold a row's d_k = 4 LK channels; bound by the state, read and written once.
template <int IO, int LK>
__global__ void __launch_bounds__(256) linear_step_kernel(const LinStep a) {
    typedef Raw<IO> R;
    constexpr int RW = 64 / LK;              // rows of a wave at a time
    constexpr int RB = 4 * RW * STEP_ROWS;   // rows of a block
    const int blocks = (a.dv + RB - 1) / RB;
    const int pair = blockIdx.x / blocks, part = blockIdx.x % blocks;
    const int b = pair / a.H, h = pair % a.H;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int d = 4 * (lane % LK), row0 = part * RB + w * RW * STEP_ROWS + lane / LK;
    const float *decay = a.decay + b * a.g_bs + h;
    const long long qo = b * a.q.bs + (long long)h * a.dk + d, ko = b * a.k.bs + (long long)h * a.dk + d;
    const long long vo = b * a.v.bs + (long long)h * a.dv;
    const size_t so = (size_t)pair * a.dv * a.dk + d;
    float4 S[STEP_ROWS];
#pragma unroll
    for (int i = 0; i < STEP_ROWS; ++i) {
        const int n = row0 + RW * i;
        S[i] = make_float4(0, 0, 0, 0);
        if (a.state_in && n < a.dv) S[i] = *reinterpret_cast<const float4 *>(a.state_in + so + (size_t)n * a.dk);
    }
    // a token's operands are read a token ahead: they do not wait for the outputs before
    typename R::Four kn, qn;
    typename R::One vn[STEP_ROWS];
    float gn;
    const auto load = [&](int t) {
        gn = decay[t * a.g_ts];
        kn = *reinterpret_cast<const typename R::Four *>(static_cast<const typename R::One *>(a.k.p) + ko + t * a.k.ts);
        qn = *reinterpret_cast<const typename R::Four *>(static_cast<const typename R::One *>(a.q.p) + qo + t * a.q.ts);
#pragma unroll
        for (int i = 0; i < STEP_ROWS; ++i)
            vn[i] = static_cast<const typename R::One *>(a.v.p)[vo + t * a.v.ts + min(row0 + RW * i, a.dv - 1)];
    };
    load(0);
    for (int t = 0; t < a.T; ++t) {
        const float ga = gn;
        const float4 k = R::four(kn), q = R::four(qn);
        float vt[STEP_ROWS];
#pragma unroll
        for (int i = 0; i < STEP_ROWS; ++i) vt[i] = R::one(vn[i]);
        if (t + 1 < a.T) load(t + 1);
#pragma unroll
        for (int i = 0; i < STEP_ROWS; ++i) {
            const int n = row0 + RW * i;
            const float v = vt[i];
            S[i].x = ga * S[i].x + v * k.x;
            S[i].y = ga * S[i].y + v * k.y;
            S[i].z = ga * S[i].z + v * k.z;
            S[i].w = ga * S[i].w + v * k.w;
            float o = (S[i].x * q.x + S[i].y * q.y) + (S[i].z * q.z + S[i].w * q.w);
            o = group_sum<(LK < 16 ? LK : 16)>(o);
            if constexpr (LK == 32) o += __shfl_xor(o, 16);
            if (lane % LK == 0 && n < a.dv) {
                const long long at = b * a.out.bs + t * a.out.ts + (long long)h * a.dv + n;
                if constexpr (IO == IO_F32) static_cast<float *>(a.out.p)[at] = o * a.scale;
                else static_cast<uint16_t *>(a.out.p)[at] = (uint16_t)f32_to_bf16_bits(o * a.scale);
            }
        }
    }
    if (a.state_out) {
#pragma unroll
        for (int i = 0; i < STEP_ROWS; ++i) {
            const int n = row0 + RW * i;
            if (n < a.dv) *reinterpret_cast<float4 *>(a.state_out + so + (size_t)n * a.dk) = S[i];
        }
    }
}

template <int IO>
hipError_t step_launch(const LinStep &a, int pairs, hipStream_t stream) {
    const auto go = [&](auto kernel, int rows) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)(pairs * ((a.dv + rows - 1) / rows))), dim3(256), 0, stream, a);
    };
    if (a.dk == 16) go(linear_step_kernel<IO, 4>, 16 * 4 * STEP_ROWS);
    else if (a.dk == 32) go(linear_step_kernel<IO, 8>, 8 * 4 * STEP_ROWS);
    else if (a.dk == 64) go(linear_step_kernel<IO, 16>, 4 * 4 * STEP_ROWS);
    else go(linear_step_kernel<IO, 32>, 2 * 4 * STEP_ROWS);
    return hipGetLastError();
}

// ---- start states of the segments -----------------------------------------------------

// slots[0] = state_in; slots[s] = gamma[s-1] slots[s-1] + slots[s].  A thread has four
// neighbouring elements of a pair's state.  Sixteen segments are read ahead of their sums and
// blocks are one wave, so that a single pair's 512 segments wait for memory 32 times, not 512,
// and on 64 CUs.
constexpr int JOIN_AHEAD = 16;
__global__ void __launch_bounds__(64) linear_join_kernel(float *slots, const float2 *gamma, const float *state_in, int nseg,
                                                         int nslots, int size) {
    const int per = size / 256;
    const int lp = blockIdx.x / per, i = (blockIdx.x % per * 64 + threadIdx.x) * 4;
    float *p = slots + (size_t)lp * nslots * size + i;
    const float2 *gm = gamma + (size_t)lp * nslots;
    f32x4_t S = {0, 0, 0, 0};
    if (state_in) S = *reinterpret_cast<const f32x4_t *>(state_in + (size_t)lp * size + i);
    *reinterpret_cast<f32x4_t *>(p) = S;
    for (int s0 = 1; s0 < nseg; s0 += JOIN_AHEAD) {
        f32x4_t x[JOIN_AHEAD];
        float2 c[JOIN_AHEAD];
#pragma unroll
        for (int k = 0; k < JOIN_AHEAD; ++k) {
            const int s = min(s0 + k, nseg - 1);
            x[k] = *reinterpret_cast<const f32x4_t *>(p + (size_t)s * size);
            c[k] = gm[s - 1];
        }
#pragma unroll
        for (int k = 0; k < JOIN_AHEAD; ++k) {
            if (s0 + k >= nseg) break;
            S = c[k].x * S + (c[k].y * S + x[k]);
            *reinterpret_cast<f32x4_t *>(p + (size_t)(s0 + k) * size) = S;
        }
    }
}

// ---- the decay's gradient ---------------------------------------------------------------

// ln a_t scales what passes from before t to t and after: with S the state before the chunk and
// U the gradient of the state behind it,
//   d ln a_t = sum_{j < t <= i} W_ij + sum_{i >= t} x_i + sum_{j < t} y_j + c,
// i, j in the chunk, W the products of scores, x what S gave to i, y what U gave to j, and
// c = e^{G_end} <U, S>.  The sweeps leave row sums r, column sums s of W (strictly below the
// diagonal), x and y; sum_{j < t <= i} W_ij = sum_{i >= t} (r_i - s_i).  <R, S> at a chunk's end
// is c + sum y, at its start c + sum x: the known product at the segment's end gives every c.
// These last sums are in 64 bits.
struct LinDecay {
    const float *r, *s, *x, *y;      // [pair][64 chunks]; x and y in two parts, half elements apart
    long long half;
    const float *slots_s, *slots_u;  // nullptr with one segment; slots_u begins with dstate_out
    const float *fin, *dstate_out;   // the last state and its gradient (nullptr: zeros)
    const float *decay;
    long long g_ts, g_bs;
    float *dlog;                     // [B,T,H] in the walk's order, or nullptr
    long long d_ts, d_bs;
    double *sums;                    // [pair of the call][nseg], or nullptr
    int H, pair0, size;
    long long T;
    int chunks, seg_chunks, nseg, nslots;
};
constexpr int MAX_SEG_CHUNKS = 16;   // of a gradient's segment: bounds how far errors of c add up

__global__ void __launch_bounds__(256) linear_decay_kernel(const LinDecay a) {
    __shared__ double part[4];
    __shared__ double xs[MAX_SEG_CHUNKS], ys[MAX_SEG_CHUNKS];
    const int lp = blockIdx.x / a.nseg, seg = blockIdx.x % a.nseg;
    const int pair = a.pair0 + lp, b = pair / a.H, h = pair % a.H;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int c0 = seg * a.seg_chunks, n = min(a.seg_chunks, a.chunks - c0);
    const float *S, *U;
    if (seg == a.nseg - 1) {
        S = a.fin + (size_t)lp * a.size;
        U = !a.dstate_out ? nullptr : a.slots_u ? a.slots_u + (size_t)lp * a.nslots * a.size : a.dstate_out + (size_t)lp * a.size;
    } else {
        S = a.slots_s + ((size_t)lp * a.nslots + seg + 1) * a.size;
        U = a.slots_u + ((size_t)lp * a.nslots + a.nseg - 1 - seg) * a.size;
    }
    const auto wave_sum = [](double v) {
        for (int o = 32; o; o /= 2) v += __shfl_xor(v, o);
        return v;
    };
    double dot = 0.0;
    if (U)
        for (int i = threadIdx.x * 4; i < a.size; i += 1024) {
            const float4 s = *reinterpret_cast<const float4 *>(S + i), u = *reinterpret_cast<const float4 *>(U + i);
            dot += (double)s.x * u.x + (double)s.y * u.y + (double)s.z * u.z + (double)s.w * u.w;
        }
    dot = wave_sum(dot);
    if (lane == 0) part[w] = dot;
    const size_t at = ((size_t)lp * a.chunks + c0) * LIN_CHUNK + lane;
    for (int c = w; c < n; c += 4) {
        const size_t i = at + c * LIN_CHUNK;
        const double x = wave_sum((double)a.x[i] + a.x[i + a.half]), y = wave_sum((double)a.y[i] + a.y[i + a.half]);
        if (lane == 0) {
            xs[c] = x;
            ys[c] = y;
        }
    }
    __syncthreads();
    double all = 0.0;
    for (int c = w; c < n; c += 4) {
        double B = part[0] + part[1] + part[2] + part[3];
        for (int k = n - 1; k > c; --k) B += xs[k] - ys[k];
        const double base = B - ys[c];
        const size_t i = at + c * LIN_CHUNK;
        double suf = (double)a.r[i] - a.s[i] + a.x[i] + a.x[i + a.half], pre = (double)a.y[i] + a.y[i + a.half];
        const double own = pre;
        for (int o = 1; o < 64; o *= 2) {
            const double u = __shfl_down(suf, o), d = __shfl_up(pre, o);
            if (lane + o < 64) suf += u;
            if (lane >= o) pre += d;
        }
        const long long t = (long long)(c0 + c) * LIN_CHUNK + lane;
        if (t < a.T) {
            const float ga = a.decay[b * a.g_bs + t * a.g_ts + h];
            const double d = ga == 0.0f ? 0.0 : suf + (pre - own) + base;
            if (a.dlog) a.dlog[b * a.d_bs + t * a.d_ts + h] = (float)d;
            all += d;
        }
    }
    if (a.sums) {
        all = wave_sum(all);
        __syncthreads();
        if (lane == 0) part[w] = all;
        __syncthreads();
        if (threadIdx.x == 0) a.sums[(size_t)pair * a.nseg + seg] = part[0] + part[1] + part[2] + part[3];
    }
}

// A decay per head: its gradient sums over batch and tokens, in a fixed order.
__global__ void __launch_bounds__(256) linear_decay_sum_kernel(const double *sums, float *dlog, int B, int H, int nseg) {
    __shared__ double part[256];
    const int h = blockIdx.x;
    double x = 0.0;
    const long long n = (long long)B * nseg;
    for (long long i = threadIdx.x; i < n; i += 256) x += sums[(i / nseg * H + h) * nseg + i % nseg];
    part[threadIdx.x] = x;
    __syncthreads();
    for (int o = 128; o; o /= 2) {
        if ((int)threadIdx.x < o) part[threadIdx.x] += part[threadIdx.x + o];
        __syncthreads();
    }
    if (threadIdx.x == 0) dlog[h] = (float)part[0];
}

__global__ void __launch_bounds__(256) linear_fill_kernel(float *p, const float *from, long long n) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = from ? from[i] : 0.0f;
}

// ---- how calls are cut --------------------------------------------------------------------

// Forward, where pairs leave CUs without a block: segments for a block a CU or for two, or none.  In a chunk's time
// of both sweeps (4.4 us, d = 128) a segment takes its chunks and three more for its start, the join and a launch,
// two blocks on a CU 1.4 times one, and a pair in one piece its chunks and one more.  Measured in segments of 1, 2, 3,
// 4 chunks: 512 tokens of 20 heads 26.6, 28.2, 31.4, 36.6 us, 1,024 36.0, 31.6, 34.5, 40.3 (320 blocks, 160, 120, 80),
// 2,048 in 2, 3, 4 43.6, 37.4, 41.9; 200 of 4 heads 16.6 in 1, 21.9 in one piece; 2 x 32,760 of 32 heads in 128
// (a block a CU) 1,010, in 64 810.  These ratios are bf16's at d = 128, and are used for all sizes and types: of every
// length there is for 4 to 600 heads of 8 to 64 chunks, d = 16 to 128, bf16 and fp32, the one chosen was the quickest or
// within 10%, but for 64 heads of 16 chunks at d = 16 and 32 (4 chunks 20.1 and 21.1 us, 2 chunks 15.9 and 17.7; fp32 27.1
// and 28.0, 21.7 and 23.5) and where fp32 at d = 128 has no room for two blocks on a CU (200 heads of 40 chunks: 20
// chunks 776, one piece 632).
int forward_seg_chunks(long long pairs, long long chunks, int ncu) {
    long long best = chunks, least = 10 * (10 * chunks + 10);
    for (int a_cu = 1; a_cu <= 2; ++a_cu) {
        const long long most = (long long)a_cu * ncu / pairs;
        if (most < 2 || chunks < 2) continue;
        const long long s = (chunks + most - 1) / most;
        const long long cost = (10 * s + 30) * (pairs * ((chunks + s - 1) / s) <= ncu ? 10 : 14);
        if (cost < least) {
            least = cost;
            best = s;
        }
    }
    return (int)best;
}
// A bound of the segments of all calls of up to `chunks` chunks (shorter ones may have more).
long long forward_most(long long pairs, long long chunks, int ncu) {
    return std::max(1LL, std::min(2LL * ncu / pairs, chunks));
}

// The gradient: segments of at most MAX_SEG_CHUNKS chunks, and pairs in groups that share one
// workspace.  At d = 128 a CU has one block of it at a time, so a segment is as long as fills the last
// round of blocks best (a chunk's time is added for the start of each): 32,760 tokens of 20 heads in
// segments of 14 chunks rather than 16 (dq 390 us against 411, dk and dv 442 against 466).  Smaller
// heads leave room for more blocks (24 KB of LDS at d = 32), but are cut alike: of the lengths 1 to 16 for 4 to 600 heads
// of 8 to 64 chunks the one chosen was the quickest or within 10%, but for 64 heads of 16 chunks at d = 16 and 32 (4
// chunks 49 and 52 us, 2 chunks 42 and 46; fp32 at d = 16 69, 61) and 64 heads of 64 chunks in bf16 at d = 128 (8 chunks 448,
// 16 chunks 389).
struct GradCut {
    int seg_chunks, nseg, nslots, group;
    size_t slot_floats, dot_floats;  // of a group: slots of one direction, one dot array
    size_t bytes;                    // whole workspace
};
constexpr size_t GRAD_WORK = size_t(512) << 20;
constexpr int DOTS = 6;              // dot arrays: r, s, two parts each of x and y

size_t grad_pair_bytes(size_t size, long long nslots, long long chunks) {
    return ((2 * (size_t)nslots + 1) * size + DOTS * (size_t)chunks * LIN_CHUNK + 4 * (size_t)nslots) * sizeof(float) +
           (size_t)nslots * sizeof(double);
}

GradCut grad_cut(int B, int H, int d_k, int d_v, long long chunks, int ncu) {
    GradCut c;
    const long long pairs = (long long)B * H, least = (pairs * chunks + 4LL * ncu - 1) / (4LL * ncu);
    long long best = -1;
    c.seg_chunks = MAX_SEG_CHUNKS;
    for (int s = (int)std::min<long long>(MAX_SEG_CHUNKS, least); s <= MAX_SEG_CHUNKS; ++s) {
        // in chunks' times: two sweeps, and with several segments their states (two blocks a CU, half the
        // work, two sweeps) and the joins
        const long long nseg = (chunks + s - 1) / s, len = std::min<long long>(s, chunks);
        const long long rounds = (pairs * nseg + ncu - 1) / ncu, before = (pairs * (nseg - 1) + 2 * ncu - 1) / (2 * ncu);
        const long long cost = 2 * rounds * (len + 1) + (nseg > 1 ? before * len + 2 : 0);
        if (best < 0 || cost <= best) {
            best = cost;
            c.seg_chunks = s;
        }
    }
    c.nseg = c.nslots = (int)((chunks + c.seg_chunks - 1) / c.seg_chunks);
    const size_t size = (size_t)d_k * d_v, a_pair = grad_pair_bytes(size, c.nslots, chunks);
    c.group = (int)std::min<long long>(pairs, std::max<long long>(1, GRAD_WORK / a_pair));
    c.slot_floats = (size_t)c.group * c.nslots * size;
    c.dot_floats = (size_t)c.group * chunks * LIN_CHUNK;
    c.bytes = (2 * c.slot_floats + (size_t)c.group * size + DOTS * c.dot_floats + 4 * (size_t)c.group * c.nslots) * sizeof(float) +
              (size_t)pairs * c.nseg * sizeof(double) + 256;
    return c;
}

// A bound of GradCut::bytes over all calls of up to `chunks` chunks (shorter ones may be cut finer):
// a pair never has more than 4 ncu / pairs + 2 segments beyond those of MAX_SEG_CHUNKS.
size_t grad_most(int B, int H, int d_k, int d_v, long long chunks, int ncu) {
    const long long pairs = (long long)B * H, nslots = 4LL * ncu / pairs + 2 + chunks / MAX_SEG_CHUNKS;
    const size_t a_pair = grad_pair_bytes((size_t)d_k * d_v, nslots, chunks);
    return std::min((size_t)pairs * a_pair, std::max(GRAD_WORK, a_pair)) + (size_t)pairs * nslots * sizeof(double) + 256;
}

// The operands of a walk: `back` walks the (padded) tokens from the last to the first.
struct Walk {
    bool turn;       // the memory's order is the walk's reversed
    long long T, Tp;
    long long shift, sign;  // memory token of walk token t: shift + sign t
    Walk(long long T_, bool reverse, bool back) : T(T_), Tp((T_ + LIN_CHUNK - 1) / LIN_CHUNK * LIN_CHUNK) {
        // forward walk: m = t, or T - 1 - t; backwards t' = Tp - 1 - t
        if (!back) {
            sign = reverse ? -1 : 1;
            shift = reverse ? T - 1 : 0;
        } else {
            sign = reverse ? 1 : -1;
            shift = reverse ? T - Tp : Tp - 1;
        }
        turn = sign < 0;
    }
};
LinRows rows(const Walk &w, const void *p, long long ts, long long bs, int bytes) {
    LinRows r;
    r.p = static_cast<const char *>(p) + w.shift * ts * bytes;
    r.ts = w.sign * ts;
    r.bs = bs;
    return r;
}
LinOut outs(const Walk &w, void *p, long long ts, long long bs, int bytes) {
    LinOut r;
    r.p = p ? static_cast<char *>(p) + w.shift * ts * bytes : nullptr;
    r.ts = w.sign * ts;
    r.bs = bs;
    return r;
}

void set_gate(const LinearArgs &a, const Walk &w, const float *&decay, long long &ts, long long &bs) {
    decay = a.decay + (a.per_head ? 0 : w.shift * a.H);
    ts = a.per_head ? 0 : w.sign * a.H;
    bs = a.per_head ? 0 : a.T * a.H;
}

hipError_t fill(float *p, const float *from, long long n, hipStream_t stream) {
    hipLaunchKernelGGL(linear_fill_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, p, from, n);
    return hipGetLastError();
}

hipError_t join(float *slots, const float2 *gamma, const float *state_in, const LinSweep &s, int pairs, hipStream_t stream) {
    const int size = s.dk * s.dv, per = size / 256;  // 16 x 16 at least
    hipLaunchKernelGGL(linear_join_kernel, dim3((unsigned)(pairs * per)), dim3(64), 0, stream, slots, gamma, state_in, s.nseg,
                       s.nslots, size);
    return hipGetLastError();
}

}  // namespace

size_t linear_work_bytes(int B, int H, int d_k, int d_v, long long max_T, int train, int ncu) {
    const long long pairs = (long long)B * H, chunks = (max_T + LIN_CHUNK - 1) / LIN_CHUNK;
    const long long nseg = forward_most(pairs, chunks, ncu);
    size_t n = nseg > 1 ? (size_t)pairs * nseg * ((size_t)d_k * d_v + 2) * sizeof(float) + 256 : 0;
    return train && chunks ? std::max(n, grad_most(B, H, d_k, d_v, chunks, ncu)) : n;
}

hipError_t launch_linear_forward(const LinearArgs &a, hipStream_t stream) {
    const long long pairs = (long long)a.B * a.H;
    const size_t size = (size_t)a.d_k * a.d_v;
    const int ib = io_in_bytes(a.io), ob = io_out_bytes(a.io);
    const float scale = 1.0f / sqrtf((float)a.d_k);
    if (a.T == 0) {
        if (a.state_out == a.state_in) return hipSuccess;
        return fill(a.state_out, a.state_in, pairs * size, stream);
    }
    const Walk w(a.T, a.reverse, false);
    if (a.T <= step_tokens(a.io)) {
        LinStep s{};
        s.q = rows(w, a.q, a.q_ts, a.q_bs, ib);
        s.k = rows(w, a.k, a.k_ts, a.k_bs, ib);
        s.v = rows(w, a.v, a.v_ts, a.v_bs, ib);
        s.out = outs(w, a.out, (long long)a.H * a.d_v, a.T * a.H * a.d_v, ob);
        set_gate(a, w, s.decay, s.g_ts, s.g_bs);
        s.state_in = a.state_in; s.state_out = a.state_out;
        s.H = a.H; s.dk = a.d_k; s.dv = a.d_v; s.T = (int)a.T; s.scale = scale;
        return a.io == IO_F32 ? step_launch<IO_F32>(s, (int)pairs, stream)
             : a.io == IO_FP8 ? step_launch<IO_FP8>(s, (int)pairs, stream)
                              : step_launch<IO_BF16>(s, (int)pairs, stream);
    }
    LinSweep s{};
    s.r1 = rows(w, a.k, a.k_ts, a.k_bs, ib);
    s.r2 = rows(w, a.v, a.v_ts, a.v_bs, ib);
    s.a1 = rows(w, a.q, a.q_ts, a.q_bs, ib);
    s.out1 = outs(w, a.out, (long long)a.H * a.d_v, a.T * a.H * a.d_v, ob);
    set_gate(a, w, s.decay, s.g_ts, s.g_bs);
    s.state_in = a.state_in; s.state_out = a.state_out; s.so_stride = (long long)size;
    s.H = a.H; s.dk = a.d_k; s.dv = a.d_v;
    s.lo = 0; s.hi = (int)a.T;
    s.chunks = (int)(w.Tp / LIN_CHUNK);
    s.seg_chunks = s.seg_first = forward_seg_chunks(pairs, s.chunks, a.ncu);
    s.nseg = s.nslots = (s.chunks + s.seg_chunks - 1) / s.seg_chunks;
    s.scale_d = s.scale_cross = scale;
    s.scale_upd = 1.0f;
    if (s.nseg > 1) {
        s.slots = static_cast<float *>(a.work);
        s.gamma = reinterpret_cast<float2 *>(s.slots + (size_t)pairs * s.nslots * size);
        hipError_t e = linear_sweep_state(s, a.io, 0, (int)pairs, stream);
        if (e == hipSuccess) e = join(s.slots, s.gamma, a.state_in, s, (int)pairs, stream);
        if (e != hipSuccess) return e;
    }
    return linear_sweep_out(s, a.io, (int)pairs, stream);
}

hipError_t launch_linear_backward(const LinearArgs &a, hipStream_t stream) {
    const int pairs = a.B * a.H;
    const size_t size = (size_t)a.d_k * a.d_v;
    const int ib = io_in_bytes(a.io), ob = io_out_bytes(a.io);
    const float scale = 1.0f / sqrtf((float)a.d_k);
    if (a.T == 0) {
        hipError_t e = hipSuccess;
        if (a.dlog_decay && a.per_head) e = fill(a.dlog_decay, nullptr, a.H, stream);
        if (e != hipSuccess || !a.dstate_in || a.dstate_in == a.dstate_out) return e;
        return fill(a.dstate_in, a.dstate_out, pairs * (long long)size, stream);
    }
    const GradCut cut = grad_cut(a.B, a.H, a.d_k, a.d_v, (a.T + LIN_CHUNK - 1) / LIN_CHUNK, a.ncu);
    if (cut.bytes > a.work_bytes) return hipErrorInvalidValue;
    double *sums = static_cast<double *>(a.work);
    float *slots_s = reinterpret_cast<float *>(sums + (size_t)pairs * cut.nseg + 1);
    slots_s = reinterpret_cast<float *>((reinterpret_cast<uintptr_t>(slots_s) + 63) & ~(uintptr_t)63);
    float *slots_u = slots_s + cut.slot_floats, *fin = slots_u + cut.slot_floats;
    float *dots = fin + (size_t)cut.group * size;
    float2 *gamma_s = reinterpret_cast<float2 *>(dots + DOTS * cut.dot_floats), *gamma_u = gamma_s + (size_t)cut.group * cut.nslots;

    const Walk fw(a.T, a.reverse, false), bw(a.T, a.reverse, true);
    const long long ts_k = (long long)a.H * a.d_k, ts_v = (long long)a.H * a.d_v;
    LinSweep s{}, u{};
    s.r1 = rows(fw, a.k, a.k_ts, a.k_bs, ib);
    s.r2 = rows(fw, a.v, a.v_ts, a.v_bs, ib);
    s.a1 = rows(fw, a.q, a.q_ts, a.q_bs, ib);
    s.a2 = rows(fw, a.dout, ts_v, a.T * ts_v, ob);
    s.out2 = outs(fw, a.dq, ts_k, a.T * ts_k, ob);
    set_gate(a, fw, s.decay, s.g_ts, s.g_bs);
    s.lo = 0; s.hi = (int)a.T;
    s.scale_d = s.scale_cross = scale; s.scale_upd = 1.0f;
    s.dot_w = dots; s.dot_x = dots + 2 * cut.dot_floats; s.dot_step = 1;
    u.r1 = rows(bw, a.q, a.q_ts, a.q_bs, ib);
    u.r2 = rows(bw, a.dout, ts_v, a.T * ts_v, ob);
    u.a1 = rows(bw, a.k, a.k_ts, a.k_bs, ib);
    u.a2 = rows(bw, a.v, a.v_ts, a.v_bs, ib);
    u.out1 = outs(bw, a.dv, ts_v, a.T * ts_v, ob);
    u.out2 = outs(bw, a.dk, ts_k, a.T * ts_k, ob);
    set_gate(a, bw, u.decay, u.g_ts, u.g_bs);
    u.lo = (int)(bw.Tp - a.T); u.hi = (int)bw.Tp;
    u.scale_d = u.scale_upd = scale; u.scale_cross = 1.0f;
    u.exclusive = 1;
    u.dot_w = dots + cut.dot_floats; u.dot_x = dots + 4 * cut.dot_floats; u.dot_step = -1;
    for (LinSweep *p : {&s, &u}) {
        p->H = a.H; p->dk = a.d_k; p->dv = a.d_v;
        p->chunks = (int)(fw.Tp / LIN_CHUNK);
        p->seg_chunks = cut.seg_chunks;
        p->nseg = cut.nseg; p->nslots = cut.nslots;
        p->dot_half = (long long)cut.dot_floats;
        p->so_stride = (long long)size;
    }
    s.seg_first = cut.seg_chunks;
    u.seg_first = u.chunks - (cut.nseg - 1) * cut.seg_chunks;  // the same cuts from the other end
    if (cut.nseg > 1) {
        s.slots = slots_s; s.gamma = gamma_s;
        u.slots = slots_u; u.gamma = gamma_u;
    }
    const bool want_u = a.dk || a.dv || a.dlog_decay || a.dstate_in, want_s = a.dq || a.dlog_decay;
    for (int p0 = 0; p0 < pairs; p0 += cut.group) {
        const int n = std::min(cut.group, pairs - p0);
        s.pair0 = u.pair0 = p0;
        s.state_in = a.state_in ? a.state_in + p0 * size : nullptr;
        s.state_out = a.dlog_decay && a.dstate_out ? fin : nullptr;
        u.state_in = a.dstate_out ? a.dstate_out + p0 * size : nullptr;
        u.state_out = a.dstate_in ? a.dstate_in + p0 * size : nullptr;
        hipError_t e = hipSuccess;
        if (cut.nseg > 1 && want_s) {
            e = linear_sweep_state(s, a.io, 0, n, stream);
            if (e == hipSuccess) e = join(slots_s, gamma_s, s.state_in, s, n, stream);
        }
        if (e == hipSuccess && cut.nseg > 1 && want_u) {
            e = linear_sweep_state(u, a.io, 1, n, stream);
            if (e == hipSuccess) e = join(slots_u, gamma_u, u.state_in, u, n, stream);
        }
        if (e == hipSuccess && want_s) e = linear_sweep_dq(s, a.io, n, stream);
        const float *dstate = u.state_in;
        if (e == hipSuccess && a.dlog_decay && cut.nseg == 1 && dstate && a.dstate_in == a.dstate_out) {
            e = fill(slots_u, dstate, n * (long long)size, stream);  // the backward walk writes over it
            dstate = slots_u;
        }
        if (e == hipSuccess && want_u) e = linear_sweep_dkv(u, a.io, n, stream);
        if (e == hipSuccess && a.dlog_decay) {
            LinDecay d{};
            d.half = (long long)cut.dot_floats;
            d.r = s.dot_w; d.x = s.dot_x; d.s = u.dot_w; d.y = u.dot_x;
            d.slots_s = s.slots; d.slots_u = u.slots;
            d.fin = fin;
            d.dstate_out = dstate;
            set_gate(a, fw, d.decay, d.g_ts, d.g_bs);
            if (a.per_head) {
                d.sums = sums;
            } else {
                d.dlog = a.dlog_decay + fw.shift * a.H;
                d.d_ts = fw.sign * a.H;
                d.d_bs = a.T * a.H;
            }
            d.H = a.H; d.pair0 = p0; d.size = (int)size;
            d.T = a.T; d.chunks = s.chunks; d.seg_chunks = cut.seg_chunks; d.nseg = cut.nseg; d.nslots = cut.nslots;
            hipLaunchKernelGGL(linear_decay_kernel, dim3((unsigned)(n * cut.nseg)), dim3(256), 0, stream, d);
            e = hipGetLastError();
        }
        if (e != hipSuccess) return e;
    }
    if (a.dlog_decay && a.per_head) {
        hipLaunchKernelGGL(linear_decay_sum_kernel, dim3((unsigned)a.H), dim3(256), 0, stream, sums, a.dlog_decay, a.B, a.H, cut.nseg);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace gdn
