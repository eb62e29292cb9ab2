// gdn_linear_sweep.h -- the sweep of linear attention with a decay, forward and gradient:
//
//     S_t = a_t S_{t-1} + v_t k_t^T,    o_t = scale S_t q_t              (scale = d_k^-1/2)
//     R_t = a_{t+1} R_{t+1} + scale do_t q_t^T                           (walked backwards)
//     dq_t = scale S_t^T do_t,  dk_t = R_t^T v_t,  dv_t = R_t k_t,  d ln a_t = a_t <R_t, S_{t-1}>
//
// All of it is one sweep over chunks of 64 tokens that carries a d_v x d_k state M from the
// products of two "row" tensors, r1 (d_k) and r2 (d_v), and reads it with "own" tensors:
//
//     out1_c = sum_{r <= c} D_cr (r1_r . a1_c) r2_r + e^{G_c} M a1_c       (d_v)
//     out2_c = sum_{r <= c} D_cr (r2_r . a2_c) r1_r + e^{G_c} M^T a2_c     (d_k)
//     M <- e^{G_end} M + sum_r e^{G_end - G_r} r2_r r1_r^T,   D_cr = e^{G_c - G_r},
//
// G the sum of the logarithms of the decays from the chunk's start.
//     forward             r = (k, v), a1 = q:           out1 = o
//     gradient, forwards  r = (k, v), a = (q, do):      out2 = dq
//     gradient, backwards r = (q, do), a = (k, v):      out1 = dv, out2 = dk
// The backward walk is the same code on tokens in the other order with G without the token's
// own decay ("exclusive"): R_t takes in a_{t+1}, not a_t.
//
// Precision: bf16 (or FP8, widened exactly) inputs go to bf16 MFMA with fp32 sums.  D r1.a1 is
// rounded to bf16 before the second product, and so is M (held in fp32) before M a1: outputs are
// bf16, and come out 2.3e-3 off (rel-L2; dq and dk, which read M in three parts, 2.0e-3) where their own rounding is
// 1.7e-3.  With two parts of both they are 1.66e-3 off, but the second part of M leaves one block
// on a CU in place of two: 2 x 32,760 tokens of 32 heads 1,165 us against 784, training step of 32,760 x 20
// heads 1,531 against 1,359.  What leaves in fp32 is held to fp32: the weighted operand of the state's update goes in as three
// bf16 parts, and where the decay's gradient reads M it is three parts too (two parts, 2^-16 of
// a term, left states 3e-6 off and that gradient, which sums differences, up to 1.6e-5).
// fp32 inputs run the same code on fp32 MFMA.  Logarithms of decays are summed in 64 bits and kept
// in two fp32 parts: a reset (a = 0) enters as 2^-200 and must not cost the differences behind it
// their digits.
#pragma once

#include "gdn_elem.h"
#include "gdn_layer.h"

namespace gdn {

typedef __bf16 lin_bf16x8_t __attribute__((ext_vector_type(8)));
typedef short lin_s16x4_t __attribute__((ext_vector_type(4)));

// Waves of a block: eight where both head dims have two steps of 32 for them, else four.
constexpr int lin_waves(int DK, int DV) { return DK >= 64 && DV >= 64 ? 8 : 4; }
constexpr int LIN_PARTS = 3;  // bf16 parts of an fp32 operand: 2^-24 of it

// Operands of 16x16 products over 32 terms.  A fragment is a lane's eight terms of row (or
// column) lane % 16; lanes of one group of 16 hold the same eight terms.  Which eight is free
// as long as both operands agree: 8 g + e (ROWS order), or 4 g + e and 16 + 4 g + e as the
// accumulators of a product hold them (ACC order), g = lane / 16.
template <bool F32>
struct LinOp;

template <>
struct LinOp<false> {
    using E = uint16_t;
    using Frag = lin_bf16x8_t;
    // LDS rows start 8 banks (mod 64) apart, and every eighth row of the state 32 more: reads of
    // 16 bytes from 16 rows and transposed reads then meet no bank twice, but for the eight-channel
    // steps of an output's rows (twice).
    static constexpr int PAD = 16, SKEW = 64;
    static __device__ __forceinline__ Frag zero() { return Frag{}; }
    static __device__ __forceinline__ f32x4_t mma(const Frag &a, const Frag &b, f32x4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ Frag row(const E *p) {
        Frag r;
        __builtin_memcpy(&r, p, 16);
        return r;
    }
    // Terms down the rows of a row-major tile, 32 rows from `tile` on, in ROWS or ACC order, and
    // for lane % 16 = l the column step (l / 4) + l % 4.  group: elements between the first rows
    // of two groups.
    template <bool ACC>
    static __device__ __forceinline__ Frag col(const E *tile, int stride, int group, int step, int l, int g) {
        typedef __attribute__((address_space(3))) lin_s16x4_t lds_t;
        const E *p0 = tile + g * group + (l >> 2) * stride + step * (l & 3);
        const E *p1 = p0 + (ACC ? 16 : 4) * stride;
        // result lane i, slot s = element i % 4 of what lane 4 s + i / 4 addresses
        const lin_s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t *)p0);
        const lin_s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t *)p1);
        Frag r;
        __builtin_memcpy(&r, &lo, 8);
        __builtin_memcpy(reinterpret_cast<char *>(&r) + 8, &hi, 8);
        return r;
    }
    static __device__ __forceinline__ Frag pack(const float (&f)[8]) {
        const uint32_t w[4] = {pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                               pack_bf16x2(f[6], f[7])};
        Frag r;
        __builtin_memcpy(&r, w, 16);
        return r;
    }
    static __device__ __forceinline__ void get(const Frag &r, float (&f)[8]) {
        uint32_t w[4];
        __builtin_memcpy(w, &r, 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        }
    }
};

template <>
struct LinOp<true> {
    using E = float;
    struct Frag {
        float v[8];
    };
    static constexpr int PAD = 4, SKEW = 0;
    static __device__ __forceinline__ Frag zero() { return Frag{}; }
    static __device__ __forceinline__ f32x4_t mma(const Frag &a, const Frag &b, f32x4_t c) {
#pragma unroll
        for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ Frag row(const E *p) {
        Frag r;
        __builtin_memcpy(&r, p, 32);
        return r;
    }
    template <bool ACC>
    static __device__ __forceinline__ Frag col(const E *tile, int stride, int group, int step, int l, int g) {
        const E *p = tile + g * group + step * (l >> 2) + (l & 3);
        Frag r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r.v[e] = p[(ACC && e >= 4 ? 12 + e : e) * stride];
        return r;
    }
    static __device__ __forceinline__ Frag pack(const float (&f)[8]) {
        Frag r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r.v[e] = f[e];
        return r;
    }
    static __device__ __forceinline__ void get(const Frag &r, float (&f)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = r.v[e];
    }
};

// Eight elements of a row as loaded (widened when they are used).  Loads go through a buffer
// descriptor: an offset beyond its 2 GB reads zeros, which is how rows and channels that do not
// exist are cleared, without a branch (which would wait for the load) or a select behind it.
typedef uint32_t lin_u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t lin_u32x2_t __attribute__((ext_vector_type(2)));
constexpr uint32_t LIN_NOWHERE = 0x80000000u;

template <int IO>
struct LinRaw {
    static constexpr int WORDS = 2 * io_in_bytes(IO);
    uint32_t r[WORDS];
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rsrc, uint32_t off, int soff) {
        if constexpr (IO == IO_FP8) {
            const lin_u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(rsrc, off, soff, 0);
            r[0] = v[0];
            r[1] = v[1];
        } else {
#pragma unroll
            for (int i = 0; i < WORDS; i += 4) {
                const lin_u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(rsrc, off + 4 * i, soff, 0);
#pragma unroll
                for (int k = 0; k < 4; ++k) r[i + k] = v[k];
            }
        }
    }
    __device__ __forceinline__ typename LinOp<IO == IO_F32>::Frag frag() const {
        typename LinOp<IO == IO_F32>::Frag f;
        if constexpr (IO == IO_FP8) {
            const uint2 a = fp8x4_to_bf16x4(r[0]), b = fp8x4_to_bf16x4(r[1]);
            const uint32_t w[4] = {a.x, a.y, b.x, b.y};
            __builtin_memcpy(&f, w, sizeof w);
        } else {
            __builtin_memcpy(&f, r, sizeof r);
        }
        return f;
    }
    __device__ __forceinline__ void put(typename LinOp<IO == IO_F32>::E *p) const {
        const auto f = frag();
        __builtin_memcpy(__builtin_assume_aligned(p, 16), &f, sizeof f);
    }
};

// One tensor of a sweep: the chunk's rows through a descriptor that moves with the chunk.  A
// thread has rows r0 + ROWS i and one place in each, so one offset in a register; i moves a scalar
// one.  Byte offsets within a chunk stay below 2^31 (64 rows of at most 2^23 elements); where the
// walk runs backwards they count from the chunk's last row, the lowest in memory.
template <int ROWS, int N>
struct LinStream {
    char *base;     // of the chunk's lowest row
    int step;       // bytes between rows, negative where the walk runs backwards
    uint32_t off;   // of the thread's row of the lowest address, or LIN_NOWHERE
    __device__ __forceinline__ LinStream(const void *p, long long ts, long long bs, int es, int b, int h, int d, int chunk, int r0, int e) {
        step = (int)ts * es;
        base = static_cast<char *>(const_cast<void *>(p)) + ((long long)b * bs + (long long)h * d) * es +
               ((long long)chunk * LIN_CHUNK + (step < 0 ? LIN_CHUNK - 1 : 0)) * step;
        off = e < d ? (uint32_t)((step < 0 ? (r0 + ROWS * (N - 1) - (LIN_CHUNK - 1)) : r0) * step + e * es) : LIN_NOWHERE;
    }
    __device__ __forceinline__ void next() { base += (long long)LIN_CHUNK * step; }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc() const {
        return __builtin_amdgcn_make_buffer_rsrc(base, 0, (int)LIN_NOWHERE, 0x00027000);
    }
    __device__ __forceinline__ int at(int i) const { return step < 0 ? (i - (N - 1)) * ROWS * step : i * ROWS * step; }
};

__device__ __forceinline__ lin_u32x4_t lin_bits(f32x4_t x) {
    lin_u32x4_t r;
    __builtin_memcpy(&r, &x, 16);
    return r;
}

template <bool F32, int DK, int DV, bool OUT1, bool OUT2>
struct LinShared {
    using Op = LinOp<F32>;
    using E = typename Op::E;
    static constexpr bool OUTS = OUT1 || OUT2;
    static constexpr int MP = OUT2 && !F32 ? LIN_PARTS : 1;  // parts of the state
    static constexpr int S1 = DK + Op::PAD, S2 = DV + Op::PAD;
    static __device__ __forceinline__ int at(int n) { return n * S1 + (n >> 3) * Op::SKEW; }  // row n of the state
    E r1[LIN_CHUNK][S1];
    E r2[LIN_CHUNK][S2];
    E m[MP][OUTS ? DV * S1 + DV / 8 * Op::SKEW : 1];
    // of this chunk and the next: G in two parts, the update's weights, e^{G_end}
    float2 G[2][LIN_CHUNK];
    float w[2][LIN_CHUNK];
    float whole[2];
    float ahead;  // of the chunks' factors
};

// Inclusive sum over the 64 lanes, by shifts within rows of 16 lanes and two broadcasts.
template <int CTRL, int ROWS>
__device__ __forceinline__ double lin_shift(double x) {
    uint32_t w[2];
    __builtin_memcpy(w, &x, 8);
    w[0] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[0], CTRL, ROWS, 0xf, false);
    w[1] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[1], CTRL, ROWS, 0xf, false);
    __builtin_memcpy(&x, w, 8);
    return x;
}
__device__ __forceinline__ double lin_scan(double x) {
    x += lin_shift<0x111, 0xf>(x);  // row_shr:1
    x += lin_shift<0x112, 0xf>(x);
    x += lin_shift<0x114, 0xf>(x);
    x += lin_shift<0x118, 0xf>(x);
    x += lin_shift<0x142, 0xa>(x);  // lane 15 of a row to the next row
    x += lin_shift<0x143, 0xc>(x);  // lane 31 to the upper half
    return x;
}

// 2^x in 64 bits, to 2^-40 and more: 2^round(x) times the series of e^y, y = ln 2 (x - round(x)), |y| <= 0.35, whose
// first term left out, y^11 / 11!, is below 3e-13.
__device__ __forceinline__ double lin_exp2(double x) {
    constexpr double C[11] = {1.0,         1.0,          1.0 / 2,       1.0 / 6,        1.0 / 24,     1.0 / 120,
                              1.0 / 720,   1.0 / 5040,   1.0 / 40320,   1.0 / 362880,   1.0 / 3628800};
    const double n = rint(x), y = (x - n) * 0.69314718055994530942;
    double p = C[10];
#pragma unroll
    for (int k = 9; k >= 0; --k) p = p * y + C[k];
    return ldexp(p, (int)fmax(fmin(n, 2000.0), -2000.0));
}

// N times eight neighbouring channels, 32 apart, to an output's row.  The offset is all in the vector register (and the
// instruction): behind a store of 16 bytes whose scalar offset is a register the compiler leaves no wait before its
// data registers are written again, and they were: word 0 of lanes 4 to 7 came out as the next store's.
template <bool F32, int N>
__device__ __forceinline__ void lin_store(const f32x4_t (&o)[2 * N], __amdgpu_buffer_rsrc_t rsrc, uint32_t off) {
    constexpr int NT = 2;  // the non-temporal hint
#pragma unroll
    for (int s = 0; s < N; ++s) {
        if constexpr (F32) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                lin_u32x4_t v;
                __builtin_memcpy(&v, &o[2 * s + u], 16);
                __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, off + 128 * s + 16 * u, 0, NT);
            }
        } else {
            const f32x4_t x = o[2 * s], y = o[2 * s + 1];
            const lin_u32x4_t v = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
            __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, off + 64 * s, 0, NT);
        }
    }
}

// Block: one (batch, head) pair and one segment of chunks, walked in order.  A wave has 16 own
// tokens (so causality halves its products without a mask over whole tiles), with eight waves
// half of their outputs' channels, and its share of the state's accumulators.  Own operands
// come straight from memory into fragments; rows and state are staged in LDS.  All products are
// formed transposed (own token = column), so that P passes from accumulators to operand in
// registers and a lane ends with eight neighbouring outputs of one token.
//
// A chunk's steps (LDS reads, dependent matrix instructions, two barriers) follow one another, so the time
// is their latency, in part hidden by the other waves: eight waves of half the work, four to a SIMD, against four that
// form the scores once, not twice: dq of 32,760 tokens of 20 heads 424 us against 509, the forward outputs of 2 x 32,760
// of 32 heads 615 against 632.  (2 x 32,760 of 32 heads: outputs 536-640 us, states 230-280, by the card's clock, which
// falls to 1.75 GHz in long runs.)
// IO is the type of q, k, v; a tensor among the operands that is an output's gradient has the
// output's (WIDE).
template <int IO, int DK, int DV, bool OUT1, bool OUT2, bool WIDE>
__global__ void __launch_bounds__(64 * lin_waves(DK, DV), lin_waves(DK, DV) / (OUT2 || IO == IO_F32 ? 4 : 2)) linear_sweep_kernel(const LinSweep a) {
    constexpr bool F32 = IO == IO_F32;
    constexpr int IO_R2 = WIDE && (OUT1 || !OUT2) ? OutIo<IO> : IO, IO_A2 = WIDE && OUT2 && !OUT1 ? OutIo<IO> : IO;
    using Op = LinOp<F32>;
    using Frag = typename Op::Frag;
    constexpr bool OUTS = OUT1 || OUT2;
    using Shared = LinShared<F32, DK, DV, OUT1, OUT2>;
    constexpr int MP = Shared::MP, S1 = Shared::S1, S2 = Shared::S2;
    constexpr int KS = DK / 32, VS = DV / 32;      // steps of 32 terms
    extern __shared__ __align__(16) unsigned char lin_smem[];
    auto &sm = *reinterpret_cast<Shared *>(lin_smem);

    constexpr int WAVES = lin_waves(DK, DV), THREADS = 64 * WAVES, HALVES = WAVES / 4;
    constexpr int T1 = DV / 16 / HALVES, T2 = DK / 16 / HALVES;  // 16-channel tiles of a wave's outputs
    const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int w = wave & 3, half = wave >> 2;  // own tokens 16 w .. 16 w + 15
    const int segs = OUTS ? a.nseg : a.nseg - 1;
    const int lp = blockIdx.x / segs, seg = blockIdx.x % segs;
    const int pair = a.pair0 + lp, b = pair / a.H, h = pair % a.H;
    const int c0 = seg == 0 ? 0 : a.seg_first + (seg - 1) * a.seg_chunks;
    const int c1 = min(a.seg_first + seg * a.seg_chunks, a.chunks);
    const int dk = a.dk, dv = a.dv;
    const size_t SZ = (size_t)dk * dv;

    // ---- loads of a chunk into registers
    constexpr int V1 = LIN_CHUNK * DK / 8 / THREADS, V2 = LIN_CHUNK * DV / 8 / THREADS;  // vectors of eight a thread
    constexpr int R1 = LIN_CHUNK / V1, R2 = LIN_CHUNK / V2;  // rows between a thread's vectors
    const int r1r = tid / (DK / 8), r1e = tid % (DK / 8) * 8, r2r = tid / (DV / 8), r2e = tid % (DV / 8) * 8;
    LinStream<R1, V1> r1(a.r1.p, a.r1.ts, a.r1.bs, io_in_bytes(IO), b, h, dk, c0, r1r, r1e);
    LinStream<R2, V2> r2(a.r2.p, a.r2.ts, a.r2.bs, io_in_bytes(IO_R2), b, h, dv, c0, r2r, r2e);
    // own operands: one row, channels 32 s + 8 g
    LinStream<LIN_CHUNK, 1> a1s(OUTS ? a.a1.p : a.r1.p, a.a1.ts, a.a1.bs, io_in_bytes(IO), b, h, dk, c0, 16 * w + l, 8 * g);
    LinStream<LIN_CHUNK, 1> a2s(OUT2 ? a.a2.p : a.r2.p, a.a2.ts, a.a2.bs, io_in_bytes(IO_A2), b, h, dv, c0, 16 * w + l, 8 * g);
    LinRaw<IO> t1[V1];
    LinRaw<IO_R2> t2[V2];
    const float *gate = a.decay + b * a.g_bs + h;
    float ga = 1.0f;
    const auto real = [&](int t) { return t >= a.lo && t < a.hi; };
    const auto load_rows = [&](int c) {
        const auto p1 = r1.rsrc(), p2 = r2.rsrc();
#pragma unroll
        for (int i = 0; i < V1; ++i) t1[i].load(p1, real(c * LIN_CHUNK + r1r + R1 * i) ? r1.off : LIN_NOWHERE, r1.at(i));
#pragma unroll
        for (int i = 0; i < V2; ++i) t2[i].load(p2, real(c * LIN_CHUNK + r2r + R2 * i) ? r2.off : LIN_NOWHERE, r2.at(i));
        r1.next();
        r2.next();
    };
    LinRaw<IO> n1[OUTS ? KS : 1];
    LinRaw<IO_A2> n2[OUT2 ? VS : 1];
    const auto load_own = [&](int c) {
        const bool in = real(c * LIN_CHUNK + 16 * w + l);
        const auto p1 = a1s.rsrc();
        // (channels beyond a head of 16, the only one that is no multiple of 32, are masked by the offset)
#pragma unroll
        for (int s = 0; s < KS; ++s) n1[s].load(p1, in ? a1s.off : LIN_NOWHERE, 32 * s * io_in_bytes(IO));
        a1s.next();
        if constexpr (OUT2) {
            const auto p2 = a2s.rsrc();
#pragma unroll
            for (int s = 0; s < VS; ++s) n2[s].load(p2, in ? a2s.off : LIN_NOWHERE, 32 * s * io_in_bytes(IO_A2));
            a2s.next();
        }
    };
    // outputs: one row, this lane's first channel of this wave's half
    constexpr int OIO = OutIo<IO>;
    LinStream<LIN_CHUNK, 1> s1(a.out1.p, a.out1.ts, a.out1.bs, io_in_bytes(OIO), b, h, dv, c0, 16 * w + l, half * (DV / HALVES) + 8 * g);
    LinStream<LIN_CHUNK, 1> s2(a.out2.p, a.out2.ts, a.out2.bs, io_in_bytes(OIO), b, h, dk, c0, 16 * w + l, half * (DK / HALVES) + 8 * g);

    // Wave 0 forms a chunk's sums a chunk ahead, from gates loaded another chunk earlier (and before
    // it asks for the chunk's rows: the wait for a gate is one for every load before it).
    double total = 0.0;  // sum of logarithms over the segment (wave 0)
    const auto load_gate = [&](int c) {
        const int t = c * LIN_CHUNK + lane;
        ga = gate[(long long)min(max(t, a.lo), a.hi - 1) * a.g_ts];
        if (!real(t)) ga = 1.0f;
    };
    const auto sum_gates = [&](int c) {
        float lg = log2f(ga);
        if (lg < -200.0f) lg = -200.0f;  // resets; a NaN stays one
        double x = lin_scan(lg);
        const double end = __shfl(x, 63);
        if (a.exclusive) x -= lg;
        const float hi = (float)x;
        sm.G[c & 1][lane] = make_float2(hi, (float)(x - hi));
        sm.w[c & 1][lane] = __builtin_amdgcn_exp2f((float)(end - x)) * a.scale_upd;
        // A chunk's factor comes from its logarithm in two parts, one step off however large the logarithm.  A decay per head
        // makes every chunk's factor the same, and that step would be raised to the number of chunks a state lives (4,096
        // tokens of memory: up to 1e-6): `ahead` is the logarithm of the factors' product over that of the exact ones, and
        // each factor takes it back.  Only where a chunk halves the state at most: there `ahead` is known to 2^-24, while
        // behind a strong decay (2^-99 of one token: 2^-18) it would be handed to what came in behind that decay;
        // and what is halved oftener does not live long enough for its steps to add up.
        const double due = c == c0 ? end : end - sm.ahead;
        const float due_hi = (float)due, due_lo = (float)(due - due_hi);
        float f = __builtin_amdgcn_exp2f(due_hi);
        f += f * (0.69314718f * due_lo);
        if (lane == 0) {
            sm.whole[c & 1] = f;
            sm.ahead = due >= -1.0 && due <= 1.0 ? (float)(log2f(f) - due) : 0.0f;
        }
        total += end;
    };

    // ---- the state: rows d = wd + 16 i + 4 g + s, columns n = wn + 16 j + l of the accumulators.
    // A wave has all d of its columns where there are tiles enough, so that the weighted operand of
    // the update is formed once in a block.
    constexpr int WN = DV / 16 < WAVES ? DV / 16 : WAVES, WD = WAVES / WN;
    constexpr int TD = DK / 16 / WD, TN = DV / 16 / WN;
    const int wd = wave / WN * (DK / WD), wn = wave % WN * (DV / WN);
    f32x4_t M[TD][TN];
    const float *start = nullptr;
    if constexpr (OUTS)
        start = a.slots ? a.slots + ((size_t)lp * a.nslots + seg) * SZ : a.state_in ? a.state_in + lp * SZ : nullptr;
#pragma unroll
    for (int i = 0; i < TD; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int d = wd + 16 * i + 4 * g, n = wn + 16 * j + l;
            M[i][j] = f32x4_t{0, 0, 0, 0};
            if (start && d < dk && n < dv) M[i][j] = *reinterpret_cast<const f32x4_t *>(start + (size_t)n * dk + d);
        }

    if (wave == 0) load_gate(c0);
    load_rows(c0);
    if constexpr (OUTS) load_own(c0);
    if (wave == 0) {
        sum_gates(c0);
        if (c0 + 1 < c1) load_gate(c0 + 1);
    }

    for (int c = c0; c < c1; ++c) {
        __syncthreads();  // the last chunk's reads are done
#pragma unroll
        for (int i = 0; i < V1; ++i) t1[i].put(&sm.r1[r1r + R1 * i][r1e]);
#pragma unroll
        for (int i = 0; i < V2; ++i) t2[i].put(&sm.r2[r2r + R2 * i][r2e]);
        if constexpr (OUTS) {
#pragma unroll
            for (int i = 0; i < TD; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const int d = wd + 16 * i + 4 * g, n = wn + 16 * j + l;
                    f32x4_t x = M[i][j];
                    if constexpr (F32) {
                        *reinterpret_cast<f32x4_t *>(&sm.m[0][Shared::at(n) + d]) = x;
                    } else {
#pragma unroll
                        for (int k = 0; k < MP; ++k) {
                            const uint2 y = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
                            *reinterpret_cast<uint2 *>(&sm.m[k][Shared::at(n) + d]) = y;
                            x -= f32x4_t{bf16_lo(y.x), bf16_hi(y.x), bf16_lo(y.y), bf16_hi(y.y)};
                        }
                    }
                }
        }
        __syncthreads();
        Frag a1[OUTS ? KS : 1], a2[OUT2 ? VS : 1];
        if constexpr (OUTS) {
#pragma unroll
            for (int s = 0; s < KS; ++s) a1[s] = n1[s].frag();
        }
        if constexpr (OUT2) {
#pragma unroll
            for (int s = 0; s < VS; ++s) a2[s] = n2[s].frag();
        }
        if (c + 1 < c1) {
            if (wave == 0) {
                sum_gates(c + 1);
                if (c + 2 < c1) load_gate(c + 2);
            }
            load_rows(c + 1);
        }

        if constexpr (OUTS) {
            const float2 Gc = sm.G[c & 1][16 * w + l];
            const float cross = __builtin_amdgcn_exp2f(Gc.x + Gc.y) * a.scale_cross;
            f32x4_t o1[OUT1 ? T1 : 1], o2[OUT2 ? T2 : 1];
            const int n1st = half * (DV / HALVES), d1st = half * (DK / HALVES);  // first channels of this wave
            float wsum = 0.0f, xsum = 0.0f;
            // what the state holds
            if constexpr (OUT1) {
#pragma unroll
                for (int t = 0; t < T1; ++t) {
                    const int n = n1st + 32 * (t / 2) + 8 * (l >> 2) + 4 * (t & 1) + (l & 3);
                    f32x4_t y = {0, 0, 0, 0};
#pragma unroll
                    for (int s = 0; s < KS; ++s) y = Op::mma(Op::row(&sm.m[0][Shared::at(n) + 32 * s + 8 * g]), a1[s], y);
                    o1[t] = y * cross;
                }
            }
            if constexpr (OUT2) {
#pragma unroll
                for (int t = 0; t < T2; ++t) {
                    const int c0t = d1st + 32 * (t / 2) + 4 * (t & 1);
                    f32x4_t y = {0, 0, 0, 0};
#pragma unroll
                    for (int s = 0; s < VS; ++s) {
#pragma unroll
                        for (int k = MP - 1; k >= 0; --k)
                            y = Op::mma(Op::template col<false>(&sm.m[k][Shared::at(32 * s) + c0t], S1, Shared::at(8), 8, l, g), a2[s], y);
                    }
                    o2[t] = y * cross;
                    float f[8];
                    Op::get(half ? a1[HALVES > 1 ? T2 / 2 + t / 2 : 0] : a1[t / 2], f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) xsum += f[4 * (t & 1) + e] * o2[t][e];
                }
            }
            // the chunk's own tokens, 32 rows at a time
#pragma unroll
            for (int tp = 0; tp < 2; ++tp) {
                if (2 * tp > w) continue;
                f32x4_t p[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}}, q[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    // (The second half of an even wave's last 32 rows is all above the diagonal, but is formed all
                    // the same: with a branch around it the compiler reads the first half's products 3 to 6
                    // instructions after the last matrix instruction, where the hardware needs 8.)
                    const int r0 = 32 * tp + 16 * u;
#pragma unroll
                    for (int s = 0; s < KS; ++s) p[u] = Op::mma(Op::row(&sm.r1[r0 + l][32 * s + 8 * g]), a1[s], p[u]);
                    if constexpr (OUT2) {
#pragma unroll
                        for (int s = 0; s < VS; ++s)
                            q[u] = Op::mma(Op::row(&sm.r2[r0 + l][32 * s + 8 * g]), a2[s], q[u]);
                    }
                }
                float pf[8], qf[8];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int r = 32 * tp + 16 * u + 4 * g + e, col = 16 * w + l;
                        const float2 Gr = sm.G[c & 1][r];
                        const float D = __builtin_amdgcn_exp2f((Gc.x - Gr.x) + (Gc.y - Gr.y)) * a.scale_d;
                        // selected, not multiplied: behind a reset or the diagonal D may be infinite
                        pf[4 * u + e] = r <= col ? p[u][e] * D : 0.0f;
                        if constexpr (OUT2) {
                            qf[4 * u + e] = r <= col ? q[u][e] * D : 0.0f;
                            wsum += r < col ? pf[4 * u + e] * q[u][e] : 0.0f;
                        }
                    }
                if constexpr (OUT1) {
                    const Frag f = Op::pack(pf);
#pragma unroll
                    for (int t = 0; t < T1; ++t)
                        o1[t] = Op::mma(Op::template col<true>(&sm.r2[32 * tp][n1st + 32 * (t / 2) + 4 * (t & 1)], S2, 4 * S2, 8, l, g), f, o1[t]);
                }
                if constexpr (OUT2) {
                    const Frag f = Op::pack(qf);
#pragma unroll
                    for (int t = 0; t < T2; ++t)
                        o2[t] = Op::mma(Op::template col<true>(&sm.r1[32 * tp][d1st + 32 * (t / 2) + 4 * (t & 1)], S1, 4 * S1, 8, l, g), f, o2[t]);
                }
            }
            const long long t = (long long)c * LIN_CHUNK + 16 * w + l;
            const bool in = real((int)t);
            if constexpr (OUT1) {
                if (a.out1.p) lin_store<F32, T1 / 2>(o1, s1.rsrc(), in ? s1.off : LIN_NOWHERE);
                s1.next();
            }
            if constexpr (OUT2) {
                if (a.out2.p) lin_store<F32, T2 / 2>(o2, s2.rsrc(), in ? s2.off : LIN_NOWHERE);
                s2.next();
            }
            if constexpr (OUT2) {
                wsum += __shfl_xor(wsum, 16);
                wsum += __shfl_xor(wsum, 32);
                xsum += __shfl_xor(xsum, 16);
                xsum += __shfl_xor(xsum, 32);
                if (g == 0) {  // padded tokens too: their sums are zero
                    const long long i = (long long)lp * a.chunks * LIN_CHUNK + (a.dot_step > 0 ? t : (long long)a.chunks * LIN_CHUNK - 1 - t);
                    if (half == 0) a.dot_w[i] = wsum;
                    a.dot_x[half * a.dot_half + i] = xsum;
                    if (HALVES == 1) a.dot_x[a.dot_half + i] = 0.0f;
                }
            }
        }

        // the next chunk's own operands take the registers of this one's
        if constexpr (OUTS) {
            if (c + 1 < c1) load_own(c + 1);
        }

        // ---- M <- e^{G_end} M + sum_r w_r r2_r r1_r^T
        // fp32 adds up 32 tokens first: with each instruction's four terms rounded to M's size, states of 4,096 tokens of
        // memory were 8e-7 off (2e-7 so).  bf16 instructions add 32 terms each and go straight to M (6e-7 off; with sums
        // first 1.3e-7, and the registers for them cost 7%: 2 x 32,760 of 32 heads 982 us against 912).
        const float whole = sm.whole[c & 1];
#pragma unroll
        for (int i = 0; i < TD; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) M[i][j] *= whole;
#pragma unroll
        for (int ks = 0; ks < LIN_CHUNK / 32; ++ks) {
            float wt[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) wt[e] = sm.w[c & 1][32 * ks + (e < 4 ? 4 * g + e : 12 + 4 * g + e)];
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                float f[8];
                Op::get(Op::template col<true>(&sm.r2[32 * ks][wn + 16 * j], S2, 4 * S2, 4, l, g), f);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] *= wt[e];
                Frag part[F32 ? 1 : LIN_PARTS];
                part[0] = Op::pack(f);
#pragma unroll
                for (int n = 1; n < (F32 ? 1 : LIN_PARTS); ++n) {
                    float fh[8];
                    Op::get(part[n - 1], fh);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] -= fh[e];
                    part[n] = Op::pack(f);
                }
#pragma unroll
                for (int i = 0; i < TD; ++i) {
                    const Frag A = Op::template col<true>(&sm.r1[32 * ks][wd + 16 * i], S1, 4 * S1, 4, l, g);
                    if constexpr (F32) {
                        M[i][j] += Op::mma(A, part[0], f32x4_t{0, 0, 0, 0});
                    } else {
#pragma unroll
                        for (int n = 0; n < LIN_PARTS; ++n) M[i][j] = Op::mma(A, part[n], M[i][j]);
                    }
                }
            }
        }
    }

    float *end = nullptr;
    if constexpr (OUTS) {
        if (seg == a.nseg - 1 && a.state_out) end = a.state_out + lp * a.so_stride;
    } else {
        end = a.slots + ((size_t)lp * a.nslots + seg + 1) * SZ;
        if (tid == 0) {
            const double p = lin_exp2(total);
            a.gamma[(size_t)lp * a.nslots + seg] = make_float2((float)p, (float)(p - (float)p));
        }
    }
    if (end) {
#pragma unroll
        for (int i = 0; i < TD; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int d = wd + 16 * i + 4 * g, n = wn + 16 * j + l;
                if (d < dk && n < dv) *reinterpret_cast<f32x4_t *>(end + (size_t)n * dk + d) = M[i][j];
            }
    }
}

template <int IO, int DK, int DV, bool OUT1, bool OUT2, bool WIDE>
hipError_t linear_sweep_launch(const LinSweep &a, int pairs, hipStream_t stream) {
    constexpr size_t lds = sizeof(LinShared<IO == IO_F32, DK, DV, OUT1, OUT2>);
    static_assert(lds <= 160 * 1024, "LDS of a CU");
    const auto kernel = linear_sweep_kernel<IO, DK, DV, OUT1, OUT2, WIDE>;
    if (lds > 64 * 1024) {
        hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    const long long blocks = (long long)pairs * (OUT1 || OUT2 ? a.nseg : a.nseg - 1);
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(64 * lin_waves(DK, DV)), lds, stream, a);
    return hipGetLastError();
}

// Head dims of 16 run in tiles of 32, the rest of them zeros.
template <int IO, bool OUT1, bool OUT2, bool WIDE>
hipError_t linear_sweep_dims(const LinSweep &a, int pairs, hipStream_t stream) {
    const int DK = a.dk < 32 ? 32 : a.dk, DV = a.dv < 32 ? 32 : a.dv;
#define GDN_LIN(K, V) \
    if (DK == K && DV == V) return linear_sweep_launch<IO, K, V, OUT1, OUT2, WIDE>(a, pairs, stream);
    GDN_LIN(32, 32) GDN_LIN(32, 64) GDN_LIN(32, 128)
    GDN_LIN(64, 32) GDN_LIN(64, 64) GDN_LIN(64, 128)
    GDN_LIN(128, 32) GDN_LIN(128, 64) GDN_LIN(128, 128)
#undef GDN_LIN
    return hipErrorInvalidValue;
}

}  // namespace gdn
