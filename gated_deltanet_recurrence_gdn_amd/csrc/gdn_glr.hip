// gdn_glr.hip -- the diagonal gated linear recurrence h_t = a_t h_{t-1} + b_t v_t and its
// gradient (include/gdn.h, gdn_glr_forward / gdn_glr_backward).
//
// Measured (a copy of 1 GB: 5.1 TB/s): 32,760 tokens of 2,560 channels, gates per channel, bf16:
// 134 us, 5.0 TB/s; 2 x 32,760 tokens of 32 heads of 128, gates per head: forward 232 us,
// gradient 428 us, 4.6 and 3.8 TB/s; one token of 64 x 2,560 channels 2.4 us.
//
// The pass is bound by HBM: 3 flops per element read and written.  A block takes a tile
// of W * R tokens by 128 channels (two per lane, so that a wave reads whole lines of a
// token's row), reads it once into registers and writes its outputs once.  The map of R
// tokens of a wave is h -> A h + H with A the product of the decays; the waves' maps are
// joined through LDS, the tiles' maps through the chain below, and with its start state a
// wave then runs its tokens in order.  The sums of a state are fp32 throughout.
//
// The chain between tiles.  A block that needs the state before its tile publishes the
// tile's map (A, H) and looks back over its predecessors' words for the nearest one with a
// known end state, folds the maps in between from the oldest to the newest, and publishes
// its own end state.  The fold is the same sequence of operations whatever is found when,
// so results do not depend on timing.
//  * Every wait ends: a block draws its tile number from a counter when it starts
//    running, and waits only for smaller numbers of the same channels, which running blocks
//    have drawn; the smallest of them waits for nobody.
//  * A published word is 64 bits, value and the call's number, read and written by single
//    relaxed atomics at device scope: nothing else has to be ordered around it.
//  * A block that waits asks for one channel's words: whole rows of words in every round would
//    fill the fabric that the tokens come through.
//  * Two waves look back, 64 channels each, four maps at a time.  Where a call has few slabs its
//    time is mostly that of the chain: there all eight waves take 16 channels each and sixteen
//    maps at a time, up to 64 tiles back, at the price of a barrier (see few_slabs).
//  * The block that draws a slab's last number sets the counter to the next call's number
//    and 0, so a call leaves the workspace ready for the next one (or for its own
//    replay in a graph) without a clearing pass.  The call's number has 32 bits.
#include "gdn_elem.h"
#include "gdn_layer.h"

#include <algorithm>

namespace gdn {
namespace {

constexpr int LANES = 64, SLAB = 2 * LANES;  // channels of a block
constexpr int WAVES = 8;
constexpr int LOOK = 16;                     // how far back a wave looks at once
constexpr int OWN = SLAB / WAVES, FEW = 8;   // channels of a wave of eight that look back; up to FEW slabs

// Tokens of a wave.  The chain costs a tile some microseconds whatever its size, so tiles are
// as long as their inputs fit in registers with two blocks on a CU (128 registers a lane): with
// 16 forward and 8 backward instead of 64 and 16 the training step of two clips with gates per
// head is 20% slower; 32 backward spill.
constexpr int fwd_tokens(int io, bool ch) { return ch ? 16 : io == IO_F32 ? 32 : 64; }
constexpr int bwd_tokens(int io, bool ch) { return ch ? 8 : 16; }

typedef unsigned long long u64;

// The chain's words.  Word i of a plane belongs to channel i % SLAB of slab
// (i / SLAB) % slabs at tile i / (SLAB * slabs), in the order of the walk.
struct Chain {
    u64 *counter;         // [slabs]: number of calls made << 32 | tiles drawn in this one
    u64 *end, *mul, *add; // planes: end state, and the map of one tile
    int slabs;            // B * ceil(C / SLAB)
    int tiles;
};

__device__ __forceinline__ u64 word(uint32_t call, float x) { return (u64)call << 32 | __float_as_uint(x); }
__device__ __forceinline__ float value(u64 w) { return __uint_as_float((uint32_t)w); }
__device__ __forceinline__ u64 peek(const u64 *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void post(u64 *p, u64 w) {
    __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool known(u64 w, uint32_t call) {  // in every lane of the wave
    return __all((uint32_t)(w >> 32) == call);
}

// The maps a lane has found behind it, a channel per thread: kept in LDS, since the waves that
// look back hold their tokens in registers meanwhile.
struct Window {
    float m[LOOK][SLAB], d[LOOK][SLAB];
    int back;
};

// State before tile k > 0 of channel i of the slab; one whole wave.  `at` and `mat` are its
// words of tile k in the planes end and add, and in mul (one word per head where a head has
// one gate: `first` marks the lane that writes it).  (A, H) is the tile's own map.
__device__ float state_before(const Chain &c, Window &win, int i, uint32_t call, int k, size_t at, size_t mat, bool first,
                              float A, float H) {
    const size_t step = (size_t)c.slabs * SLAB;
    const int lane = threadIdx.x % LANES, far = k < LOOK ? k : LOOK;
    post(c.add + at, word(call, H));
    if (first) post(c.mul + mat, word(call, A));
    for (;;) {
        // Lane l asks for one word of the tile l + 1 back: whole rows of words in every
        // round would fill the fabric that the tokens come through.
        const u64 e = peek(c.end + at - lane - step * (lane < far ? lane + 1 : far));
        const u64 found = __ballot(lane < far && (uint32_t)(e >> 32) == call);
        if (found) {
            // the nearest known end state, and the maps of the tiles behind it
            const int j = __ffsll(found);
            const u64 end = peek(c.end + at - step * j);
            bool ok = true;
#pragma unroll 1
            for (int g = 1; g < j; g += 4) {
                u64 wm[4], wd[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const size_t back = step * (g + q < j ? g + q : j - 1);
                    wm[q] = peek(c.mul + mat - back);
                    wd[q] = peek(c.add + at - back);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (g + q < j) {
                        win.m[g + q - 1][i] = value(wm[q]);
                        win.d[g + q - 1][i] = value(wd[q]);
                        ok &= known(wm[q], call) && known(wd[q], call);
                    }
            }
            if (ok && known(end, call)) {
                float s = value(end);
#pragma unroll 1
                for (int q = j - 2; q >= 0; --q) s = fmaf(win.m[q][i], s, win.d[q][i]);
                return s;
            }
        }
        __builtin_amdgcn_s_sleep(1);
    }
}

// Between lanes of one wave that write LDS and others that read it (and before it is written
// anew): the order that the compiler has to keep.  LDS serves a wave's accesses in order, so
// no instruction comes of it.
__device__ __forceinline__ void wave_order_lds() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// State before tile k > 0 of channel `c` of the slab; the whole block, lanes l, l + 16, l + 32
// and l + 48 of wave w for channel 16 w + l.  `base` is the slab's first word of tile k;
// `share` channels have one word in the plane mul.  (A, H) is the tile's own map.
__device__ float state_before_by_block(const Chain &ch, Window &win, uint32_t call, int k, size_t base, int share, float A,
                                       float H) {
    const size_t step = (size_t)ch.slabs * SLAB;
    const int lane = threadIdx.x % LANES, wave = threadIdx.x / LANES, c = wave * OWN + lane % OWN, q = lane / OWN;
    const size_t at = base + c, mat = at - c % share;
    if (q == 0) {
        post(ch.add + at, word(call, H));
        if (c % share == 0) post(ch.mul + mat, word(call, A));
    }
    if (wave == 0) {
        // lane l: the tile l + 1 back; the nearest known end state with known maps behind it
        const int far = k < LANES ? k : LANES;
        const size_t there = base - step * (lane < far ? lane + 1 : far);
        int j;
        for (;;) {
            const u64 e = peek(ch.end + there), d = peek(ch.add + there);
            const u64 ends = __ballot(lane < far && (uint32_t)(e >> 32) == call);
            const u64 maps = __ballot((uint32_t)(d >> 32) == call);
            j = __ffsll(ends);
            const u64 behind = j ? ((u64)1 << (j - 1)) - 1 : 0;
            if (j && (maps & behind) == behind) break;
            __builtin_amdgcn_s_sleep(1);
        }
        if (lane == 0) win.back = j;
    }
    __syncthreads();
    // These words are there or on their way: the blocks that post them do not wait for this one.
    const int j = win.back;
    u64 e;
    do e = peek(ch.end + at - step * j);
    while (!known(e, call));
    float s = value(e);
#pragma unroll 1
    for (int hi = j - 1; hi >= 1; hi -= 16) {
        u64 wm[4], wd[4];
        bool ok;
        do {
            ok = true;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int o = hi - 4 * u - q;
                const size_t back = step * (o >= 1 ? o : 1);
                wm[u] = peek(ch.mul + mat - back);
                wd[u] = peek(ch.add + at - back);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) ok = ok && known(wm[u], call) && known(wd[u], call);
        } while (!ok);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            win.m[4 * u + q][c] = value(wm[u]);
            win.d[4 * u + q][c] = value(wd[u]);
        }
        wave_order_lds();  // the four lanes of a channel read what all four wrote
        const int n = hi < 16 ? hi : 16;
#pragma unroll 1
        for (int t = 0; t < n; ++t) s = fmaf(win.m[t][c], s, win.d[t][c]);
        wave_order_lds();
    }
    return s;
}

// Two neighbouring elements, as they lie in memory: elements c and c + 1 of a row.  bf16 and
// FP8 rows are read past the caches (the training step of two clips 643 us against 655); fp32
// ones are not, which the gradient right behind a forward pass finds there (25 us against 26 at
// 3 x 1,561 x 320).
template <int IO>
struct Pair;
template <>
struct Pair<IO_F32> {
    float2 r;
    static constexpr int BYTES = 4;
    __device__ __forceinline__ void load(const char *row, unsigned c) { r = *reinterpret_cast<const float2 *>(row + c * 4); }
    __device__ __forceinline__ void zero() { r = make_float2(0.0f, 0.0f); }
    __device__ __forceinline__ float2 get() const { return r; }
    static __device__ __forceinline__ void store(char *row, unsigned c, float2 x) {
        const f32x2_t v = {x.x, x.y};
        stream_out(reinterpret_cast<f32x2_t *>(row + c * 4), v);
    }
};
template <>
struct Pair<IO_BF16> {
    uint32_t r;
    static constexpr int BYTES = 2;
    __device__ __forceinline__ void load(const char *row, unsigned c) { r = stream_in(reinterpret_cast<const uint32_t *>(row + c * 2)); }
    __device__ __forceinline__ void zero() { r = 0; }
    __device__ __forceinline__ float2 get() const { return make_float2(bf16_lo(r), bf16_hi(r)); }
    static __device__ __forceinline__ void store(char *row, unsigned c, float2 x) {
        stream_out(reinterpret_cast<uint32_t *>(row + c * 2), pack_bf16x2(x.x, x.y));
    }
};
template <>
struct Pair<IO_FP8> {
    uint32_t r;
    static constexpr int BYTES = 1;
    __device__ __forceinline__ void load(const char *row, unsigned c) { r = stream_in(reinterpret_cast<const uint16_t *>(row + c)); }
    __device__ __forceinline__ void zero() { r = 0; }
    __device__ __forceinline__ float2 get() const {
        float f[4];
        fp8x4_to_f32(r, f);
        return make_float2(f[0], f[1]);
    }
};
// Makes the compiler forget what it formed from these registers: widened copies kept from one
// pass over the tokens to the next would take twice the registers.
template <int R, int IO>
__device__ __forceinline__ void anew(Pair<IO> (&v)[R]) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if constexpr (IO == IO_F32)
            asm volatile("" : "+v"(v[r].r.x), "+v"(v[r].r.y));
        else
            asm volatile("" : "+v"(v[r].r));
    }
}
// Keeps the loads of one stretch of tokens from being moved before those of the last.
__device__ __forceinline__ void stretch(int r) {
    if (r % 8 == 0) __builtin_amdgcn_sched_barrier(0);
}
template <int IO>
using OutPair = Pair<IO == IO_F32 ? IO_F32 : IO_BF16>;

// The gates of a wave's R tokens.  Per channel: in registers.  Per head: the tile's gates of
// the slab's heads are staged in LDS by the block (one load per token and head instead of one
// per lane) as a row of tokens per head, and read from there where they are used; a row's
// pitch of four more keeps the up to eight heads of a wave on different banks.
template <bool CH, int R>
struct Gates;
template <int R>
struct Gates<true, R> {
    float2 r[R];
    static constexpr int STAGE = 1;
    __device__ __forceinline__ float2 get(int i) const { return r[i]; }
};
template <int R>
struct Gates<false, R> {
    const float *r;
    static constexpr int PITCH = WAVES * R + 4, STAGE = PITCH * (SLAB / 16);
    // The whole block, before the barrier that precedes get.  Past the end stands `past`.
    __device__ __forceinline__ void stage(float *lds, const float *p, const GlrArgs &a, int b, int slab_c0, long long tile0,
                                          int tokens, float past) {
        const int heads = SLAB / a.d, h0 = slab_c0 / a.d;
        for (int i = threadIdx.x; i < tokens * heads; i += blockDim.x) {
            const long long t = tile0 + i / heads;
            const int h = h0 + i % heads < a.H ? h0 + i % heads : a.H - 1;
            lds[i % heads * PITCH + i / heads] = t < a.T ? p[((size_t)b * a.T + (a.reverse ? a.T - 1 - t : t)) * a.H + h] : past;
        }
    }
    __device__ __forceinline__ void place(const float *lds, int wave, int lane, int d) {
        r = lds + 2 * lane / d * PITCH + wave * R;
    }
    __device__ __forceinline__ float2 get(int i) const { return make_float2(r[i], r[i]); }
};

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return make_float2(a.x * b.x, a.y * b.y); }

__device__ __forceinline__ float2 &lds2(float *row, int lane) { return reinterpret_cast<float2 *>(row)[lane]; }

// Which slab and tile this block has: a slab's tiles in the order in which its blocks start
// running.  Blocks go round the 8 XCDs in turn; slabs that lie side by side share lines of
// the gates (and of rows that are not whole lines), so they are given to one XCD.
struct Place {
    int slab, tile;
    uint32_t call;
};
__device__ __forceinline__ Place draw(const Chain &c, Place *lds) {
    const unsigned blk = blockIdx.x;
    const int slab = c.slabs % 8 == 0 ? (int)(blk % 8 * (c.slabs / 8) + blk / 8 % (c.slabs / 8)) : (int)(blk % c.slabs);
    if (c.tiles == 1) return {slab, 0, 0};
    if (threadIdx.x == 0) {
        const u64 w = __hip_atomic_fetch_add(c.counter + slab, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const uint32_t call = (uint32_t)(w >> 32) + 1, tile = (uint32_t)w;  // 0 marks what was never written
        if ((int)tile == c.tiles - 1) post(c.counter + slab, (u64)call << 32);
        *lds = {slab, (int)tile, call};
    }
    __syncthreads();
    return *lds;
}

// What a wave has: R tokens from number `first` of the walk on, n of them inside the call.
struct Part {
    int b, c, n;
    unsigned slab_c0;
    bool on;         // lanes past the last channel repeat the last two and write nothing
    long long first, row;  // row of the first token (of the last one of all, if none is inside)
};
__device__ __forceinline__ Part part_of(const GlrArgs &a, const Chain &chain, int slab, long long first, int R, int lane) {
    const int C = a.H * a.d, per = chain.slabs / a.B;
    Part p;
    p.b = slab / per;
    p.slab_c0 = slab % per * SLAB;
    const int c = p.slab_c0 + 2 * lane;
    p.on = c < C;
    p.c = p.on ? c : C - 2;
    p.first = first;
    p.n = a.T - first >= R ? R : a.T > first ? (int)(a.T - first) : 0;
    const long long i = p.n ? first : a.T - 1;
    p.row = (long long)p.b * a.T + (a.reverse ? a.T - 1 - i : i);
    return p;
}

// The R rows of one tensor, row by row from the first token; the rows past the end repeat the
// last one.
template <int R, typename F>
__device__ __forceinline__ void each_row(const void *base, long long row_bytes, const Part &p, int reverse, F f) {
    const char *at = static_cast<const char *>(base) + p.row * row_bytes;
    const long long step = reverse ? -row_bytes : row_bytes;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        f(r, at);
        if (r + 1 < p.n) at += step;
    }
}
template <int R>
__device__ __forceinline__ void load_gates(Gates<true, R> &g, const float *base, int C, const Part &p, int reverse, float past) {
    each_row<R>(base, 4LL * C, p, reverse, [&](int r, const char *at) {
        g.r[r] = *reinterpret_cast<const float2 *>(at + (unsigned)p.c * 4);
    });
    if (p.n < R)
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (r >= p.n) g.r[r] = make_float2(past, past);
}
template <int R, typename P>
__device__ __forceinline__ void load_pairs(P (&v)[R], const void *base, int C, const Part &p, int reverse) {
    each_row<R>(base, (long long)P::BYTES * C, p, reverse, [&](int r, const char *at) { v[r].load(at, p.c); });
    if (p.n < R)
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (r >= p.n) v[r].zero();
}

template <int IO, bool CH, bool BETA, int R, bool FEWS>
__global__ __launch_bounds__(WAVES * LANES, 4) void glr_forward_kernel(GlrArgs a, Chain chain) {
    __shared__ float sA[WAVES][SLAB], sH[WAVES][SLAB], sC[SLAB];
    __shared__ float sGa[Gates<CH, R>::STAGE], sGb[BETA ? Gates<CH, R>::STAGE : 1];
    __shared__ Window window;
    __shared__ Place sP;
    const int lane = threadIdx.x % LANES, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / LANES), waves = blockDim.x / LANES;
    const Place at = draw(chain, &sP);
    const int C = a.H * a.d;
    const long long tile0 = (long long)at.tile * (WAVES * R);
    const Part p = part_of(a, chain, at.slab, tile0 + wave * R, R, lane);

    // Past the end a = 1 and b v = 0: the map that changes nothing.
    Gates<CH, R> ga, gb;
    Pair<IO> v[R];
    load_pairs<R>(v, a.v, C, p, a.reverse);
    if constexpr (CH) {
        load_gates<R>(ga, a.decay, C, p, a.reverse, 1.0f);
        if (BETA) load_gates<R>(gb, a.beta, C, p, a.reverse, 0.0f);
    } else {
        ga.stage(sGa, a.decay, a, p.b, p.slab_c0, tile0, waves * R, 1.0f);
        if (BETA) gb.stage(sGb, a.beta, a, p.b, p.slab_c0, tile0, waves * R, 0.0f);
        ga.place(sGa, wave, lane, a.d);
        if (BETA) gb.place(sGb, wave, lane, a.d);
        __syncthreads();
    }
    // b v: per channel formed once (the gates' registers are free then), per head where it is used
    float2 x[CH ? R : 1];
    if constexpr (CH)
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = BETA ? mul2(gb.get(r), v[r].get()) : v[r].get();
    auto input = [&](int r) { return CH ? x[CH ? r : 0] : BETA ? mul2(gb.get(r), v[r].get()) : v[r].get(); };
    float2 A = {1.0f, 1.0f}, H = {0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < R; ++r) {
        stretch(r);
        A = mul2(A, ga.get(r));
        H = fma2(ga.get(r), H, input(r));
    }
    lds2(sA[wave], lane) = A;
    lds2(sH[wave], lane) = H;
    __syncthreads();
    // the tile's map and start state: a channel per thread of the first two waves, or all waves
    // for 16 channels each
    const int share = CH ? 1 : a.d;  // channels with one decay
    for (int i = FEWS ? wave * OWN + lane % OWN : threadIdx.x; i < SLAB; i += FEWS ? SLAB : blockDim.x) {
        float tA = sA[0][i], tH = sH[0][i], s = 0.0f;
        for (int w = 1; w < waves; ++w) {
            tH = fmaf(sA[w][i], tH, sH[w][i]);
            tA *= sA[w][i];
        }
        const int ch = p.slab_c0 + i;
        const size_t st = (size_t)p.b * C + ch, wd = ((size_t)at.tile * chain.slabs + at.slab) * SLAB + i;
        if (at.tile > 0) {
            if constexpr (FEWS)
                s = state_before_by_block(chain, window, at.call, at.tile, wd - i, share, tA, tH);
            else
                s = state_before(chain, window, i, at.call, at.tile, wd, wd - i % share, i % share == 0, tA, tH);
        } else if (a.state_in && ch < C)
            s = a.state_in[st];
        const float e = fmaf(tA, s, tH);
        if (FEWS && lane >= OWN) continue;  // these lanes repeat the first ones' channels
        if (at.tile + 1 < chain.tiles)
            post(chain.end + wd, word(at.call, e));
        else if (a.state_out && ch < C)
            a.state_out[st] = e;
        sC[i] = s;
    }
    __syncthreads();
    float2 s = lds2(sC, lane);
    for (int w = 0; w < wave; ++w) s = fma2(lds2(sA[w], lane), s, lds2(sH[w], lane));
    const long long marks = (a.T + GLR_TILE - 1) / GLR_TILE;
    if (!CH) anew(v);
    each_row<R>(a.out, (long long)OutPair<IO>::BYTES * C, p, a.reverse, [&](int r, const char *row) {
        stretch(r);
        if (r >= p.n) return;
        if (r % 16 == 0 && a.saved_out && (p.first + r) % GLR_TILE == 0 && p.on)
            *reinterpret_cast<float2 *>(a.saved_out + ((size_t)p.b * marks + (p.first + r) / GLR_TILE) * C + p.c) = s;
        s = fma2(ga.get(r), s, input(r));
        if (p.on) OutPair<IO>::store(const_cast<char *>(row), p.c, s);
    });
}

// One token: a lane has two channels, and nothing is joined.  The same fused product and sum
// as a tile's, so a token on its own gives the bits that it gives as a tile of one.
template <int IO, bool CH, bool BETA>
__global__ __launch_bounds__(256) void glr_step_kernel(GlrArgs a) {
    const unsigned i = 2 * (blockIdx.x * 256 + threadIdx.x);  // channel of the batch
    if (i >= (unsigned)a.B * a.H * a.d) return;
    const char *v = static_cast<const char *>(a.v);
    Pair<IO> x;
    x.load(v, i);
    const unsigned head = i / (unsigned)a.d;
    auto gate = [&](const float *p) {
        return CH ? *reinterpret_cast<const float2 *>(p + i) : make_float2(p[head], p[head]);
    };
    float2 s = {0.0f, 0.0f}, in = x.get();
    if (a.state_in) s = *reinterpret_cast<const float2 *>(a.state_in + i);
    const float2 A = gate(a.decay);
    if (BETA) in = mul2(gate(a.beta), in);
    if (a.saved_out) *reinterpret_cast<float2 *>(a.saved_out + i) = s;
    s = fma2(A, s, in);
    if (a.state_out) *reinterpret_cast<float2 *>(a.state_out + i) = s;
    OutPair<IO>::store(static_cast<char *>(a.out), i, s);
}

// Sums of N = 8 or 16 values over groups of L = 8, 16, 32 or 64 neighbouring lanes.  Each
// step sends half of a lane's values to a partner and adds the partner's other half: N - 1
// moves for N = 16 instead of N log2 L.  Afterwards lane l of a group has value
// l % 8 (N = 8 or L = 8) or l % 16 in v[0], and for N = 16, L = 8 value 8 + l % 8 in v[1].
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], int L, int lane) {
    auto halve = [&](int n, int bit, auto move) {
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float keep = lane & bit ? v[2 * i + 1] : v[2 * i], send = lane & bit ? v[2 * i] : v[2 * i + 1];
            v[i] = keep + move(send);
        }
    };
    halve(N, 1, [](float x) { return dpp_mov<0xB1>(x); });     // lane ^ 1
    halve(N / 2, 2, [](float x) { return dpp_mov<0x4E>(x); });  // lane ^ 2
    halve(N / 4, 4, [](float x) { return __shfl_xor(x, 4); });
    if (L >= 16) {
        if constexpr (N == 16)
            halve(N / 8, 8, [](float x) { return dpp_mov<0x128>(x); });  // row_ror 8: lane ^ 8
        else
            v[0] += dpp_mov<0x128>(v[0]);
    }
    if (L >= 32) v[0] += __shfl_xor(v[0], 16);
    if (L >= 64) v[0] += __shfl_xor(v[0], 32);
}

template <int IO, bool CH, bool BETA, int R, bool FEWS>
__global__ __launch_bounds__(WAVES * LANES, 4) void glr_backward_kernel(GlrArgs a, Chain chain) {
    static_assert(WAVES * R % GLR_TILE == 0 && GLR_TILE % R == 0 && R % 8 == 0, "a tile starts at a saved state");
    __shared__ float sA[WAVES][SLAB], sH[WAVES][SLAB], sG[WAVES][SLAB], sC[SLAB];
    __shared__ float sGa[Gates<CH, R>::STAGE], sGb[BETA ? Gates<CH, R>::STAGE : 1];
    __shared__ Window window;
    __shared__ Place sP;
    const int lane = threadIdx.x % LANES, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / LANES), waves = blockDim.x / LANES;
    const Place at = draw(chain, &sP);
    const int C = a.H * a.d;
    const int tile = chain.tiles - 1 - at.tile;  // the gradient's walk: from the last tile to the first
    const long long tile0 = (long long)tile * (WAVES * R);
    const Part p = part_of(a, chain, at.slab, tile0 + wave * R, R, lane);

    // Past the end a = 1, b v = 0 and dout = 0: both maps change nothing.
    Gates<CH, R> ga, gb;
    Pair<IO> v[R];
    OutPair<IO> dy[R];
    load_pairs<R>(v, a.v, C, p, a.reverse);
    load_pairs<R>(dy, a.dout, C, p, a.reverse);
    if constexpr (CH) {
        load_gates<R>(ga, a.decay, C, p, a.reverse, 1.0f);
        if (BETA) load_gates<R>(gb, a.beta, C, p, a.reverse, 0.0f);
    } else {
        ga.stage(sGa, a.decay, a, p.b, p.slab_c0, tile0, waves * R, 1.0f);
        if (BETA) gb.stage(sGb, a.beta, a, p.b, p.slab_c0, tile0, waves * R, 0.0f);
        ga.place(sGa, wave, lane, a.d);
        if (BETA) gb.place(sGb, wave, lane, a.d);
        __syncthreads();
    }
    // the saved state at or before this wave's first token
    const long long marks = (a.T + GLR_TILE - 1) / GLR_TILE, mark = p.first / GLR_TILE < marks ? p.first / GLR_TILE : marks - 1;
    float2 s = *reinterpret_cast<const float2 *>(a.saved + ((size_t)p.b * marks + mark) * C + p.c);
    auto input = [&](int r) { return BETA ? mul2(gb.get(r), v[r].get()) : v[r].get(); };
    // the wave's maps: h -> A h + H forward, and backward c -> A c + G of c = a_{t+1} G_{t+1}
    float2 A = {1.0f, 1.0f}, H = {0.0f, 0.0f}, G = {0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < R; ++r) {
        stretch(r);
        A = mul2(A, ga.get(r));
        H = fma2(ga.get(r), H, input(r));
    }
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
        stretch(r);
        const float2 d = dy[r].get();
        G = mul2(ga.get(r), make_float2(d.x + G.x, d.y + G.y));
    }
    lds2(sA[wave], lane) = A;
    lds2(sH[wave], lane) = H;
    lds2(sG[wave], lane) = G;
    __syncthreads();
    const int share = CH ? 1 : a.d;
    for (int i = FEWS ? wave * OWN + lane % OWN : threadIdx.x; i < SLAB; i += FEWS ? SLAB : blockDim.x) {
        float tA = 1.0f, tG = 0.0f, in = 0.0f;
        for (int w = waves - 1; w >= 0; --w) {
            tG = fmaf(sA[w][i], tG, sG[w][i]);
            tA *= sA[w][i];
        }
        const int ch = p.slab_c0 + i;
        const size_t st = (size_t)p.b * C + ch, wd = ((size_t)at.tile * chain.slabs + at.slab) * SLAB + i;
        if (at.tile > 0) {
            if constexpr (FEWS)
                in = state_before_by_block(chain, window, at.call, at.tile, wd - i, share, tA, tG);
            else
                in = state_before(chain, window, i, at.call, at.tile, wd, wd - i % share, i % share == 0, tA, tG);
        } else if (a.dstate_out && ch < C)
            in = a.dstate_out[st];
        const float e = fmaf(tA, in, tG);
        if (FEWS && lane >= OWN) continue;
        if (tile > 0)
            post(chain.end + wd, word(at.call, e));
        else if (a.dstate_in && ch < C)
            a.dstate_in[st] = e;
        sC[i] = in;
    }
    __syncthreads();
    for (int w = wave / (GLR_TILE / R) * (GLR_TILE / R); w < wave; ++w) s = fma2(lds2(sA[w], lane), s, lds2(sH[w], lane));
    float2 g = lds2(sC, lane);
    for (int w = waves - 1; w > wave; --w) g = fma2(lds2(sA[w], lane), g, lds2(sG[w], lane));
    anew(v);
    anew(dy);
    // the states before every fourth token; those between are formed again where they are
    // used (a product more, 3/4 of the registers less)
    float2 start[R / 4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        stretch(r);
        if (r % 4 == 0) start[r / 4] = s;
        s = fma2(ga.get(r), s, input(r));
    }
    anew(v);
    const long long dir = a.reverse ? -1 : 1;
    constexpr int N = BETA ? 16 : 8;
    float sum[N];  // per head: ddecay and dbeta of eight tokens, this lane's two channels
#pragma unroll
    for (int q = R / 4 - 1; q >= 0; --q) {
        stretch(4 * q);
        float2 before[4];
        before[0] = start[q];
#pragma unroll
        for (int i = 1; i < 4; ++i) before[i] = fma2(ga.get(4 * q + i - 1), before[i - 1], input(4 * q + i - 1));
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            const int r = 4 * q + i;
            const float2 d = dy[r].get(), x = v[r].get();
            g = make_float2(d.x + g.x, d.y + g.y);
            const float2 da = mul2(g, before[i]), db = mul2(g, x);
            if (r < p.n && p.on) {
                const size_t row = (size_t)(p.row + dir * r) * C;
                if (a.dv)
                    OutPair<IO>::store(static_cast<char *>(a.dv) + row * OutPair<IO>::BYTES, p.c, BETA ? mul2(gb.get(r), g) : g);
                if (CH && a.ddecay) Pair<IO_F32>::store(reinterpret_cast<char *>(a.ddecay + row), p.c, da);
                if (CH && BETA && a.dbeta) Pair<IO_F32>::store(reinterpret_cast<char *>(a.dbeta + row), p.c, db);
            }
            if (!CH) {
                sum[r % 8] = da.x + da.y;
                if constexpr (BETA) sum[8 + r % 8] = db.x + db.y;
            }
            g = mul2(ga.get(r), g);
        }
        if (!CH && q % 2 == 0) {
            const int L = a.d / 2, l = lane & (L - 1);
            group_sums<N>(sum, L, lane);
            auto put = [&](int i, float x) {
                const int r = 4 * q + i % 8;
                float *to = i >= 8 ? a.dbeta : a.ddecay;
                if (to && p.on && r < p.n) to[(size_t)(p.row + dir * r) * a.H + p.c / a.d] = x;
            };
            if (L == 8) {
                put(l, sum[0]);
                if constexpr (N == 16) put(8 + l, sum[1]);
            } else if (l < N) {
                put(l, sum[0]);
            }
        }
    }
}

// T = 0: the state passes through.
__global__ void glr_copy_state_kernel(float *to, const float *from, size_t n) {
    for (size_t i = blockIdx.x * (size_t)blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x)
        to[i] = from ? from[i] : 0.0f;
}

hipError_t copy_state(const GlrArgs &a, float *to, const float *from, hipStream_t s) {
    const size_t n = (size_t)a.B * a.H * a.d;
    glr_copy_state_kernel<<<dim3((unsigned)std::min<size_t>((n + 255) / 256, 4096)), dim3(256), 0, s>>>(to, from, n);
    return hipGetLastError();
}

int slabs_of(int B, int H, int d) { return B * ((H * d + SLAB - 1) / SLAB); }
size_t counter_bytes(int slabs) { return ((size_t)slabs * sizeof(u64) + 255) / 256 * 256; }

Chain chain_of(const GlrArgs &a, int tile) {
    Chain c;
    c.slabs = slabs_of(a.B, a.H, a.d);
    c.tiles = (int)((a.T + tile - 1) / tile);
    const size_t plane = (size_t)c.slabs * SLAB * c.tiles;
    c.counter = static_cast<u64 *>(a.work);
    c.end = reinterpret_cast<u64 *>(static_cast<char *>(a.work) + counter_bytes(c.slabs));
    c.mul = c.end + plane;
    c.add = c.mul + plane;
    return c;
}

// Waves of a block: a single tile of few tokens needs fewer.
int waves_of(const GlrArgs &a, int R) { return (int)std::min<long long>(WAVES, (a.T + R - 1) / R); }

// Long tiles only where calls have whole ones and they fill the device twice over (two blocks
// fit on a CU): below that they leave waves or CUs idle (2 x 4,680 tokens of 32 heads of 128,
// 2.5 long tiles a CU: 47 us forward, with long tiles 52; 16,000 tokens, 4 a CU: 80 and 76).
bool fills(const GlrArgs &a, int R) {
    return a.T >= WAVES * R && slabs_of(a.B, a.H, a.d) * ((a.T + WAVES * R - 1) / (WAVES * R)) >= 4LL * a.ncu;
}

// The look-back by all waves, up to FEW slabs.  Against the other form, bf16, beta, 128 channels a
// slab, us (forward; gradient):
//   33,000 tokens, gates per head:     2 slabs 35 : 60; 64 : 111   4: 41 : 64; 69 : 68
//                                      8: 56 : 69; 95 : 78   12: 67 : 73; 113 : 96   16: 83 : 72; 141 : 120
//   33,000 tokens, gates per channel:  2 slabs 42 : 67; 65 : 110   4: 50 : 69; 87 : 117
//                                      8: 85 : 85; 148 : 164   12: 123 : 120; 220 : 217
//   4,680 tokens, gates per head:      2 slabs 11 : 14; 15 : 21   8: 15 : 16; 24 : 28   20: 19 : 19; 31 : 32
//   1,500 tokens: the gradient of 2 to 8 slabs 5 to 11% less, else within 6%
// So it gains most at the fewest slabs and costs from 16 on; in between a threshold on slabs alone
// is not the better choice everywhere (long gradients with gates per head, which the other form
// takes in tiles twice as long, would want 4; long forward passes with them 12).
bool few_slabs(const GlrArgs &a, int R) { return slabs_of(a.B, a.H, a.d) <= FEW && a.T > WAVES * R; }

template <int IO, bool CH, bool BETA, int R, bool FEWS = false>
hipError_t forward_by(const GlrArgs &a, hipStream_t s) {
    const Chain c = chain_of(a, WAVES * R);
    glr_forward_kernel<IO, CH, BETA, R, FEWS>
        <<<dim3((unsigned)(c.slabs * c.tiles)), dim3(waves_of(a, R) * LANES), 0, s>>>(a, c);
    return hipGetLastError();
}
template <int IO, bool CH, bool BETA>
hipError_t forward(const GlrArgs &a, hipStream_t s) {
    if (a.T == 1) {
        const long long lanes = (long long)a.B * a.H * a.d / 2;  // at most 2^28 channels: B * slabs is below 2^22
        glr_step_kernel<IO, CH, BETA><<<dim3((unsigned)((lanes + 255) / 256)), dim3(256), 0, s>>>(a);
        return hipGetLastError();
    }
    if (few_slabs(a, 16)) return forward_by<IO, CH, BETA, 16, true>(a, s);
    constexpr int R = fwd_tokens(IO, CH);
    if constexpr (R > 16)
        if (fills(a, R)) return forward_by<IO, CH, BETA, R>(a, s);
    return forward_by<IO, CH, BETA, 16>(a, s);
}
template <int IO, bool CH, bool BETA, int R, bool FEWS = false>
hipError_t backward_by(const GlrArgs &a, hipStream_t s) {
    const Chain c = chain_of(a, WAVES * R);
    glr_backward_kernel<IO, CH, BETA, R, FEWS>
        <<<dim3((unsigned)(c.slabs * c.tiles)), dim3(waves_of(a, R) * LANES), 0, s>>>(a, c);
    return hipGetLastError();
}
template <int IO, bool CH, bool BETA>
hipError_t backward(const GlrArgs &a, hipStream_t s) {
    if (few_slabs(a, 8)) return backward_by<IO, CH, BETA, 8, true>(a, s);
    constexpr int R = bwd_tokens(IO, CH);
    if constexpr (R > 8)
        if (fills(a, R)) return backward_by<IO, CH, BETA, R>(a, s);
    return backward_by<IO, CH, BETA, 8>(a, s);
}

// f<IO, per-channel gates, beta>(a, s) for the call's kind.
#define GLR_DISPATCH(f)                                                                                   \
    const bool ch = a.gate_dim != 1, be = a.beta != nullptr;                                              \
    if (a.io == IO_F32)                                                                                   \
        return ch ? be ? f<IO_F32, true, true>(a, s) : f<IO_F32, true, false>(a, s)                       \
                  : be ? f<IO_F32, false, true>(a, s) : f<IO_F32, false, false>(a, s);                    \
    if (a.io == IO_BF16)                                                                                  \
        return ch ? be ? f<IO_BF16, true, true>(a, s) : f<IO_BF16, true, false>(a, s)                     \
                  : be ? f<IO_BF16, false, true>(a, s) : f<IO_BF16, false, false>(a, s);                  \
    return ch ? be ? f<IO_FP8, true, true>(a, s) : f<IO_FP8, true, false>(a, s)                           \
              : be ? f<IO_FP8, false, true>(a, s) : f<IO_FP8, false, false>(a, s);

}  // namespace

size_t glr_work_bytes(int B, int H, int d, long long max_T) {
    const size_t slabs = (size_t)slabs_of(B, H, d), tiles = (size_t)((max_T + GLR_TILE - 1) / GLR_TILE);
    return tiles < 2 ? 0 : counter_bytes((int)slabs) + 3 * slabs * SLAB * tiles * sizeof(u64);
}

hipError_t launch_glr_forward(const GlrArgs &a, hipStream_t s) {
    if (a.T == 0) return copy_state(a, a.state_out, a.state_in, s);
    GLR_DISPATCH(forward)
}

hipError_t launch_glr_backward(const GlrArgs &a, hipStream_t s) {
    if (a.T == 0) return copy_state(a, a.dstate_in, a.dstate_out, s);
    GLR_DISPATCH(backward)
}

}  // namespace gdn
