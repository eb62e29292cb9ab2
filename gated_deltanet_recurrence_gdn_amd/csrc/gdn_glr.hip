// gdn_glr.hip -- the diagonal gated linear recurrence h_t = a_t h_{t-1} + b_t v_t and its
// gradient (include/gdn.h, gdn_glr_forward / gdn_glr_backward).
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
constexpr int FWD_R = 16, BWD_R = 8;         // tokens of a wave
constexpr int LOOK = 16;                     // how far back a tile looks at once

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

// State before tile k > 0 of this lane's channel (word `at` of tile k); one whole wave.
// (A, H) is the tile's own map, published if the state is not there yet.
__device__ float state_before(const Chain &c, uint32_t call, int k, size_t at, float A, float H) {
    const size_t step = (size_t)c.slabs * SLAB;
    bool posted = false;
    for (;;) {
        const u64 last = peek(c.end + at - step);
        if (known(last, call)) return value(last);
        if (!posted) {
            post(c.mul + at, word(call, A));
            post(c.add + at, word(call, H));
            posted = true;
        }
        // the nearest known end state within LOOK tiles, four at a time
        int j = 0;
        float s = 0.0f;
        const int far = k < LOOK ? k : LOOK;
        for (int j0 = 2; j0 <= far && !j; j0 += 4) {
            u64 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = peek(c.end + at - step * (j0 + i <= far ? j0 + i : far));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (!j && known(w[i], call)) {
                    j = j0 + i <= far ? j0 + i : far;
                    s = value(w[i]);
                }
        }
        bool ready = j > 0;  // a map may be missing: its tile found its state at once, and posts that
        for (int i = j - 1; i >= 1 && ready; i -= 4) {
            u64 m[4], d[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const size_t p = at - step * (i - q >= 1 ? i - q : 1);
                m[q] = peek(c.mul + p);
                d[q] = peek(c.add + p);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (i - q >= 1 && ready) {
                    ready = known(m[q], call) && known(d[q], call);
                    s = fmaf(value(m[q]), s, value(d[q]));
                }
        }
        if (ready) return s;
        __builtin_amdgcn_s_sleep(1);
    }
}

// Two neighbouring elements, as they lie in memory.
template <int IO>
struct Pair;
template <>
struct Pair<IO_F32> {
    float2 r;
    __device__ __forceinline__ void load(const void *p, size_t i) { r = *reinterpret_cast<const float2 *>(static_cast<const float *>(p) + i); }
    __device__ __forceinline__ float2 get() const { return r; }
    static __device__ __forceinline__ void store(void *p, size_t i, float2 x) { *reinterpret_cast<float2 *>(static_cast<float *>(p) + i) = x; }
};
template <>
struct Pair<IO_BF16> {
    uint32_t r;
    __device__ __forceinline__ void load(const void *p, size_t i) { r = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p) + i); }
    __device__ __forceinline__ float2 get() const { return make_float2(bf16_lo(r), bf16_hi(r)); }
    static __device__ __forceinline__ void store(void *p, size_t i, float2 x) {
        *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p) + i) = pack_bf16x2(x.x, x.y);
    }
};
template <>
struct Pair<IO_FP8> {
    uint16_t r;
    __device__ __forceinline__ void load(const void *p, size_t i) { r = *reinterpret_cast<const uint16_t *>(static_cast<const uint8_t *>(p) + i); }
    __device__ __forceinline__ float2 get() const {
        float f[4];
        fp8x4_to_f32(r, f);
        return make_float2(f[0], f[1]);
    }
};
template <int IO>
using OutPair = Pair<IO == IO_F32 ? IO_F32 : IO_BF16>;

// A gate of two channels: one value per channel, or the head's (d is even, so a lane's
// channels are of one head).
template <bool CH>
struct Gate;
template <>
struct Gate<true> {
    float2 r;
    __device__ __forceinline__ void load(const float *p, size_t row, int C, int, int c, int) { r = *reinterpret_cast<const float2 *>(p + row * C + c); }
    __device__ __forceinline__ float2 get() const { return r; }
    __device__ __forceinline__ void set(float x) { r = make_float2(x, x); }
};
template <>
struct Gate<false> {
    float r;
    __device__ __forceinline__ void load(const float *p, size_t row, int, int H, int, int h) { r = p[row * H + h]; }
    __device__ __forceinline__ float2 get() const { return make_float2(r, r); }
    __device__ __forceinline__ void set(float x) { r = x; }
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

template <int IO, bool CH, bool BETA>
__global__ __launch_bounds__(WAVES * LANES, 4) void glr_forward_kernel(GlrArgs a, Chain chain) {
    constexpr int R = FWD_R;
    __shared__ float sA[WAVES][SLAB], sH[WAVES][SLAB], sC[SLAB];
    __shared__ Place sP;
    const int lane = threadIdx.x % LANES, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / LANES), waves = blockDim.x / LANES;
    const Place at = draw(chain, &sP);
    const int C = a.H * a.d, per = chain.slabs / a.B, b = at.slab / per;
    const int c0 = at.slab % per * SLAB + 2 * lane;
    const bool on = c0 < C;
    const int c = on ? c0 : C - 2, h = c / a.d;  // lanes past the end repeat the last channels
    const long long first = (long long)at.tile * (WAVES * R) + wave * R;
    const long long base = (long long)b * a.T;

    Gate<CH> ga[R], gb[R];
    Pair<IO> v[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const long long i = first + r < a.T ? first + r : a.T - 1;
        const size_t row = (size_t)(base + (a.reverse ? a.T - 1 - i : i));
        ga[r].load(a.decay, row, C, a.H, c, h);
        if (BETA) gb[r].load(a.beta, row, C, a.H, c, h);
        v[r].load(a.v, row * C + c);
    }
    float2 x[R], A = {1.0f, 1.0f}, H = {0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < R; ++r) {
        x[r] = BETA ? mul2(gb[r].get(), v[r].get()) : v[r].get();
        if (first + r >= a.T) {  // past the end: the map that changes nothing
            ga[r].set(1.0f);
            x[r] = {0.0f, 0.0f};
        }
        A = mul2(A, ga[r].get());
        H = fma2(ga[r].get(), H, x[r]);
    }
    lds2(sA[wave], lane) = A;
    lds2(sH[wave], lane) = H;
    __syncthreads();
    // the tile's map and start state, a channel per thread
    for (int i = threadIdx.x; i < SLAB; i += blockDim.x) {
        float tA = sA[0][i], tH = sH[0][i], s = 0.0f;
        for (int w = 1; w < waves; ++w) {
            tH = fmaf(sA[w][i], tH, sH[w][i]);
            tA *= sA[w][i];
        }
        const int ch = at.slab % per * SLAB + i;
        const size_t st = (size_t)b * C + ch, wd = ((size_t)at.tile * chain.slabs + at.slab) * SLAB + i;
        if (at.tile > 0)
            s = state_before(chain, at.call, at.tile, wd, tA, tH);
        else if (a.state_in && ch < C)
            s = a.state_in[st];
        const float e = fmaf(tA, s, tH);
        if (at.tile + 1 < chain.tiles)
            post(chain.end + wd, word(at.call, e));
        else if (a.state_out && ch < C)
            a.state_out[st] = e;
        sC[i] = s;
    }
    __syncthreads();
    float2 s = lds2(sC, lane);
    for (int w = 0; w < wave; ++w) s = fma2(lds2(sA[w], lane), s, lds2(sH[w], lane));
    if (a.saved_out && on && first % GLR_TILE == 0 && first < a.T) {
        const long long tiles = (a.T + GLR_TILE - 1) / GLR_TILE;
        *reinterpret_cast<float2 *>(a.saved_out + ((size_t)b * tiles + first / GLR_TILE) * C + c) = s;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        s = fma2(ga[r].get(), s, x[r]);
        if (first + r < a.T && on) {
            const size_t row = (size_t)(base + (a.reverse ? a.T - 1 - first - r : first + r));
            OutPair<IO>::store(a.out, row * C + c, s);
        }
    }
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

template <int IO, bool CH, bool BETA>
__global__ __launch_bounds__(WAVES * LANES, 4) void glr_backward_kernel(GlrArgs a, Chain chain) {
    constexpr int R = BWD_R;
    static_assert(WAVES * R == GLR_TILE, "a tile starts at a saved state");
    __shared__ float sA[WAVES][SLAB], sH[WAVES][SLAB], sG[WAVES][SLAB], sC[SLAB];
    __shared__ Place sP;
    const int lane = threadIdx.x % LANES, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / LANES), waves = blockDim.x / LANES;
    const Place at = draw(chain, &sP);
    const int C = a.H * a.d, per = chain.slabs / a.B, b = at.slab / per;
    const int c0 = at.slab % per * SLAB + 2 * lane;
    const bool on = c0 < C;
    const int c = on ? c0 : C - 2, h = c / a.d;
    const int tile = chain.tiles - 1 - at.tile;  // the gradient's walk: from the last tile to the first
    const long long first = (long long)tile * (WAVES * R) + wave * R;
    const long long base = (long long)b * a.T;

    Gate<CH> ga[R], gb[R];
    Pair<IO> v[R];
    OutPair<IO> dy[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const long long i = first + r < a.T ? first + r : a.T - 1;
        const size_t row = (size_t)(base + (a.reverse ? a.T - 1 - i : i));
        ga[r].load(a.decay, row, C, a.H, c, h);
        if (BETA) gb[r].load(a.beta, row, C, a.H, c, h);
        v[r].load(a.v, row * C + c);
        dy[r].load(a.dout, row * C + c);
    }
    float2 s = *reinterpret_cast<const float2 *>(a.saved + ((size_t)b * chain.tiles + tile) * C + c);
    auto input = [&](int r) { return BETA ? mul2(gb[r].get(), v[r].get()) : v[r].get(); };
    // the wave's maps: h -> A h + H forward, and backward c -> A c + G of c = a_{t+1} G_{t+1}
    float2 A = {1.0f, 1.0f}, H = {0.0f, 0.0f}, G = {0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (first + r >= a.T) ga[r].set(1.0f);
        const bool in = first + r < a.T;
        A = mul2(A, ga[r].get());
        H = fma2(ga[r].get(), H, in ? input(r) : make_float2(0.0f, 0.0f));
    }
#pragma unroll
    for (int r = R - 1; r >= 0; --r)
        if (first + r < a.T) {
            const float2 d = dy[r].get();
            G = mul2(ga[r].get(), make_float2(d.x + G.x, d.y + G.y));
        }
    lds2(sA[wave], lane) = A;
    lds2(sH[wave], lane) = H;
    lds2(sG[wave], lane) = G;
    __syncthreads();
    for (int i = threadIdx.x; i < SLAB; i += blockDim.x) {
        float tA = 1.0f, tG = 0.0f, in = 0.0f;
        for (int w = waves - 1; w >= 0; --w) {
            tG = fmaf(sA[w][i], tG, sG[w][i]);
            tA *= sA[w][i];
        }
        const int ch = at.slab % per * SLAB + i;
        const size_t st = (size_t)b * C + ch, wd = ((size_t)at.tile * chain.slabs + at.slab) * SLAB + i;
        if (at.tile > 0)
            in = state_before(chain, at.call, at.tile, wd, tA, tG);
        else if (a.dstate_out && ch < C)
            in = a.dstate_out[st];
        const float e = fmaf(tA, in, tG);
        if (tile > 0)
            post(chain.end + wd, word(at.call, e));
        else if (a.dstate_in && ch < C)
            a.dstate_in[st] = e;
        sC[i] = in;
    }
    __syncthreads();
    for (int w = 0; w < wave; ++w) s = fma2(lds2(sA[w], lane), s, lds2(sH[w], lane));
    float2 g = lds2(sC, lane);
    for (int w = waves - 1; w > wave; --w) g = fma2(lds2(sA[w], lane), g, lds2(sG[w], lane));
    float2 before[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        before[r] = s;
        s = fma2(ga[r].get(), s, input(r));
    }
    constexpr int N = BETA ? 2 * R : R;
    float sum[N];  // per head: ddecay and dbeta of each token, this lane's two channels
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
        const bool in = first + r < a.T;
        const float2 d = dy[r].get(), x = v[r].get();
        if (in) g = make_float2(d.x + g.x, d.y + g.y);
        const float2 da = mul2(g, before[r]), db = mul2(g, x);
        if (in && on) {
            const size_t row = (size_t)(base + (a.reverse ? a.T - 1 - first - r : first + r));
            if (a.dv) OutPair<IO>::store(a.dv, row * C + c, BETA ? mul2(gb[r].get(), g) : g);
            if (CH && a.ddecay) *reinterpret_cast<float2 *>(a.ddecay + row * C + c) = da;
            if (CH && BETA && a.dbeta) *reinterpret_cast<float2 *>(a.dbeta + row * C + c) = db;
        }
        if (!CH) {
            sum[r] = da.x + da.y;
            if constexpr (BETA) sum[R + r] = db.x + db.y;
        }
        if (in) g = mul2(ga[r].get(), g);
    }
    if (!CH) {
        const int L = a.d / 2, l = lane & (L - 1);
        group_sums<N>(sum, L, lane);
        auto put = [&](int i, float x) {
            const int r = i & (R - 1);
            float *to = BETA && i >= R ? a.dbeta : a.ddecay;
            if (!to || !on || first + r >= a.T) return;
            to[(size_t)(base + (a.reverse ? a.T - 1 - first - r : first + r)) * a.H + h] = x;
        };
        if (L == 8) {
            put(l, sum[0]);
            if constexpr (N == 16) put(8 + l, sum[1]);
        } else if (l < N) {
            put(l, sum[0]);
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

template <int IO, bool CH, bool BETA>
hipError_t forward(const GlrArgs &a, hipStream_t s) {
    const Chain c = chain_of(a, WAVES * FWD_R);
    glr_forward_kernel<IO, CH, BETA><<<dim3((unsigned)(c.slabs * c.tiles)), dim3(waves_of(a, FWD_R) * LANES), 0, s>>>(a, c);
    return hipGetLastError();
}
template <int IO, bool CH, bool BETA>
hipError_t backward(const GlrArgs &a, hipStream_t s) {
    const Chain c = chain_of(a, WAVES * BWD_R);
    glr_backward_kernel<IO, CH, BETA><<<dim3((unsigned)(c.slabs * c.tiles)), dim3(waves_of(a, BWD_R) * LANES), 0, s>>>(a, c);
    return hipGetLastError();
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
