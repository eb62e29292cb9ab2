// gdn_matmul.hip -- matrix product of 8-bit integers with a scale per row of each operand:
//
//     out[m][n] = (sum_k a[m][k] w[n][k]) a_scale[m] w_scale[n] + bias[n]
//
// a [M, K] tokens, w [N, K] output channels, both row-major.  Sums are whole numbers (32 bits:
// K <= 65,536), so their order changes nothing; one rounding to fp32 and the scales follow.
//
// Products are formed transposed (rows of the matrix instruction = channels n, columns = tokens
// m), so a lane ends with neighbouring channels of one token and stores them as vectors.
#include "gdn_elem.h"
#include "gdn_layer.h"

#include <algorithm>

namespace gdn {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

// Four and eight neighbouring channels from n on of token m.  (Without the non-temporal hint: a row's
// lines are filled by several stores, which the L2 joins; 4,681 x 2,560 x 2,560 to fp32 took 93 us with it, 50
// without.)
template <bool F32>
__device__ __forceinline__ void store4(const MatmulArgs &a, long long m, int n, const float (&y)[4]) {
    if constexpr (F32) {
        const f32x4_t v = {y[0], y[1], y[2], y[3]};
        *reinterpret_cast<f32x4_t *>(static_cast<float *>(a.out) + m * a.out_stride + n) = v;
    } else {
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + m * a.out_stride + n) =
            make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    }
}
template <bool F32>
__device__ __forceinline__ void store8(const MatmulArgs &a, long long m, int n, const float (&y)[8]) {
    if constexpr (F32) {
        f32x4_t *p = reinterpret_cast<f32x4_t *>(static_cast<float *>(a.out) + m * a.out_stride + n);
        p[0] = f32x4_t{y[0], y[1], y[2], y[3]};
        p[1] = f32x4_t{y[4], y[5], y[6], y[7]};
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + m * a.out_stride + n) =
            make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
    }
}
// N sums of token m's scale with their channels' scales.  The scales' product is taken first; where it leaves the
// normal range (below it digits are lost, and a sum of zero times infinity is NaN) the sums are scaled in 64
// bits, whose range holds any product of the three.
template <int N>
__device__ __forceinline__ void scaled(const int (&acc)[N], float am, const float (&s)[N], float (&y)[N]) {
    bool within = true;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float p = am * s[e];
        within &= fabsf(p) >= 0x1p-126f && fabsf(p) < __builtin_inff();
        y[e] = (float)acc[e] * p;
    }
    if (within) return;
#pragma unroll 1
    for (int e = 0; e < N; ++e) y[e] = (float)((double)acc[e] * am * s[e]);
}

// ---- few tokens: bound by the weights, each read once for up to 64 ----------------------------------
//
// A block has 16 channels and up to 16 MT tokens; its waves share K and are joined in LDS.
// Operands come straight from memory: 16 rows of 64 bytes an instruction.
// Steps of 64 terms are dealt out to the waves in turn; U of them are on their way before the first
// product (16 x 12,288 x 8,192: 25 us, 4.0 TB/s, against 33 with one at a time; 8 x 7,680 x 2,560: 7 us
// of kernel either way, of which the loads are 4).
constexpr int FEW_WAVES = 8;
constexpr uint32_t NOWHERE = 0x80000000u;  // beyond a descriptor's 2 GB: reads zeros
typedef uint32_t u32x4_raw_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i32x4_t load16(const int8_t *base, uint32_t off, int k) {
    const u32x4_raw_t v = __builtin_amdgcn_raw_buffer_load_b128(
        __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(base), 0, (int)NOWHERE, 0x00027000), off, k, 0);
    i32x4_t r;
    __builtin_memcpy(&r, &v, 16);
    return r;
}
template <int MT, bool F32>
__global__ void __launch_bounds__(64 * FEW_WAVES) matmul_few_kernel(const MatmulArgs a) {
    constexpr int U = 8 / MT;
    __shared__ i32x4_t part[FEW_WAVES][MT][64];
    const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16;
    const long long m0 = (long long)blockIdx.y * (16 * MT);
    const int8_t *w = a.w + (size_t)n0 * a.K, *x = a.a + m0 * a.K;
    const uint32_t ow = n0 + l < a.N ? (uint32_t)l * (uint32_t)a.K + 16 * g : NOWHERE;
    uint32_t ox[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) ox[i] = m0 + 16 * i + l < a.M ? (uint32_t)(16 * i + l) * (uint32_t)a.K + 16 * g : NOWHERE;
    i32x4_t acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = i32x4_t{0, 0, 0, 0};
    for (int k0 = 64 * wave; k0 < a.K; k0 += 64 * FEW_WAVES * U) {
        i32x4_t wf[U], xf[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + 64 * FEW_WAVES * u;
            const bool in = k + 16 * g < a.K;
            wf[u] = load16(w, in ? ow : NOWHERE, k);
#pragma unroll
            for (int i = 0; i < MT; ++i) xf[u][i] = load16(x, in ? ox[i] : NOWHERE, k);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[u], xf[u][i], acc[i], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    // tile i is finished by wave i (MT <= FEW_WAVES)
    if (wave >= MT) return;
    i32x4_t s = part[0][wave][lane];
#pragma unroll
    for (int v = 1; v < FEW_WAVES; ++v) s += part[v][wave][lane];
    const long long m = m0 + 16 * wave + l;
    const int n = n0 + 4 * g;
    if (m < a.M && n < a.N) {
        const float4 sw = *reinterpret_cast<const float4 *>(a.w_scale + n);
        float y[4];
        scaled<4>({s[0], s[1], s[2], s[3]}, a.a_scale[m], {sw.x, sw.y, sw.z, sw.w}, y);
        if (a.bias) {
            const float4 b = *reinterpret_cast<const float4 *>(a.bias + n);
            y[0] += b.x;
            y[1] += b.y;
            y[2] += b.z;
            y[3] += b.w;
        }
        store4<F32>(a, m, n, y);
    }
}

// ---- many tokens: tiles of BM x BN, 128 terms a stage ----------------------------------
//
// Stages go from memory to LDS without passing registers, one ahead of the products.  A row of
// a stage is 128 bytes, eight pieces of 16; piece c of row r lies at place c ^ (r / 2 % 8), so
// that the 16 rows that are read at a time fall on all 64 banks (c ^ (r % 8) had half of them twice).  Rows beyond the matrix and pieces
// beyond K are read from beyond the descriptor's range, as zeros.
//
// The two stages are LDS variables of their own: the compiler waits for every load to LDS in
// flight before a read of the same variable (65,520 x 12,288 x 4,096: 4,450 us with one array,
// 3,600 so, with the next).  Tiles are dealt to the eight XCDs in runs and run through bands of eight
// rows of tiles, so that the tiles at work on an XCD at a time share operands in its L2.
constexpr int BK = 128;
constexpr int BAND = 8;
constexpr int XCDS = 8;

// 16 or 4 bytes a lane from base + off + k to LDS, in the order of the lanes.
__device__ __forceinline__ void load16_to_lds(int8_t *base, uint32_t off, int k, int8_t *to) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(__builtin_amdgcn_make_buffer_rsrc(base, 0, (int)NOWHERE, 0x00027000),
                                             (__attribute__((address_space(3))) void *)to, 16, off, k, 0, 0);
}
__device__ __forceinline__ void load4_to_lds(int8_t *base, uint32_t off, int k, int8_t *to) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(__builtin_amdgcn_make_buffer_rsrc(base, 0, (int)NOWHERE, 0x00027000),
                                             (__attribute__((address_space(3))) void *)to, 4, off, k, 0, 0);
}

template <int BM, int BN, int WM, int WN, bool F32>
__global__ void __launch_bounds__(64 * WM * WN) matmul_tile_kernel(const MatmulArgs a, int tiles_m, int tiles_n) {
    constexpr int WAVES = WM * WN;
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32;  // 32 x 32 tiles of a wave
    constexpr int NA = BM / 8 / WAVES, NW = BN / 8 / WAVES;  // loads a stage: a wave fills 1 KB (8 rows) at a time
    __shared__ __align__(16) int8_t sa0[BM * BK];
    __shared__ __align__(16) int8_t sa1[BM * BK];
    __shared__ __align__(16) int8_t sw0[BN * BK];
    __shared__ __align__(16) int8_t sw1[BN * BK];
    constexpr bool TOUCH = BM == 256;
    __shared__ __align__(16) int8_t sink[TOUCH ? 256 * WAVES : 16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;

    const int tiles = tiles_m * tiles_n, per = (tiles + XCDS - 1) / XCDS;
    const int place = blockIdx.x % XCDS * per + blockIdx.x / XCDS;
    if (place >= tiles) return;
    const int band = place / (BAND * tiles_n), in = place % (BAND * tiles_n);
    const int rows = min(BAND, tiles_m - band * BAND);
    const int tm = band * BAND + in % rows, tn = in / rows;
    const long long m0 = (long long)tm * BM;
    const int n0 = tn * BN;

    // row r = 8 (wave + WAVES i) + rr, WAVES even: (r / 2) % 8 does not depend on i
    const int rr = lane >> 3, piece = (lane & 7) ^ ((wave & 1) << 2 | rr >> 1);
    uint32_t oa[NA], ow[NW];
#pragma unroll
    for (int i = 0; i < NA; ++i) {
        const int r = 8 * (wave + WAVES * i) + rr;
        oa[i] = m0 + r < a.M ? (uint32_t)r * (uint32_t)a.K + 16 * piece : NOWHERE;
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const int r = 8 * (wave + WAVES * i) + rr;
        ow[i] = n0 + r < a.N ? (uint32_t)r * (uint32_t)a.K + 16 * piece : NOWHERE;
    }
    int8_t *const ba = const_cast<int8_t *>(a.a + m0 * a.K), *const bw = const_cast<int8_t *>(a.w + (size_t)n0 * a.K);
    const auto fill = [&](int8_t *pa, int8_t *pw, int k) {
        const bool in = k + 16 * piece < a.K;
#pragma unroll
        for (int i = 0; i < NA; ++i) load16_to_lds(ba, in ? oa[i] : NOWHERE, k, pa + 8 * (wave + WAVES * i) * BK);
#pragma unroll
        for (int i = 0; i < NW; ++i) load16_to_lds(bw, in ? ow[i] : NOWHERE, k, pw + 8 * (wave + WAVES * i) * BK);
    };

    // A stage has one load time to arrive, and some of its lines come from beyond the L2.  So each line
    // of a stage is touched AHEAD stages before by one of the blocks that share it (BAND tiles of a
    // column of tiles, about XCD CUs / BAND of a row): one load of a few lanes a wave and stage, whose
    // data goes nowhere (65,520 x 12,288 x 4,096: 3,340 us against 3,560; products alone take 2,970, at
    // a clock of 1.8 GHz.  Tiles of 128, two blocks a CU, lose by it: 1,560 x 7,680 x 2,560 50 us against 45).
    constexpr int AHEAD = 3, SA = BM / 4 / (WAVES / 2), SW = BN / BAND / (WAVES / 2);  // lines of a wave: half for a, half for w
    int8_t *const bt = wave < WAVES / 2 ? ba : bw;
    const int ta = tn % 4 * (BM / 4) + wave * SA + lane, tw = tm % BAND * (BN / BAND) + (wave - WAVES / 2) * SW + lane;
    const uint32_t ot = wave < WAVES / 2 ? (lane < SA && m0 + ta < a.M ? (uint32_t)ta * (uint32_t)a.K : NOWHERE)
                                         : (lane < SW && n0 + tw < a.N ? (uint32_t)tw * (uint32_t)a.K : NOWHERE);
    const auto touch = [&](int k) {
        if constexpr (TOUCH) {
            // it stays the youngest load, the one that the wait before a barrier leaves under way
            __builtin_amdgcn_sched_barrier(0);
            load4_to_lds(bt, k < a.K ? ot : NOWHERE, k, sink + 256 * wave);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    i32x16_t acc[TN][TM];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[j][i][e] = 0;

    // row of the instruction -> channel: a lane's 16 sums are 16 neighbouring channels
    const int l = lane & 31, hi = lane >> 5;
    const int ln = ((l >> 2) & 1) * 16 + (l >> 3) * 4 + (l & 3);
    // Fragments of 32 terms in two sets: one is read while the other is multiplied, also across the
    // barrier between two stages, whose first products are the last of the stage before.
    i32x4_t fa[2][TM], fw[2][TN];
    const auto read = [&](int set, const int8_t *pa, const int8_t *pw, int kk) {
        const int c = 2 * kk + hi;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int r = wm * (BM / WM) + 32 * i + l;
            fa[set][i] = *reinterpret_cast<const i32x4_t *>(pa + r * BK + 16 * (c ^ (r >> 1 & 7)));
        }
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int r = wn * (BN / WN) + 32 * j + ln;
            fw[set][j] = *reinterpret_cast<const i32x4_t *>(pw + r * BK + 16 * (c ^ (r >> 1 & 7)));
        }
        __builtin_amdgcn_sched_barrier(0);  // reads go out before the products that follow
    };
    const auto multiply = [&](int set) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int i = 0; i < TM; ++i) acc[j][i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[set][j], fa[set][i], acc[j][i], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    const auto stage = [&](const int8_t *pa, const int8_t *pw) {
        static_assert(BK == 128, "four steps of 32");
        read(0, pa, pw, 0);
        multiply(1);
        read(1, pa, pw, 1);
        multiply(0);
        read(0, pa, pw, 2);
        multiply(1);
        read(1, pa, pw, 3);
        multiply(0);
    };
    // Before the barrier this wave's part of the next stage is there (all of its loads but the last, which touches
    // lines), and its last reads of the other stage, whose products come behind the barrier, are over: behind it every
    // wave's copies write that stage anew, and the barrier itself waits for nothing.  To the compiler it is no
    // fence either, so one stands on both sides.  (The reads went out a step of products before: no change in time.)
    const auto arrive = [&] {
        if constexpr (TOUCH) asm volatile("s_waitcnt vmcnt(1) lgkmcnt(0)" ::: "memory");
        else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < TM; ++i) fa[1][i] = i32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < TN; ++j) fw[1][j] = i32x4_t{0, 0, 0, 0};
    // stages in pairs; a stage beyond K is read as zeros, so an odd last one needs no case of its own
    fill(sa0, sw0, 0);
    touch(BK);
    for (int k = 0; k < a.K; k += 2 * BK) {
        arrive();
        fill(sa1, sw1, k + BK);
        touch(k + AHEAD * BK);
        stage(sa0, sw0);
        arrive();
        fill(sa0, sw0, k + 2 * BK);
        touch(k + (AHEAD + 1) * BK);
        stage(sa1, sw1);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load to LDS is in flight when the block ends
    multiply(1);
    float am[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) am[i] = a.a_scale[min(m0 + wm * (BM / WM) + 32 * i + l, a.M - 1)];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {  // eight channels at a time
            const int n = n0 + wn * (BN / WN) + 32 * j + 16 * hi + 8 * q;
            if (n >= a.N) continue;
            float s[8], b[8];
            Vec<IO_F32> v;
            v.load(a.w_scale + n, 0);
            v.get(s);
            if (a.bias) {
                v.load(a.bias + n, 0);
                v.get(b);
            }
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const long long m = m0 + wm * (BM / WM) + 32 * i + l;
                if (m >= a.M) continue;
                int sum[8];
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] = acc[j][i][8 * q + e];
                scaled(sum, am[i], s, y);
                if (a.bias) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] += b[e];
                }
                store8<F32>(a, m, n, y);
            }
        }
    }
}

template <int BM, int BN, int WM, int WN, bool F32>
hipError_t tile_launch(const MatmulArgs &a, hipStream_t stream) {
    const long long tm = (a.M + BM - 1) / BM, tn = (a.N + BN - 1) / BN, blocks = (tm * tn + XCDS - 1) / XCDS * XCDS;
    hipLaunchKernelGGL((matmul_tile_kernel<BM, BN, WM, WN, F32>), dim3((unsigned)blocks), dim3(64 * WM * WN), 0, stream, a,
                       (int)tm, (int)tn);
    return hipGetLastError();
}

template <int MT, bool F32>
hipError_t few_launch(const MatmulArgs &a, hipStream_t stream) {
    hipLaunchKernelGGL((matmul_few_kernel<MT, F32>), dim3((unsigned)((a.N + 15) / 16), (unsigned)((a.M + 16 * MT - 1) / (16 * MT))),
                       dim3(64 * FEW_WAVES), 0, stream, a);
    return hipGetLastError();
}

// Few tokens, or few tokens and channels: the kernel whose operands come straight from memory reads a and w
// N K (1 + M / 16) bytes in all, the tiles take 0.6 us for 128 of K however few they are.
//   up to 16 tokens; up to 64 with N (16 + M) to 600,000 (against tiles: 32 x 12,288 x 4,096 18 us, 22; 64 x 2,560 x
//   2,560 8.0, 13; past it 64 x 12,288 x 4,096 30, 23); more with N (16 + M) to 270,000 (400 x 640 x 2,560 11 us, 13; 192 x
//   1,280 x 5,120 13, 22; past it 800 x 640 x 2,560 18, 14; 1,024 x 264 x 4,096 20, 19).
// K does not enter, as the time of both grows with it: at ten sizes next to these borders and K of 256, 1,024, 2,560, 5,120 and
// 16,384 the other side would have been quicker by up to 8%, but for 64 x 8,000 (K = 1,024: 7.6 us, tiles 9.2; 5,120: 25.3,
// 27.8), 1,024 x 264 (1,024: 7.8, 9.2) and 100 x 2,328, whose tiles take up to 1.24 times as long (5,120: 21.9, 22.4;
// 16,384: 63, 72).
bool few(long long M, long long N) { return M <= 16 || N * (16 + M) <= (M <= 64 ? 600000 : 270000); }

// Tiles of 256 x 256, one a CU, or of 128 x 128, two a CU, whichever rounds of blocks take less: a round of
// 256 takes 7/4 of one of 128 (4,681 x 12,288 x 4,096: 62 us, 36).  1,560 x 12,288 x 4,096: 93 us in three rounds of 128, 111 in
// two of 256; 4,681 x 12,288 x 8,192: 473 us in seven of 128, 452 in four of 256; 65,520 x 12,288 x 4,096: 96 rounds, 48.
bool large_tiles(const MatmulArgs &a) {
    const auto rounds = [&](long long side, long long at_once) {
        return (((a.M + side - 1) / side) * ((a.N + side - 1) / side) + at_once - 1) / at_once;
    };
    return 7 * rounds(256, a.ncu) <= 4 * rounds(128, 2 * a.ncu);
}

template <bool F32>
hipError_t launch(const MatmulArgs &a, hipStream_t stream) {
    if (few(a.M, a.N)) {
        if (a.M <= 16) return few_launch<1, F32>(a, stream);
        // 32 tokens a block while a block a CU has them all (64 x 1,280 x 5,120: 9 us against 13 with 64)
        if (a.M <= 32 || ((a.M + 31) / 32) * ((a.N + 15) / 16) <= a.ncu) return few_launch<2, F32>(a, stream);
        return few_launch<4, F32>(a, stream);
    }
    return large_tiles(a) ? tile_launch<256, 256, 2, 4, F32>(a, stream) : tile_launch<128, 128, 2, 2, F32>(a, stream);
}

}  // namespace

hipError_t launch_matmul_int8(const MatmulArgs &a, hipStream_t stream) {
    if (a.M == 0) return hipSuccess;
    return a.f32 ? launch<true>(a, stream) : launch<false>(a, stream);
}

}  // namespace gdn
