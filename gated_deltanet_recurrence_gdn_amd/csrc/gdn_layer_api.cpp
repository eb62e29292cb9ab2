// gdn_layer_api.cpp -- the C ABI of the operators around the recurrence (include/gdn.h):
// rotary positions, the diagonal gated linear recurrence, group norm with an
// activation.  Validation and dispatch, as gdn_api.cpp does for the recurrence:
// everything is checked before the first launch, nothing is thrown or allocated.
#include "gdn.h"
#include "gdn_ctx.h"
#include "gdn_layer.h"

#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstring>
#include <new>

static_assert((int)GDN_F32 == (int)gdn::IO_F32 && (int)GDN_BF16 == (int)gdn::IO_BF16 &&
                  (int)GDN_FP8 == (int)gdn::IO_FP8,
              "gdn_dtype values are the kernels' IoType values");
static_assert(GDN_GLR_SAVED_TOKENS == gdn::GLR_TILE, "saved states stand a kernel tile apart");

namespace {

int bad(int code, const char *fmt, ...) {  // a call without a handle
    va_list ap;
    va_start(ap, fmt);
    set_err(g_create_err, code, fmt, ap);
    va_end(ap);
    return code;
}

bool valid_io(int io) { return io == GDN_F32 || io == GDN_BF16 || io == GDN_FP8; }

// One tensor of a call: its place, extent in bytes and alignment.  NULL tensors are
// skipped (the caller has refused those that may not be NULL).
struct Tensor {
    const char *name;
    const void *p;
    size_t bytes;
    unsigned align;
    bool out;
};

// Alignment, overlap of every output with every other tensor, device.  ok_a and ok_b
// name a pair that may be the same memory from the same address on (in place).
int check_tensors(gdn_ctx *h, const Tensor *t, int n, int ok_a = -1, int ok_b = -1) {
    for (int i = 0; i < n; ++i)
        if (reinterpret_cast<uintptr_t>(t[i].p) % t[i].align)
            return fail(h, GDN_ERR_ALIGN, "%s is not %u-byte aligned", t[i].name, t[i].align);
    for (int i = 0; i < n; ++i) {
        if (!t[i].out) continue;
        const Range a = rng(t[i].name, t[i].p, t[i].bytes);
        for (int j = 0; j < n; ++j) {
            if (j == i || (t[j].out && j < i)) continue;
            if (((i == ok_a && j == ok_b) || (i == ok_b && j == ok_a)) && t[i].p == t[j].p) continue;
            if (overlap(a, rng(t[j].name, t[j].p, t[j].bytes)))
                return fail(h, GDN_ERR_ALIAS, "%s overlaps %s%s", t[i].name, t[j].out ? "" : "input ", t[j].name);
        }
    }
    for (int i = 0; i < n; ++i)
        if (t[i].bytes)
            if (int st = check_device_ptr(h, t[i].name, t[i].p)) return st;
    return GDN_OK;
}

// The device exists and is a gfx950; its CU count.  Devices that passed are remembered
// (the answer cannot change), so that a call without a handle asks the runtime once.
constexpr int MAX_DEVICES = 64;
std::atomic<int> g_ncu[MAX_DEVICES];

int check_device(int device, int *ncu) {
    if (device < MAX_DEVICES && (*ncu = g_ncu[device].load(std::memory_order_relaxed)) > 0) return GDN_OK;
    int n = 0;
    hipError_t e = hipGetDeviceCount(&n);
    if (e != hipSuccess || n == 0) {
        (void)hipGetLastError();
        return bad(GDN_ERR_DEVICE, "no HIP device available (%s)",
                   e != hipSuccess ? hipGetErrorString(e) : "0 devices");
    }
    if (device >= n) return bad(GDN_ERR_DEVICE, "device %d does not exist (%d devices)", device, n);
    hipDeviceProp_t prop;
    e = hipGetDeviceProperties(&prop, device);
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return bad(GDN_ERR_DEVICE, "hipGetDeviceProperties: %s", hipGetErrorString(e));
    }
    if (strncmp(prop.gcnArchName, "gfx950", 6) != 0)
        return bad(GDN_ERR_DEVICE, "device %d is %s; this library is built for gfx950", device, prop.gcnArchName);
    *ncu = prop.multiProcessorCount;
    if (device < MAX_DEVICES) g_ncu[device].store(*ncu, std::memory_order_relaxed);
    return GDN_OK;
}

// A new handle of `kind` with `bytes` of device workspace, set to zero if asked for.
int make_handle(int kind, int device, size_t bytes, bool zeroed, gdn_ctx **out) {
    int ncu = 0;
    void *work = nullptr;
    if (device >= 0) {
        if (int st = check_device(device, &ncu)) return st;
        if (bytes) {
            DeviceGuard g(device);
            hipError_t e = hipMalloc(&work, bytes);
            if (e == hipSuccess && zeroed) {
                e = hipMemset(work, 0, bytes);
                if (e == hipSuccess) e = hipStreamSynchronize(nullptr);
                if (e != hipSuccess) (void)hipFree(work);
            }
            if (e != hipSuccess) {
                (void)hipGetLastError();
                return bad(GDN_ERR_OOM, "hipMalloc(%zu bytes) for the workspace: %s", bytes, hipGetErrorString(e));
            }
        }
    }
    gdn_ctx *h = new (std::nothrow) gdn_ctx;
    if (!h) {
        if (work) (void)hipFree(work);
        return bad(GDN_ERR_OOM, "out of host memory");
    }
    h->kind = kind;
    h->device = device;
    h->ncu = ncu;
    h->work = work;
    h->work_bytes = bytes;
    *out = h;
    g_create_err[0] = 0;
    return GDN_OK;
}

int refused(const char *fn, int st) {
    fprintf(stderr, "%s failed: %s\n", fn, g_create_err);
    return st;
}

// ---- rotary -------------------------------------------------------------------------

int rotary_check(gdn_ctx *h, const gdn_rotary_config &c, long long T, long long x_ts, long long x_bs,
                 long long o_ts, long long o_bs) {
    if (c.device < -1) return fail(h, GDN_ERR_ARG, "device = %d", c.device);
    if (c.B < 1 || c.H < 1) return fail(h, GDN_ERR_ARG, "B = %d and H = %d must be >= 1", c.B, c.H);
    if (c.d < 8 || c.d > 2 * gdn::ROTARY_MAX_PAIRS || c.d % 8)
        return fail(h, GDN_ERR_UNSUPPORTED, "d = %d must be a multiple of 8 from 8 to %d", c.d,
                    2 * gdn::ROTARY_MAX_PAIRS);
    if (!valid_io(c.io_dtype))
        return fail(h, GDN_ERR_UNSUPPORTED, "io_dtype = %d is not GDN_F32, GDN_BF16 or GDN_FP8", c.io_dtype);
    long long sum = 0;
    for (int s = 0; s < 3; ++s) {
        if (c.axis_dim[s] < 0 || c.axis_dim[s] % 2)
            return fail(h, GDN_ERR_ARG, "axis_dim[%d] = %d must be even and >= 0", s, c.axis_dim[s]);
        sum += c.axis_dim[s];
    }
    if (sum > c.d) return fail(h, GDN_ERR_ARG, "the axis_dim sum to %lld, above d = %d", sum, c.d);
    if (!(c.theta >= 1.0) || !std::isfinite(c.theta)) return fail(h, GDN_ERR_ARG, "theta must be >= 1 and finite");
    if (c.flags & ~(GDN_ROTARY_HALVES | GDN_ROTARY_INVERSE)) return fail(h, GDN_ERR_ARG, "unknown flags 0x%x", c.flags);
    if (T < 0) return fail(h, GDN_ERR_ARG, "T = %lld is negative", T);
    const long long row = (long long)c.H * c.d;
    const long long most = 1LL << 24;
    const long long ts[2] = {x_ts, o_ts}, bs[2] = {x_bs, o_bs};
    const size_t es[2] = {(size_t)gdn::io_in_bytes(c.io_dtype), (size_t)gdn::io_out_bytes(c.io_dtype)};
    const char *names[2] = {"x", "out"};
    for (int i = 0; i < 2; ++i) {
        if (ts[i] < row)
            return fail(h, GDN_ERR_ARG, "%s_token_stride = %lld is below H * d = %lld", names[i], ts[i], row);
        if (ts[i] > most)
            return fail(h, GDN_ERR_UNSUPPORTED, "%s_token_stride = %lld exceeds %lld", names[i], ts[i], most);
        if (bs[i] < 0) return fail(h, GDN_ERR_ARG, "%s_batch_stride = %lld is negative", names[i], bs[i]);
        const long long step = es[i] == 1 ? 8 : 16 / (long long)es[i];
        if (ts[i] % step || bs[i] % step)
            return fail(h, GDN_ERR_ALIGN, "%s strides must be multiples of %lld elements", names[i], step);
        if (((double)(c.B - 1) * bs[i] + (double)T * ts[i]) * es[i] > 9.0e18)
            return fail(h, GDN_ERR_ARG, "the extent of %s is too large", names[i]);
    }
    if (c.B > 1 && T > 0 && (double)o_bs < (double)(T - 1) * o_ts + row)
        return fail(h, GDN_ERR_ARG, "out_batch_stride = %lld lets the batch elements of out overlap", o_bs);
    if ((double)c.B * (double)T > 2.0e9)
        return fail(h, GDN_ERR_UNSUPPORTED, "B * T = %d * %lld is too large (at most 2e9 token rows a call)", c.B, T);
    return GDN_OK;
}

// ---- the diagonal recurrence --------------------------------------------------------

// Bytes of the tensors of one call.
struct GlrSizes {
    size_t v, out, gate, state, saved;
    unsigned gate_align;
};
GlrSizes glr_sizes(const gdn_glr_config &c, long long T) {
    const size_t heads = (size_t)c.B * c.H, tok = heads * (size_t)T;
    GlrSizes s;
    s.v = tok * c.d * gdn::io_in_bytes(c.io_dtype);
    s.out = tok * c.d * gdn::io_out_bytes(c.io_dtype);
    s.gate = tok * c.gate_dim * sizeof(float);
    s.state = heads * c.d * sizeof(float);
    s.saved = heads * (size_t)((T + gdn::GLR_TILE - 1) / gdn::GLR_TILE) * c.d * sizeof(float);
    s.gate_align = c.gate_dim == 1 ? 4 : 16;
    return s;
}

int glr_check_T(gdn_ctx *h, long long T) {
    if (T < 0) return fail(h, GDN_ERR_ARG, "T = %lld is negative", T);
    if (T > h->glr.max_T) return fail(h, GDN_ERR_ARG, "T = %lld exceeds max_T = %lld", T, h->glr.max_T);
    return GDN_OK;
}

gdn::GlrArgs glr_args(const gdn_ctx *h, long long T) {
    gdn::GlrArgs a{};
    a.B = h->glr.B; a.H = h->glr.H; a.d = h->glr.d; a.T = T;
    a.io = h->glr.io_dtype; a.gate_dim = h->glr.gate_dim;
    a.reverse = (h->glr.flags & GDN_FLAG_REVERSE) != 0;
    a.work = h->work; a.ncu = h->ncu;
    return a;
}

// ---- group norm ---------------------------------------------------------------------

int gn_check_sizes(gdn_ctx *h, long long N, long long S) {
    if (N < 0 || S < 0) return fail(h, GDN_ERR_ARG, "N = %lld and S = %lld must be >= 0", N, S);
    if (N > h->gn.max_N) return fail(h, GDN_ERR_ARG, "N = %lld exceeds max_N = %lld", N, h->gn.max_N);
    if (S > (1LL << 30)) return fail(h, GDN_ERR_UNSUPPORTED, "S = %lld exceeds 2^30", S);
    if ((double)N * (double)S * h->gn.C * sizeof(float) >= 4611686018427387904.0)  // 2^62
        return fail(h, GDN_ERR_ARG, "the extent of N * S * C = %lld * %lld * %d values is too large", N, S, h->gn.C);
    return GDN_OK;
}

gdn::GroupNormArgs gn_args(const gdn_ctx *h, long long N, long long S) {
    gdn::GroupNormArgs a{};
    a.N = N; a.S = S; a.max_N = h->gn.max_N; a.C = h->gn.C; a.G = h->gn.G;
    a.io = h->gn.io_dtype; a.silu = h->gn.act == GDN_ACT_SILU; a.eps = h->gn.eps;
    a.work = h->work; a.ncu = h->ncu;
    return a;
}

}  // namespace

extern "C" {

int gdn_rotary(const gdn_rotary_config *cfg, const void *x, long long x_token_stride, long long x_batch_stride,
               void *out, long long out_token_stride, long long out_batch_stride, const int *positions,
               long long positions_batch_stride, long long first_token, int height, int width, long long T,
               void *hip_stream) {
    g_create_err[0] = 0;
    if (!cfg) return bad(GDN_ERR_ARG, "gdn_rotary: cfg must be non-NULL");
    const gdn_rotary_config c = *cfg;
    gdn_ctx ctx;
    ctx.device = c.device;
    int ncu = 0;
    int st = rotary_check(&ctx, c, T, x_token_stride, x_batch_stride, out_token_stride, out_batch_stride);
    if (!st && positions && positions_batch_stride != 0 && positions_batch_stride < 3 * T)
        st = fail(&ctx, GDN_ERR_ARG, "positions_batch_stride = %lld must be 0 or at least 3 T", positions_batch_stride);
    if (!st && positions && (double)(c.B - 1) * positions_batch_stride * 4.0 > 9.0e18)
        st = fail(&ctx, GDN_ERR_ARG, "the extent of positions is too large");
    if (!st && !positions) {
        if (first_token < 0 || height < 1 || width < 1)
            st = fail(&ctx, GDN_ERR_ARG, "first_token = %lld must be >= 0, height = %d and width = %d >= 1",
                      first_token, height, width);
        else if (first_token > (1LL << 61) ||
                 (double)(first_token + T) > 2147483648.0 * (double)height * (double)width)
            st = fail(&ctx, GDN_ERR_ARG, "first_token = %lld leaves the 2^31 frames of the grid", first_token);
    }
    if (!st && T > 0) {
        if (!x || !out) {
            st = fail(&ctx, GDN_ERR_ARG, "x and out must be non-NULL when T > 0");
        } else {
            const size_t row = (size_t)c.H * c.d;
            const size_t xb = ((size_t)(c.B - 1) * x_batch_stride + (size_t)(T - 1) * x_token_stride + row) *
                              gdn::io_in_bytes(c.io_dtype);
            const size_t ob = ((size_t)(c.B - 1) * out_batch_stride + (size_t)(T - 1) * out_token_stride + row) *
                              gdn::io_out_bytes(c.io_dtype);
            const size_t pb = ((size_t)(c.B - 1) * positions_batch_stride + 3 * (size_t)T) * sizeof(int);
            const bool in_place = x == out && x_token_stride == out_token_stride &&
                                  (c.B == 1 || x_batch_stride == out_batch_stride) && c.io_dtype != GDN_FP8;
            const Tensor t[] = {{"x", x, xb, c.io_dtype == GDN_FP8 ? 8u : 16u, false}, {"out", out, ob, 16, true},
                                {"positions", positions, positions ? pb : 0, 4, false}};
            st = check_tensors(&ctx, t, 3, in_place ? 1 : -1, in_place ? 0 : -1);
        }
    }
    if (st) return bad(st, "gdn_rotary: %s", ctx.err);
    if (c.device < 0 || T == 0) return GDN_OK;
    if ((st = check_device(c.device, &ncu))) return st;

    gdn::RotaryArgs a{};
    a.x = x; a.out = out;
    a.x_ts = x_token_stride; a.x_bs = x_batch_stride; a.out_ts = out_token_stride; a.out_bs = out_batch_stride;
    a.positions = positions; a.pos_bs = positions_batch_stride;
    a.first_token = first_token; a.height = height; a.width = width;
    a.B = c.B; a.H = c.H; a.d = c.d; a.T = T; a.io = c.io_dtype;
    a.halves = (c.flags & GDN_ROTARY_HALVES) != 0;
    a.inverse = (c.flags & GDN_ROTARY_INVERSE) != 0;
    a.log2_theta = std::log2(c.theta);
    for (int s = 0; s < 3; ++s) {
        a.dim[s] = c.axis_dim[s];
        a.pairs += c.axis_dim[s] / 2;
    }
    DeviceGuard g(c.device);
    st = launch_status(&ctx, gdn::launch_rotary(a, reinterpret_cast<hipStream_t>(hip_stream)), "rotary");
    return st ? bad(st, "gdn_rotary: %s", ctx.err) : GDN_OK;
}

int gdn_glr_create(const gdn_glr_config *cfg, gdn_handle *out_h) {
    if (out_h) *out_h = nullptr;
    const char *fn = "gdn_glr_create";
    if (!cfg || !out_h) return refused(fn, bad(GDN_ERR_ARG, "cfg and out_h must be non-NULL"));
    const gdn_glr_config c = *cfg;
    int st = GDN_OK;
    if (c.device < -1) st = bad(GDN_ERR_ARG, "device = %d", c.device);
    else if (c.B < 1 || c.H < 1) st = bad(GDN_ERR_ARG, "B = %d and H = %d must be >= 1", c.B, c.H);
    else if (c.B > 32767) st = bad(GDN_ERR_UNSUPPORTED, "B = %d is too large (at most 32767)", c.B);
    else if (c.d != 16 && c.d != 32 && c.d != 64 && c.d != 128)
        st = bad(GDN_ERR_UNSUPPORTED, "d = %d must be 16, 32, 64 or 128", c.d);
    else if ((long long)c.H * c.d > (1 << 20)) st = bad(GDN_ERR_UNSUPPORTED, "H * d = %lld exceeds 2^20", (long long)c.H * c.d);
    else if (!valid_io(c.io_dtype))
        st = bad(GDN_ERR_UNSUPPORTED, "io_dtype = %d is not GDN_F32, GDN_BF16 or GDN_FP8", c.io_dtype);
    else if (c.gate_dim != 1 && c.gate_dim != c.d)
        st = bad(GDN_ERR_ARG, "gate_dim = %d must be 1 or d = %d", c.gate_dim, c.d);
    else if (c.max_T < 0) st = bad(GDN_ERR_ARG, "max_T = %lld is negative", c.max_T);
    else if (c.flags & ~GDN_FLAG_REVERSE) st = bad(GDN_ERR_ARG, "unknown flags 0x%x", c.flags);
    else if ((double)c.B * ((c.H * c.d + 127) / 128) * ((double)c.max_T / gdn::GLR_TILE + 1.0) > 4194304.0)
        // a launch has a block of up to 512 threads for each, below 2^32 threads in all
        st = bad(GDN_ERR_UNSUPPORTED, "B * ceil(H d / 128) * ceil(max_T / %d) exceeds 2^22", gdn::GLR_TILE);
    if (st) return refused(fn, st);
    gdn_ctx *h = nullptr;
    if ((st = make_handle(KIND_GLR, c.device, gdn::glr_work_bytes(c.B, c.H, c.d, c.max_T), true, &h))) return refused(fn, st);
    h->glr = c;
    *out_h = h;
    return GDN_OK;
}

int gdn_glr_forward(gdn_handle h, const void *v, const float *beta, const float *decay, const float *state_in,
                    float *state_out, float *saved, void *out, long long T, void *hip_stream) {
    if (!h) return bad(GDN_ERR_ARG, "gdn_glr_forward: NULL handle");
    h->err[0] = 0;
    int st = check_kind(h, KIND_GLR, "gdn_glr_forward");
    if (st || (st = glr_check_T(h, T))) return st;
    const GlrSizes s = glr_sizes(h->glr, T);
    if (T > 0 && (!v || !decay || !out)) return fail(h, GDN_ERR_ARG, "v, decay and out must be non-NULL when T > 0");
    const Tensor t[] = {{"v", v, s.v, 16, false},
                        {"beta", beta, s.gate, s.gate_align, false},
                        {"decay", decay, s.gate, s.gate_align, false},
                        {"state_in", state_in, s.state, 16, false},
                        {"state_out", state_out, s.state, 16, true},
                        {"saved", saved, s.saved, 16, true},
                        {"out", out, s.out, 16, true}};
    if ((st = check_tensors(h, t, 7, 4, 3))) return st;
    if (h->device < 0 || (T == 0 && !state_out)) return GDN_OK;
    gdn::GlrArgs a = glr_args(h, T);
    a.v = v; a.beta = beta; a.decay = decay; a.state_in = state_in; a.state_out = state_out;
    a.saved_out = saved; a.out = out;
    DeviceGuard g(h->device);
    return launch_status(h, gdn::launch_glr_forward(a, reinterpret_cast<hipStream_t>(hip_stream)),
                         "diagonal recurrence");
}

int gdn_glr_backward(gdn_handle h, const void *v, const float *beta, const float *decay, const float *saved,
                     const void *dout, const float *dstate_out, void *dv, float *dbeta, float *ddecay,
                     float *dstate_in, long long T, void *hip_stream) {
    if (!h) return bad(GDN_ERR_ARG, "gdn_glr_backward: NULL handle");
    h->err[0] = 0;
    int st = check_kind(h, KIND_GLR, "gdn_glr_backward");
    if (st || (st = glr_check_T(h, T))) return st;
    const GlrSizes s = glr_sizes(h->glr, T);
    if (T > 0 && (!v || !decay || !saved || !dout))
        return fail(h, GDN_ERR_ARG, "v, decay, saved and dout must be non-NULL when T > 0");
    if (dbeta && !beta) return fail(h, GDN_ERR_ARG, "dbeta must be NULL when beta is");
    const Tensor t[] = {{"v", v, s.v, 16, false},
                        {"beta", beta, s.gate, s.gate_align, false},
                        {"decay", decay, s.gate, s.gate_align, false},
                        {"saved", saved, s.saved, 16, false},
                        {"dout", dout, s.out, 16, false},
                        {"dstate_out", dstate_out, s.state, 16, false},
                        {"dv", dv, s.out, 16, true},
                        {"dbeta", dbeta, s.gate, s.gate_align, true},
                        {"ddecay", ddecay, s.gate, s.gate_align, true},
                        {"dstate_in", dstate_in, s.state, 16, true}};
    if ((st = check_tensors(h, t, 10, 9, 5))) return st;
    if (h->device < 0) return GDN_OK;
    if (T == 0 && !dstate_in) return GDN_OK;
    gdn::GlrArgs a = glr_args(h, T);
    a.v = v; a.beta = beta; a.decay = decay; a.saved = saved; a.dout = dout; a.dstate_out = dstate_out;
    a.dv = dv; a.dbeta = dbeta; a.ddecay = ddecay; a.dstate_in = dstate_in;
    DeviceGuard g(h->device);
    return launch_status(h, gdn::launch_glr_backward(a, reinterpret_cast<hipStream_t>(hip_stream)),
                         "diagonal recurrence gradient");
}

int gdn_group_norm_create(const gdn_group_norm_config *cfg, gdn_handle *out_h) {
    if (out_h) *out_h = nullptr;
    const char *fn = "gdn_group_norm_create";
    if (!cfg || !out_h) return refused(fn, bad(GDN_ERR_ARG, "cfg and out_h must be non-NULL"));
    const gdn_group_norm_config c = *cfg;
    int st = GDN_OK;
    if (c.device < -1) st = bad(GDN_ERR_ARG, "device = %d", c.device);
    else if (c.C < 8 || c.C > 8192 || c.C % 8)
        st = bad(GDN_ERR_UNSUPPORTED, "C = %d must be a multiple of 8 from 8 to 8192", c.C);
    else if (c.G < 1 || c.C % c.G) st = bad(GDN_ERR_ARG, "G = %d must divide C = %d", c.G, c.C);
    else if (!valid_io(c.io_dtype))
        st = bad(GDN_ERR_UNSUPPORTED, "io_dtype = %d is not GDN_F32, GDN_BF16 or GDN_FP8", c.io_dtype);
    else if (c.act != GDN_ACT_NONE && c.act != GDN_ACT_SILU)
        st = bad(GDN_ERR_UNSUPPORTED, "act = %d is not GDN_ACT_NONE or GDN_ACT_SILU", c.act);
    else if (!std::isnormal(c.eps) || c.eps < 0.0f) st = bad(GDN_ERR_ARG, "eps must be a positive normal number");
    else if (c.max_N < 0 || c.max_N > (1LL << 24))
        st = bad(GDN_ERR_ARG, "max_N = %lld must be from 0 to 2^24", c.max_N);
    if (st) return refused(fn, st);
    gdn_ctx *h = nullptr;
    if ((st = make_handle(KIND_GROUP_NORM, c.device, gdn::group_norm_work_bytes(c.C, c.G, c.max_N), false, &h)))
        return refused(fn, st);
    h->gn = c;
    *out_h = h;
    return GDN_OK;
}

int gdn_group_norm_forward(gdn_handle h, const void *x, const float *weight, const float *bias, void *out,
                           float *stats, long long N, long long S, void *hip_stream) {
    if (!h) return bad(GDN_ERR_ARG, "gdn_group_norm_forward: NULL handle");
    h->err[0] = 0;
    int st = check_kind(h, KIND_GROUP_NORM, "gdn_group_norm_forward");
    if (st || (st = gn_check_sizes(h, N, S))) return st;
    if (N == 0 || S == 0) return GDN_OK;
    const size_t n = (size_t)N * S * h->gn.C, cb = (size_t)h->gn.C * sizeof(float);
    if (!x || !out) return fail(h, GDN_ERR_ARG, "x and out must be non-NULL");
    const Tensor t[] = {{"x", x, n * gdn::io_in_bytes(h->gn.io_dtype), 16, false},
                        {"weight", weight, cb, 16, false},
                        {"bias", bias, cb, 16, false},
                        {"out", out, n * gdn::io_out_bytes(h->gn.io_dtype), 16, true},
                        {"stats", stats, (size_t)N * h->gn.G * 2 * sizeof(float), 16, true}};
    if ((st = check_tensors(h, t, 5))) return st;
    if (h->device < 0) return GDN_OK;
    gdn::GroupNormArgs a = gn_args(h, N, S);
    a.x = x; a.weight = weight; a.bias = bias; a.out = out; a.stats_out = stats;
    DeviceGuard g(h->device);
    return launch_status(h, gdn::launch_group_norm_forward(a, reinterpret_cast<hipStream_t>(hip_stream)),
                         "group norm");
}

int gdn_group_norm_backward(gdn_handle h, const void *x, const float *weight, const float *bias, const float *stats,
                            const void *dout, void *dx, float *dweight, float *dbias, long long N, long long S,
                            void *hip_stream) {
    if (!h) return bad(GDN_ERR_ARG, "gdn_group_norm_backward: NULL handle");
    h->err[0] = 0;
    int st = check_kind(h, KIND_GROUP_NORM, "gdn_group_norm_backward");
    if (st || (st = gn_check_sizes(h, N, S))) return st;
    const size_t n = (size_t)N * S * h->gn.C, cb = (size_t)h->gn.C * sizeof(float);
    const size_t ob = n * gdn::io_out_bytes(h->gn.io_dtype);
    if (n && (!x || !stats || !dout)) return fail(h, GDN_ERR_ARG, "x, stats and dout must be non-NULL");
    const Tensor t[] = {{"x", x, n * gdn::io_in_bytes(h->gn.io_dtype), 16, false},
                        {"weight", weight, cb, 16, false},
                        {"bias", bias, cb, 16, false},
                        {"stats", stats, n ? (size_t)N * h->gn.G * 2 * sizeof(float) : 0, 16, false},
                        {"dout", dout, ob, 16, false},
                        {"dx", dx, ob, 16, true},
                        {"dweight", dweight, cb, 16, true},
                        {"dbias", dbias, cb, 16, true}};
    if ((st = check_tensors(h, t, 8))) return st;
    if (h->device < 0) return GDN_OK;
    gdn::GroupNormArgs a = gn_args(h, N, S);
    a.x = x; a.weight = weight; a.bias = bias; a.stats = stats; a.dout = dout;
    a.dx = dx; a.dweight = dweight; a.dbias = dbias;
    DeviceGuard g(h->device);
    return launch_status(h, gdn::launch_group_norm_backward(a, reinterpret_cast<hipStream_t>(hip_stream)),
                         "group norm gradient");
}

}  // extern "C"
