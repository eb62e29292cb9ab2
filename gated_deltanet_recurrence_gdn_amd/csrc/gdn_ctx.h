// gdn_ctx.h -- the handle behind the C ABI and the argument checks its entry points
// share.  Internal to the C-ABI layer.
#pragma once

#include "gdn.h"

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstddef>
#include <cstdint>
#include <cstdio>

// Messages live in fixed buffers, so no call but gdn_create allocates host memory.
constexpr size_t ERR_LEN = 512;

// What a handle was created for; a call with a handle of another kind is refused.
enum HandleKind { KIND_GDN = 0, KIND_GLR = 1, KIND_GROUP_NORM = 2 };

struct gdn_ctx {
    int kind = KIND_GDN;
    int device = -1;           // -1: dry run
    gdn_config cfg{};
    char err[ERR_LEN] = {0};
    float *scratch = nullptr;  // bidirectional form: two fp32 [B, max_T, H, d_v] partials, then
                               // two fp32 [B, H, d_v, d_k] states (the MFMA kernel's split sweep)
    size_t scratch_bytes = 0;
    uint16_t *tm = nullptr;    // per-chunk triangular inverses of the MFMA chunked kernel
    long long tm_chunks = 0;   // their capacity: directions x B x H x ceil(max_T / 64)
    // bidirectional MFMA path: a second stream (default priority) and three events, so that
    // most inverses are formed beside the first sweep launches
    hipStream_t side = nullptr;
    hipEvent_t ev_fork = nullptr, ev_join = nullptr, ev_join_mid = nullptr;
    // segment-parallel causal form (GDN_FLAG_SEGMENTS on a handle the MFMA kernel serves):
    // one allocation holding the buffers gdn::PassArgs describes, and the CU count that
    // bounds the segment count
    float *seg = nullptr;
    int ncu = 0;
    // the operators around the recurrence (KIND_GLR, KIND_GROUP_NORM)
    gdn_glr_config glr{};
    gdn_group_norm_config gn{};
    void *work = nullptr;      // their device workspace
    size_t work_bytes = 0;
};

// Last failure of a create call, or of a call that takes no handle, on this thread
// (defined in gdn_api.cpp).
extern thread_local char g_create_err[ERR_LEN];

inline int set_err(char *dst, int code, const char *fmt, va_list ap) {
    vsnprintf(dst, ERR_LEN, fmt, ap);
    return code;
}

inline int fail(gdn_ctx *h, int code, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    set_err(h->err, code, fmt, ap);
    va_end(ap);
    return code;
}

struct Range {
    const char *name;
    uintptr_t lo, hi;  // [lo, hi)
};

inline bool overlap(const Range &a, const Range &b) {
    return a.hi > a.lo && b.hi > b.lo && a.lo < b.hi && b.lo < a.hi;
}

inline Range rng(const char *name, const void *p, size_t bytes) {
    uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{name, lo, p ? lo + bytes : lo};
}

// Checks that p is device memory of `device` (not host memory, which would
// fault on the GPU).  Skipped for dry-run handles.
inline int check_device_ptr(gdn_ctx *h, const char *name, const void *p) {
    if (!p || h->device < 0) return GDN_OK;
    hipPointerAttribute_t attr;
    hipError_t e = hipPointerGetAttributes(&attr, p);
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return fail(h, GDN_ERR_ARG, "%s: not a HIP allocation (%s)", name, hipGetErrorString(e));
    }
    if (attr.type != hipMemoryTypeDevice && attr.type != hipMemoryTypeManaged)
        return fail(h, GDN_ERR_ARG, "%s: not device memory", name);
    if (attr.device != h->device)
        return fail(h, GDN_ERR_ARG, "%s: lives on device %d, handle is on device %d", name,
                    attr.device, h->device);
    return GDN_OK;
}

struct DeviceGuard {
    int prev = -1;
    bool changed = false;
    explicit DeviceGuard(int dev) {
        if (hipGetDevice(&prev) == hipSuccess && prev != dev) {
            changed = hipSetDevice(dev) == hipSuccess;
        }
    }
    ~DeviceGuard() {
        if (changed) (void)hipSetDevice(prev);
    }
};

inline int launch_status(gdn_ctx *h, hipError_t e, const char *what) {
    if (e == hipSuccess) e = hipGetLastError();
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return fail(h, GDN_ERR_LAUNCH, "%s launch failed: %s", what, hipGetErrorString(e));
    }
    return GDN_OK;
}

inline int check_kind(gdn_ctx *h, int kind, const char *fn) {
    if (h->kind == kind) return GDN_OK;
    return fail(h, GDN_ERR_ARG, "%s: the handle was created for another operator", fn);
}
