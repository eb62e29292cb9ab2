// The C-ABI validation of the operators around the recurrence with no GPU, as
// dryrun_check.cpp does for the recurrence: dry-run calls (device = -1) on fake
// addresses, with AddressSanitizer and UndefinedBehaviorSanitizer on the host code.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "gdn.h"

namespace {

int g_fail = 0;
#define EXPECT(cond)                                                          \
    do {                                                                      \
        if (!(cond)) {                                                        \
            std::fprintf(stderr, "line %d: expected %s\n", __LINE__, #cond);  \
            ++g_fail;                                                         \
        }                                                                     \
    } while (0)

const uintptr_t BASE = 1ull << 40, GiB = 1ull << 30;
void *addr(int i, uintptr_t off = 0) { return reinterpret_cast<void *>(BASE + (uintptr_t)i * GiB + off); }
float *faddr(int i, uintptr_t off = 0) { return static_cast<float *>(addr(i, off)); }

int rot(gdn_rotary_config c, long long xts, long long xbs, long long ots, long long obs, const int *pos, long long pbs,
        long long first, int h, int w, long long T, void *out = addr(1)) {
    return gdn_rotary(&c, addr(0), xts, xbs, out, ots, obs, pos, pbs, first, h, w, T, nullptr);
}

void rotary_cases() {
    const gdn_rotary_config c = {-1, 2, 3, 64, GDN_BF16, {16, 24, 24}, 1e4, 0};
    const int *pos = static_cast<const int *>(addr(2));
    const long long big = 1ll << 62;
    EXPECT(rot(c, 192, 19200, 192, 19200, nullptr, 0, 0, 30, 52, 100) == GDN_OK);
    EXPECT(rot(c, 192, 19200, 192, 19200, pos, 300, 0, 0, 0, 100) == GDN_OK);
    EXPECT(rot(c, 192, 19200, 192, 19200, nullptr, 0, 0, 30, 52, 100, addr(0)) == GDN_OK);
    // extremes of every size: refused or accepted, without an overflow on the way
    const long long ext[] = {-big, -1, 0, 1, 8, 192, 1ll << 24, 1ll << 31, 1ll << 40, big, INT64_MAX, INT64_MIN};
    for (long long e : ext) {
        rot(c, e, 19200, 192, 19200, nullptr, 0, 0, 30, 52, 100);
        rot(c, 192, e, 192, 19200, nullptr, 0, 0, 30, 52, 100);
        rot(c, 192, 19200, 192, e, nullptr, 0, 0, 30, 52, 100);
        rot(c, 192, 19200, 192, 19200, pos, e, 0, 30, 52, 100);
        rot(c, 192, 19200, 192, 19200, nullptr, 0, e, 30, 52, 100);
        rot(c, 192, 19200, 192, 19200, nullptr, 0, e, INT32_MAX, INT32_MAX, 100);
        rot(c, 192, 19200, 192, 19200, nullptr, 0, 0, 30, 52, e);
        rot(c, 192, big / 8, 192, big / 8, pos, 0, 0, 30, 52, e);
        const int i = (int)(e & 0x7fffffff);
        rot({-1, i, 3, 64, GDN_F32, {16, 24, 24}, 1e4, 0}, 192, 19200, 192, 19200, nullptr, 0, 0, 30, 52, 100);
        rot({-1, 2, i, 512, GDN_F32, {16, 24, 24}, 1e4, 0}, 192, 19200, 192, 19200, nullptr, 0, 0, 30, 52, 100);
        rot({-1, 2, 3, i, GDN_F32, {16, 24, 24}, 1e4, 0}, 192, 19200, 192, 19200, nullptr, 0, 0, 30, 52, 100);
        rot({-1, 2, 3, 64, GDN_F32, {i, i, i}, 1e4, 0}, 192, 19200, 192, 19200, nullptr, 0, 0, 30, 52, 100);
    }
    EXPECT(gdn_rotary(nullptr, addr(0), 0, 0, addr(1), 0, 0, nullptr, 0, 0, 1, 1, 1, nullptr) == GDN_ERR_ARG);
    EXPECT(gdn_last_error(nullptr)[0] != 0);
}

void glr_cases() {
    for (int gate : {1, 64}) {
        gdn_handle h = nullptr;
        gdn_glr_config c = {-1, 2, 3, 64, GDN_BF16, gate, 1000, GDN_FLAG_REVERSE};
        EXPECT(gdn_glr_create(&c, &h) == GDN_OK && h);
        for (long long T : {0ll, 1ll, 1000ll, 1001ll, -1ll, (long long)INT64_MAX, (long long)INT64_MIN}) {
            const int want = T < 0 || T > 1000 ? GDN_ERR_ARG : GDN_OK;
            EXPECT(gdn_glr_forward(h, addr(0), faddr(1), faddr(2), faddr(3), faddr(3), faddr(4), addr(5), T, nullptr) == want);
            EXPECT(gdn_glr_backward(h, addr(0), faddr(1), faddr(2), faddr(3), addr(4), faddr(5), addr(6), faddr(7), faddr(8),
                                    faddr(5), T, nullptr) == want);
        }
        EXPECT(gdn_glr_forward(h, addr(0), faddr(1), faddr(2), faddr(3), faddr(4), nullptr, addr(0, 64), 9, nullptr) ==
               GDN_ERR_ALIAS);
        gdn_free(h);
    }
    gdn_handle h = nullptr;
    for (int i : {INT32_MIN, -1, 0, 1, 16, 32767, 1 << 20, INT32_MAX})
        for (long long T : {0ll, 1ll << 31, (long long)INT64_MAX}) {
            gdn_glr_config k[] = {{-1, i, 1, 16, GDN_F32, 1, T, 0}, {-1, 1, i, 128, GDN_F32, 1, T, 0},
                                  {-1, 32767, 8192, i, GDN_F32, i, T, 0}, {-1, 1, 1, 16, i, 1, T, 0}};
            for (const auto &c : k)
                if (gdn_glr_create(&c, &h) == GDN_OK) gdn_free(h);
                else EXPECT(h == nullptr);
        }
    EXPECT(gdn_glr_create(nullptr, &h) == GDN_ERR_ARG && !h);
    EXPECT(gdn_glr_forward(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr) == GDN_ERR_ARG);
}

void group_norm_cases() {
    gdn_handle h = nullptr;
    gdn_group_norm_config c = {-1, 64, 4, GDN_BF16, GDN_ACT_SILU, 1e-5f, 100};
    EXPECT(gdn_group_norm_create(&c, &h) == GDN_OK && h);
    const long long ext[] = {INT64_MIN, -1, 0, 1, 100, 101, 1ll << 31, 1ll << 40, 1ll << 62, INT64_MAX};
    for (long long N : ext)
        for (long long S : ext) {
            gdn_group_norm_forward(h, addr(0), faddr(1), faddr(2), addr(3), faddr(4), N, S, nullptr);
            gdn_group_norm_backward(h, addr(0), faddr(1), faddr(2), faddr(3), addr(4), addr(5), faddr(6), faddr(7), N, S,
                                    nullptr);
        }
    EXPECT(gdn_group_norm_forward(h, addr(0), nullptr, nullptr, addr(3), nullptr, 100, 5, nullptr) == GDN_OK);
    EXPECT(gdn_group_norm_forward(h, addr(0), nullptr, nullptr, addr(3), nullptr, 101, 5, nullptr) == GDN_ERR_ARG);
    gdn_free(h);
    for (int i : {INT32_MIN, -8, 0, 8, 8192, 8200, INT32_MAX}) {
        gdn_group_norm_config k[] = {{-1, i, 1, GDN_F32, 0, 1e-5f, 1}, {-1, 64, i, GDN_F32, 0, 1e-5f, 1},
                                     {-1, 64, 4, i, 0, 1e-5f, 1}, {-1, 64, 4, GDN_F32, i, 1e-5f, 1},
                                     {-1, 64, 4, GDN_F32, 0, (float)i, 1}, {-1, 64, 4, GDN_F32, 0, INFINITY, 1},
                                     {-1, 8192, 8192, GDN_F32, 0, 1e-5f, i}};
        for (const auto &cc : k)
            if (gdn_group_norm_create(&cc, &h) == GDN_OK) gdn_free(h);
            else EXPECT(h == nullptr);
    }
    EXPECT(gdn_group_norm_create(&c, nullptr) == GDN_ERR_ARG);
}

}  // namespace

int main() {
    rotary_cases();
    glr_cases();
    group_norm_cases();
    if (g_fail) {
        std::fprintf(stderr, "%d expectation(s) failed\n", g_fail);
        return 1;
    }
    std::puts("dry-run check ok");
    return 0;
}
