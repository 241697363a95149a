// Host-side checks of the rotary, 8-bit cache and beam calls under
// AddressSanitizer and UndefinedBehaviorSanitizer: the argument checks of
// serving_api.hip over arguments from the ends of every range, and the plans of
// attention8_plans.hip and beam_plans.hip: every part lies within the workspace
// that the query asks for, and every grid is one that can be launched.  Exit
// status 0 when every check holds.
#include <cmath>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "../../compensated_fp32_projection_amd/csrc/attention8.h"
#include "../../compensated_fp32_projection_amd/csrc/beam.h"
#include "../../include/cfp32.h"

using namespace cfp32;

static long failures = 0, checks = 0;

#define CHECK(cond, ...)                                                      \
    do {                                                                      \
        ++checks;                                                             \
        if (!(cond) && ++failures <= 20) {                                    \
            std::fprintf(stderr, "line %d: %s: ", __LINE__, #cond);           \
            std::fprintf(stderr, __VA_ARGS__);                                \
            std::fprintf(stderr, "\n");                                       \
        }                                                                     \
    } while (0)

static uint64_t state = 1;
static uint64_t next_random()
{
    state = state * 6364136223846793005ull + 1442695040888963407ull;
    return state >> 33;
}
template <class T, size_t N>
static T pick(const T (&from)[N]) { return from[next_random() % N]; }

static char *const kBase = (char *)(uintptr_t)(1ull << 40);  // never dereferenced

static void decodes()
{
    for (int64_t b : {1, 2, 3, 12, 64, 511, 512, 5000})
        for (int64_t g : {1, 2, 4, 16, 17, 80})
            for (int64_t h : {1, 2, 8, 12, 96})
                for (int64_t d : {1, 40, 64, 72, 128})
                    for (int lg : {0, 2, 4, 6, 16})
                        for (int blg : {0, 2, 4})
                            for (int64_t w : {0, 1, 3, 100, 1000, 30000}) {
                                if (blg > lg) continue;
                                Decode8Args a = {};
                                a.B = (int)b, a.Hq = (int)(g * h), a.W = (int)w;
                                a.c.P = 7, a.c.Hkv = (int)h, a.c.D = (int)d, a.c.page_log2 = lg, a.c.block_log2 = blg;
                                a.c.k = a.c.v = {kBase, (h << lg) * d, d << lg, d};
                                const size_t need = attention8_decode_workspace(b, g * h, h, d, w, lg);
                                const Decode8Plan p = plan_decode8(a, kBase);
                                const int64_t rows = b * g * h;
                                if (p.error != hipSuccess) {
                                    CHECK(rows > 1 << 20, "%ld x %ld/%ld refused", (long)b, (long)(g * h), (long)h);
                                    continue;
                                }
                                CHECK(p.parts >= 1 && p.groups == (g + 15) / 16 && p.blocks == b * p.groups * p.parts, "parts");
                                CHECK(p.blocks * 256 < (1ll << 32), "grid");
                                CHECK(p.to.dim == (d <= 64 ? 64 : 128) && p.to.slots == p.parts, "slots");
                                if (p.parts == 1) CHECK(p.to.o == nullptr && need == 0, "one part needs %zu bytes", need);
                                else {
                                    const int64_t n = rows * p.parts;
                                    CHECK((char *)p.to.o == kBase && p.to.m == p.to.o + n * p.to.dim && p.to.l == p.to.m + n &&
                                              (char *)(p.to.l + n) <= kBase + need, "%ld rows x %d parts beyond %zu bytes", (long)rows, p.parts, need);
                                }
                                CHECK(!p.fast || (lg >= 4 && blg >= 2 && d % 8 == 0), "fast");
                                CHECK(p.align == 1 || d % p.align == 0, "align");
                            }
}

static void beams()
{
    for (int64_t s : {1, 2, 32, 1000})
        for (int64_t b : {1, 4, 64})
            for (int64_t v : {1, 63, 64, 511, 512, 513, 2047, 2048, 2049, 32003, 128000, 2000000})
                for (int64_t n : {1, 8, 64}) {
                    const BeamPlan p = plan_beam(s, b, v, n);
                    CHECK(p.each == 8 || p.each == 32, "each %d", p.each);
                    CHECK((int64_t)p.chunks * 64 * p.each >= v && (int64_t)(p.chunks - 1) * 64 * p.each < v, "%d chunks", p.chunks);
                    CHECK(p.bytes == (size_t)(s * b * p.chunks) * (8 + 8 * (size_t)n), "bytes");
                    const size_t need = cfp32_beam_select_workspace_bytes(s, b, v, n);
                    CHECK(need == p.bytes + 256, "%zu bytes", need);
                }
}

// Frequencies of every scaling: within the array, positive, and none faster than one radian a position where theta >= 1.
static void frequencies()
{
    for (int64_t r : {2, 4, 6, 128, 1024})
        for (int scaling = 0; scaling < 4; ++scaling)
            for (double factor : {1.0, 1.5, 8.0, 1e6}) {
                double f[512], a;
                const cfp32_status st = cfp32_rotary_frequencies(10000.0, r, scaling, factor, 4096.0, 1.0, 32.0, f, &a);
                if (st != CFP32_OK) {
                    CHECK(scaling == CFP32_ROTARY_NTK, "refused");
                    continue;
                }
                CHECK(a >= 1.0 && std::isfinite(a), "amplitude %g", a);
                for (int64_t i = 0; i < r / 2; ++i) CHECK(f[i] > 0.0 && f[i] <= 1.0, "f[%ld] = %g", (long)i, f[i]);
            }
}

// Every argument from the ends of its range; without a device no call gets further than the checks.
static void arguments()
{
    const int64_t n[] = {-1, 0, 1, 2, 3, 16, 64, 128, 129, 1 << 16, 0x7FFFFFFF, 1ll << 31, 1ll << 40, (1ll << 48) - 1, 1ll << 48, INT64_MAX, INT64_MIN};
    const int64_t small[] = {-1, 0, 1, 2, 3, 16, 64, 128};
    void *const ptr[] = {nullptr, kBase, kBase + 1, kBase + 2, kBase + 4, kBase + 8, kBase + 4096};
    const double reals[] = {0.125, 0.0, -1.0, 1e-60, 1e39, -1e300, INFINITY, NAN, 2.0, 10000.0};
    const size_t sizes[] = {0, 1, 255, 256, 1 << 20, (size_t)1 << 40, SIZE_MAX};
    long accepted = 0;
    for (long i = 0; i < 400000; ++i) {
        auto N = [&] { return next_random() % 4 ? pick(small) : pick(n); };
        auto P = [&] { return next_random() % 8 ? (void *)kBase : pick(ptr); };
        auto f = [&] { return (float *)P(); };
        auto d = [&] { return (int32_t *)P(); };
        cfp32_cache8 c = {P(), P(), N(), N(), N(), N(), N(), N(), f(), f(), N(), N(), N(), N(), N(), N(), 16, 16, 64, (int64_t)(next_random() % 2)};
        if (next_random() % 2) {  // a good one but for a field or two
            c.k_page = c.v_page = 1 << 20, c.k_head = c.v_head = 4096, c.k_tok = c.v_tok = 64;
            c.ks_page = c.vs_page = 1 << 10, c.ks_head = c.vs_head = 16, c.P = 8, c.Hkv = 2;
        }
        if (next_random() % 8 == 0) c.page = N(), c.block = N();
        if (next_random() % 8 == 0) c.D = N(), c.code_type = N();
        const cfp32_cache8 *cache = next_random() % 64 ? &c : nullptr;
        const int kv = next_random() % 16 ? (int)(next_random() % 2) : 7;
        double out[512];
        cfp32_status st = CFP32_OK;
        switch (next_random() % 9) {
        case 0:
            st = cfp32_rotary(P(), N(), N(), P(), N(), N(), kv, (int64_t *)P(), (double *)P(), pick(reals), (int)(next_random() % 3), 1, P(),
                              N(), N(), P(), N(), N(), N(), N(), N(), N(), N(), nullptr);
            break;
        case 1: {
            const int64_t r = N();
            st = cfp32_rotary_frequencies(pick(reals), r, (int)(next_random() % 5), pick(reals), pick(reals), pick(reals), pick(reals), out,
                                          next_random() % 16 ? &out[0] : nullptr);
            break;
        }
        case 2: st = cfp32_cache8_append(f(), N(), N(), f(), N(), N(), d(), d(), (int32_t *)(kBase + 4096), cache, d(), N(), N(), N(), N(), nullptr); break;
        case 3: st = cfp32_cache8_read(cache, d(), N(), d(), d(), P(), N(), N(), P(), N(), N(), kv, N(), N(), N(), nullptr); break;
        case 4: st = cfp32_cache8_copy_pages(cache, d(), d(), N(), nullptr); break;
        case 5:
            st = cfp32_cache8_fork(cache, d(), N(), d(), d(), d(), (int32_t *)(kBase + 4096), N(), (int32_t *)(kBase + 4096), d(), d(), N(), N(),
                                   N(), P(), pick(sizes), nullptr);
            break;
        case 6: st = cfp32_cache8_compact(cache, d(), N(), d(), d(), N(), d(), d(), N(), N(), P(), pick(sizes), nullptr); break;
        case 7:
            st = cfp32_attention8_decode(f(), N(), N(), cache, d(), N(), N(), d(), f(), N(), N(), N(), N(), pick(reals), P(), pick(sizes), nullptr);
            break;
        default:
            st = next_random() % 2 ? cfp32_beam_select(f(), N(), f(), (uint8_t *)P(), N(), N(), N(), N(), N(), d(), d(), f(), (uint8_t *)P(), P(),
                                                       pick(sizes), nullptr)
                                   : cfp32_beam_reorder(P(), N(), P(), N(), d(), N(), N(), N(), nullptr);
        }
        CHECK(st == CFP32_OK || st == CFP32_ERR_INVALID_VALUE || st == CFP32_ERR_UNSUPPORTED_DEVICE, "status %d", st);
        accepted += st == CFP32_ERR_UNSUPPORTED_DEVICE;
    }
    CHECK(accepted > 1000, "%ld calls got as far as the device", accepted);
    for (long i = 0; i < 200000; ++i) {
        cfp32_attention8_decode_workspace_bytes(pick(n), pick(n), pick(n), pick(n), pick(n), pick(n));
        cfp32_beam_select_workspace_bytes(pick(n), pick(n), pick(n), pick(n));
    }
}

int main(int argc, char **argv)
{
    decodes();
    beams();
    frequencies();
    if (argc > 1 && !std::strcmp(argv[1], "no-device")) arguments();
    std::fprintf(stderr, "%ld checks, %ld failure(s)\n", checks, failures);
    return failures != 0;
}
