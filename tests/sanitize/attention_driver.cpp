// Host-side checks of the attention and cache calls under AddressSanitizer and
// UndefinedBehaviorSanitizer: the argument checks of attention_api.hip over
// arguments from the ends of every range, and the plans of
// attention_plans.hip and cache_plans.hip: every part, slot and plane lies
// within the workspace that the query asks for, without knowing the rows, every
// grid is one that can be launched, and pages are moved whole.  Exit status 0 when every check holds.
#include <cmath>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "../../compensated_fp32_projection_amd/csrc/attention.h"
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

// A grid of the runtime's: blocks of each dimension, and threads of the first, in range.
static bool grid(int64_t x, int64_t y, int threads) { return x >= 1 && x <= 0x7FFFFFFF && x * threads < (1ll << 32) && y >= 1 && y <= 65536; }

static bool inside(const Partials &to, int64_t rows, const char *from, size_t bytes)
{
    if (to.slots <= 1) return to.o == nullptr;
    const int64_t n = rows * to.slots;
    const char *end = from + bytes;
    return (char *)to.o >= from && to.m == to.o + n * to.dim && to.l == to.m + n && (char *)(to.l + n) <= end &&
           (uintptr_t)to.o % 16 == 0;
}

static void prompts()
{
    const int64_t S[] = {1, 2, 3, 7, 8, 70, 200, 512, 8192, 1 << 20}, T[] = {1, 15, 64, 65, 500, 1000, 1500, 6001, 8192, 100000, 1 << 20};
    const int64_t G[] = {1, 2, 4, 7, 32}, H[] = {1, 2, 8, 12, 96}, D[] = {1, 40, 64, 72, 128};
    for (int64_t s : S)
        for (int64_t tk : T)
            for (int64_t h : H)
                for (int64_t d : D)
                    for (int f16 = 0; f16 < 2; ++f16) {
                        const size_t need = cfp32_attention_prompt_workspace_bytes(s, tk, h, d, f16);
                        for (int64_t tq : T)
                            for (int64_t g : G) {
                                PromptArgs a = {};
                                a.S = (int)s, a.Tq = (int)tq, a.Tk = (int)tk, a.Hq = (int)(g * h), a.Hkv = (int)h, a.D = (int)d;
                                a.kv_f16 = f16, a.causal = tq % 2;
                                a.k.data = a.v.data = kBase, a.k.tok = a.v.tok = h * d, a.k.head = a.v.head = d;
                                const PromptPlan p = plan_prompt(a, kBase);
#define WHAT "S %ld Tq %ld Tk %ld heads %ld/%ld x %ld f16 %d", (long)s, (long)tq, (long)tk, (long)(g * h), (long)h, (long)d, f16
                                const int64_t rows = tq * g * h;
                                if (p.error != hipSuccess) {
                                    CHECK(s * h * 512 > (1ll << 31) || rows >= (1ll << 27), WHAT);
                                    continue;
                                }
                                // The API's pointer is rounded up within 256 bytes of it.
                                const size_t have = need > 256 ? need - 256 : 0;
                                CHECK(grid(p.blocks, p.to.slots, p.eight ? 512 : 256), WHAT);
                                CHECK(p.to.slots <= 1 || grid(join_blocks(p.to, rows), 1, 256), WHAT);
                                const int per = p.tiles ? (p.eight ? 256 : 128) : kRows;
                                CHECK(p.blocks >= ((tq * g + per - 1) / per) * h, WHAT);
                                if (p.tiles && !f16) {
                                    const Planes &m = p.planes;
                                    const int dp = d <= 64 ? 64 : 128;
                                    CHECK(grid(m.slots, h, 256) && m.count >= tk + 63 && m.slots >= tk / 64 + s, WHAT);
                                    CHECK(m.keys == kBase && (char *)m.key_shifts == m.keys + m.count * h * plane_key_bytes(dp), WHAT);
                                    CHECK(m.shifts == m.key_shifts + 2 * m.count * h, WHAT);
                                    const char *end = (char *)(m.shifts + 2 * m.slots * h);
                                    CHECK(end <= kBase + have && (p.to.slots <= 1 || (char *)p.to.o >= end), WHAT);
                                }
                                CHECK(inside(p.to, rows, kBase, have), WHAT);
#undef WHAT
                            }
                    }
}

static void decodes()
{
    const int64_t B[] = {1, 2, 12, 32, 40, 1000}, G[] = {1, 4, 7, 64}, H[] = {1, 2, 8, 12}, D[] = {1, 64, 80, 128};
    for (int64_t b : B)
        for (int64_t g : G)
            for (int64_t h : H)
                for (int64_t d : D)
                    for (int lg : {0, 3, 4, 6, 8, 16})
                        for (int64_t keys : {1l, 17l, 130l, 2000l, 65536l, 3000000l})
                            for (int share = 0; share < 4; ++share)
                                for (int f16 = 0; f16 < 2; ++f16) {
                                    const int64_t W = (keys + (1l << lg) - 1) >> lg, shared = share == 0 ? 0 : share == 1 ? W / 2 : share == 2 ? W - W / 5 : W;
                                    const size_t need = cfp32_attention_decode_workspace_bytes(b, g * h, h, d, W, 1l << lg, shared, f16);
                                    DecodeArgs a = {};
                                    a.B = (int)b, a.Hq = (int)(g * h), a.Hkv = (int)h, a.D = (int)d, a.P = 5, a.page_log2 = lg;
                                    a.W = (int)W, a.shared_pages = (int)shared, a.kv_f16 = f16;
                                    a.k.data = a.v.data = kBase, a.k.tok = a.v.tok = d, a.k.head = a.v.head = d << lg;
                                    a.k.page = a.v.page = h * d << lg;
                                    const DecodePlan p = plan_decode(a, kBase);
#define WHAT "B %ld heads %ld/%ld x %ld page 2^%d W %ld shared %ld f16 %d", (long)b, (long)(g * h), (long)h, (long)d, lg, (long)W, (long)shared, f16
                                    CHECK(p.error == hipSuccess, WHAT);
                                    const DecodeParts &c = p.parts;
                                    const int64_t rows = b * g * h;
                                    CHECK(inside(c.to, rows, kBase, need > 256 ? need - 256 : 0), WHAT);
                                    CHECK(c.to.slots == c.tiles + c.shared + c.own && c.to.slots >= 1, WHAT);
                                    CHECK(!c.tiles || c.to.slots > 1, WHAT);
                                    CHECK(c.shared_groups * (int64_t)kRows >= b * g && c.own_groups * (int64_t)kRows >= g, WHAT);
                                    CHECK(grid(p.blocks, c.tiles ? 1 : h, c.eight ? 512 : 256), WHAT);
                                    CHECK(c.to.slots <= 1 || grid(join_blocks(c.to, rows), 1, 256), WHAT);
                                    CHECK(c.own_from == (b > 1 ? shared << lg : 0), WHAT);
                                    if (c.tiles) {
                                        // As the kernel cuts them: parts of an even number of tiles, whose pages its list holds.
                                        const int n = (int)(((shared << lg) + kTile - 1) / kTile), per = ((n + c.tiles - 1) / c.tiles + 1) & ~1;
                                        CHECK((int64_t)per * c.tiles >= n, WHAT);
                                        for (int part = 0; part < c.tiles; ++part) {
                                            const int64_t t0 = (int64_t)part * per < n ? part * per : n, t1 = t0 + per < n ? t0 + per : n;
                                            if (t0 >= t1) continue;
                                            const int64_t last = (t1 * kTile < (shared << lg) ? t1 * kTile : shared << lg) - 1;
                                            CHECK((last >> lg) - (t0 * kTile >> lg) < kPageIds, WHAT);
                                        }
                                    }
#undef WHAT
                                }
}

// Every value of a page is moved once, in vectors that its addresses allow.
static void pages()
{
    for (int64_t d : {1l, 2l, 3l, 8l, 40l, 64l, 128l})
        for (int64_t h : {1l, 2l, 5l, 8l, 65536l, 0x7FFFFFFFl})
            for (int lg : {0, 1, 4, 6, 16})
                for (int eb : {2, 4})
                    for (int layout = 0; layout < 4; ++layout) {
                        const int64_t page = 1l << lg, pad = layout == 3 ? d + 3 : d;
                        if (h * page > ((1l << 47) / pad)) continue;
                        Pool p = {};
                        p.P = 3, p.page_log2 = lg, p.Hkv = (int)h, p.D = (int)d, p.elem_bytes = eb;
                        const PagesView by_head = {kBase, h * page * pad, page * pad, pad}, by_tok = {kBase + eb, h * page * pad, pad, h * pad};
                        p.k = layout == 1 ? by_tok : by_head, p.v = layout == 0 ? by_head : by_tok;
                        const PageShape g = page_shape(p);
                        CHECK(g.rows >= 1 && g.vecs >= 1 && g.n2 >= 1, "%ld x 2^%d x %ld", (long)h, lg, (long)d);
                        CHECK((__int128)g.rows * g.vecs * g.vec_bytes == (__int128)h * page * d * eb, "%ld x 2^%d x %ld layout %d", (long)h, lg,
                              (long)d, layout);
                        CHECK(g.vec_bytes >= eb && g.vec_bytes <= 16 && (uintptr_t)p.k.data % g.vec_bytes == 0 &&
                                  (uintptr_t)p.v.data % g.vec_bytes == 0, "vectors of %d", g.vec_bytes);
                        if (g.rows > 1) CHECK(g.n2 == page && g.rows == h * page, "rows");
                    }
}

// Every argument from the ends of its range; without a device no call gets further than the checks.
static void arguments()
{
    const int64_t n[] = {-1, 0, 1, 2, 3, 16, 64, 128, 129, 1 << 16, 0x7FFFFFFF, 1ll << 31, 1ll << 40, (1ll << 48) - 1, 1ll << 48, INT64_MAX, INT64_MIN};
    const int64_t small[] = {-1, 0, 1, 2, 3, 16, 64, 128};
    void *const ptr[] = {nullptr, kBase, kBase + 1, kBase + 2, kBase + 4, kBase + 8, kBase + 4096};
    const double scales[] = {0.125, 0.0, -1.0, 1e-60, 1e39, -1e300, INFINITY, NAN};
    const size_t sizes[] = {0, 1, 255, 256, 1 << 20, (size_t)1 << 40, SIZE_MAX};
    long accepted = 0;
    for (long i = 0; i < 400000; ++i) {
        auto N = [&] { return next_random() % 4 ? pick(small) : pick(n); };
        auto P = [&] { return next_random() % 8 ? (void *)kBase : pick(ptr); };
        auto f = [&] { return (float *)P(); };
        auto d = [&] { return (int32_t *)P(); };
        const int kv = (int)(next_random() % 4) - 1 == 2 ? 7 : (int)(next_random() % 2);
        const int64_t page = next_random() % 4 ? 16 : N();
        cfp32_status st = CFP32_OK;
        switch (next_random() % 8) {
        case 0:
            st = cfp32_attention_prompt(f(), N(), N(), P(), N(), N(), P(), N(), N(), kv, d(), d(), f(), N(), N(), N(), N(), N(), N(), N(),
                                        N(), 1, pick(scales), P(), pick(sizes), nullptr);
            break;
        case 1:
            st = cfp32_attention_decode(f(), N(), N(), P(), N(), N(), N(), P(), N(), N(), N(), kv, N(), page, d(), N(), N(), d(), N(), f(),
                                        N(), N(), N(), N(), N(), N(), pick(scales), P(), pick(sizes), nullptr);
            break;
        case 2: st = cfp32_cache_reserve(d(), N(), d(), d(), d(), d(), N(), d(), d(), N(), N(), N(), page, nullptr); break;
        case 3:
            st = cfp32_cache_append(f(), N(), N(), f(), N(), N(), d(), d(), (int32_t *)(kBase + 4096), P(), N(), N(), N(), P(), N(), N(), N(),
                                    kv, N(), page, d(), N(), N(), N(), N(), N(), N(), nullptr);
            break;
        case 4:
            st = cfp32_cache_copy_pages(P(), N(), N(), N(), P(), N(), N(), N(), kv, N(), page, N(), N(), d(), d(), N(), nullptr);
            break;
        case 5:
            st = cfp32_cache_fork(P(), N(), N(), N(), P(), N(), N(), N(), kv, N(), page, N(), N(), d(), N(), d(), d(), d(),
                                  (int32_t *)(kBase + 4096), N(), (int32_t *)(kBase + 4096), d(), d(), N(), N(), N(), P(), pick(sizes), nullptr);
            break;
        case 6: st = cfp32_cache_free(d(), N(), d(), d(), N(), N(), N(), nullptr); break;
        default:
            st = cfp32_cache_compact(P(), N(), N(), N(), P(), N(), N(), N(), kv, N(), page, N(), N(), d(), N(), d(), d(), N(), d(), d(), N(),
                                     N(), P(), pick(sizes), nullptr);
        }
        CHECK(st == CFP32_OK || st == CFP32_ERR_INVALID_VALUE || st == CFP32_ERR_UNSUPPORTED_DEVICE, "status %d", st);
        accepted += st == CFP32_ERR_UNSUPPORTED_DEVICE;
    }
    CHECK(accepted > 1000, "%ld calls got as far as the device", accepted);
    for (long i = 0; i < 200000; ++i) {
        cfp32_attention_prompt_workspace_bytes(pick(n), pick(n), pick(n), pick(n), (int)(next_random() % 3));
        cfp32_attention_decode_workspace_bytes(pick(n), pick(n), pick(n), pick(n), pick(n), pick(n), pick(n), (int)(next_random() % 3));
        cfp32_cache_fork_workspace_bytes(pick(n));
        cfp32_cache_compact_workspace_bytes(pick(n));
    }
}

int main(int argc, char **argv)
{
    prompts();
    decodes();
    pages();
    if (argc > 1 && !std::strcmp(argv[1], "no-device")) arguments();
    std::fprintf(stderr, "%ld checks, %ld failure(s)\n", checks, failures);
    return failures != 0;
}
