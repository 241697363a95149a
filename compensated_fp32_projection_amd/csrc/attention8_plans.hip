// Host-side planning of attention over an 8-bit cache (no device code): see
// attention_plans.hip.
#include "attention8.h"

namespace cfp32 {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int padded(int64_t D) { return D <= 64 ? 64 : 128; }
bool grid_ok(int64_t blocks, int threads) { return blocks <= 0x7FFFFFFF && blocks * threads <= 0xFFFFFFFF; }

// Parts are made until the grid has kBlocks blocks, each of a step of all waves
// (128 or 256 keys) or more: two to a compute unit, which is what its registers
// hold (with 256 / 512 / 1024 blocks at the most 16 x 4000 x 32/8 x 128 INT8 takes
// 35 / 32 / 37 us, 12 x 2000 x 12 x 64 E4M3 22 / 17 / 18, 2 x 65536 x 32/8 x 128 50 /
// 44 / 50).  Of up to three steps none are made, since joining them is a launch of
// its own: in one part and in several 300 keys x 16 x 32/8 x 128 take 10.0 / 11.7 us,
// 500 x 12 x 12 x 64 8.4 / 11.0; of four 500 x 4 x 32/8 x 128 11.4 / 10.2.  Blocks of
// eight waves were no faster (1 x 500 11.3 us against 9.6).
constexpr int64_t kBlocks = 512, kOneBlock = 3;
int key_parts(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t keys)
{
    const int64_t unit = 4 * (D <= 64 ? 64 : 32), steps = ceil_div(keys, unit);
    const int64_t want = kBlocks / (B * ceil_div(Hq / Hkv, kRows) * Hkv);
    return (int)(want <= 1 || steps <= kOneBlock ? 1 : steps < want ? steps : want);
}

}  // namespace

size_t attention8_decode_workspace(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t W, int page_log2)
{
    if (B == 0 || Hq == 0 || Hkv == 0) return 0;
    const int parts = key_parts(B, Hq, Hkv, D, W << page_log2);
    return parts > 1 ? (size_t)(B * Hq * parts) * (padded(D) + 2) * 4 : 0;
}

Decode8Plan plan_decode8(const Decode8Args &a, void *workspace)
{
    Decode8Plan p = {};
    const Cache8 &c = a.c;
    const int64_t rows = (int64_t)a.B * a.Hq;
    p.error = hipErrorInvalidConfiguration;
    if (c.Hkv > 65535 || rows > 0x7FFFFFFF) return p;
    const int64_t m = 16 | c.D | (int64_t)((uintptr_t)c.k.data | (uintptr_t)c.v.data) | c.k.page | c.k.head | c.k.tok | c.v.page |
                      c.v.head | c.v.tok;
    p.align = m % 16 == 0 ? 16 : m % 8 == 0 ? 8 : 1;
    p.fast = p.align >= 8 && c.page_log2 >= 4 && c.block_log2 >= 2 && c.k.tok < (int64_t)1 << 26 && c.v.tok < (int64_t)1 << 26;
    p.groups = (int)ceil_div(a.Hq / c.Hkv, kRows);
    p.parts = key_parts(a.B, a.Hq, c.Hkv, c.D, (int64_t)a.W << c.page_log2);
    p.blocks = (int64_t)a.B * p.groups * p.parts;
    p.to.slots = p.parts;
    p.to.dim = padded(c.D);
    if (p.parts > 1) {
        const int64_t n = rows * p.parts;
        p.to.o = (float *)workspace;
        p.to.m = p.to.o + n * p.to.dim;
        p.to.l = p.to.m + n;
    }
    if (grid_ok(p.blocks, 256) && (p.parts <= 1 || grid_ok(join_blocks(p.to, rows), 256))) p.error = hipSuccess;
    return p;
}

}  // namespace cfp32
