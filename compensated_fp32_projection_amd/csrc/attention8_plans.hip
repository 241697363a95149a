// Host-side planning of attention over an 8-bit cache (no device code): see
// attention_plans.hip.
#include "attention8.h"

namespace cfp32 {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int padded(int64_t D) { return D <= 64 ? 64 : 128; }
bool grid_ok(int64_t blocks, int threads) { return blocks <= 0x7FFFFFFF && blocks * threads <= 0xFFFFFFFF; }

// Parts are made until the grid has kBlocks blocks, of a step of all waves each
// (a little more than one makes no parts).
constexpr int64_t kBlocks = 512;
int key_parts(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t keys)
{
    const int64_t unit = 4 * (D <= 64 ? 64 : 32), blocks = B * ceil_div(Hq / Hkv, kRows) * Hkv;
    const int64_t most = 4 * keys <= 5 * unit ? 1 : ceil_div(keys, unit), want = kBlocks / blocks;
    return (int)(want <= 1 || most <= 1 ? 1 : most < want ? most : want);
}

}  // namespace

size_t attention8_decode_workspace(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t W, int page_log2)
{
    if (B == 0 || Hkv == 0) return 0;
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
