// Host-side planning of the attention calls (no device code): which kernel
// takes a call, how its keys are cut into parts, what workspace that needs and
// whether every grid can be launched, all before the first launch.  Kept apart
// from the kernels so that the host logic can be built on its own, for
// instance with the host sanitizers.
#include "attention.h"

namespace cfp32 {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int padded(int64_t D) { return D <= 64 ? 64 : 128; }

// The threads of a grid's first dimension are counted in 32 bits.
bool grid_ok(int64_t blocks, int threads) { return blocks <= 0x7FFFFFFF && blocks * threads <= 0xFFFFFFFF; }

size_t partial_bytes(int64_t rows, int slots, int dim) { return slots > 1 ? (size_t)rows * slots * (dim + 2) * 4 : 0; }

void place_partials(Partials &to, int64_t rows, void *at)
{
    if (to.slots <= 1) return;
    const int64_t n = rows * to.slots;
    to.o = (float *)at;
    to.m = to.o + n * to.dim;
    to.l = to.m + n;
}

// The join's grid (a wave or a block to a row).
bool join_ok(const Partials &to, int64_t rows) { return to.slots <= 1 || grid_ok(join_blocks(to, rows), 256); }

bool wide(const void *p, int64_t strides, int D, bool f16)
{
    const int64_t eb = f16 ? 2 : 4;
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(strides * eb)) & 15) == 0 && D % (16 / eb) == 0;
}

// Parts are made until the grid has `target` blocks (of 4 waves), of a step
// of all waves each (a little more than one makes no parts).
constexpr int64_t kDecodeBlocks = 512, kPromptBlocks = 256;
int key_parts(int64_t keys, int64_t unit, int64_t blocks, int64_t target)
{
    const int64_t most = 4 * keys <= 5 * unit ? 1 : ceil_div(keys, unit), want = target / (blocks ? blocks : 1);
    return (int)(want <= 1 || most <= 1 ? 1 : most < want ? most : want);
}
int64_t wave_step(int64_t D) { return D <= 64 ? 64 : 32; }

// Blocks of eight waves where that makes their keys one step instead of two
// (400 x 12 x 64 FP32 14.4 -> 12.5 us, 130 keys x 32/8 x 128 FP16 11.2 -> 9.3);
// with more keys than that, or fewer, four are as good or better (500 x 16/2 x
// 128 FP16 20 against 26 us).
bool eight_waves(int64_t keys, int64_t D) { return keys > 4 * wave_step(D) && keys <= 8 * wave_step(D); }

// How many parts the keys of a short prompt make: by the average sequence's.
int prompt_parts(int64_t S, int64_t Tk, int64_t blocks, int64_t D)
{
    return key_parts(ceil_div(Tk, S), 4 * wave_step(D), blocks, kPromptBlocks);
}

// Which kernel a prompt goes through, by estimates in microseconds beyond what
// both have in common: here FP32 matrix products (45 TFLOP/s of the useful
// ones, 75 with FP16 keys) and the blocks, there the way through the longest
// sequence's tiles and what comes before (for FP32 K and V a pass over them).
// Measured, 16 rows to a block against tiles: FP32 500 / 750 / 1000 x 12 x 64
// 17 / 26 / 38 against 25 / 30 / 36 us, 300 / 500 x 32/8 x 128 26 / 48 against
// 31 / 38; FP16 500 / 1500 x 12 x 64 13 / 38 against 17 / 34, 300 / 500 x 32/8 x
// 128 20 / 33 against 21 / 25, 8 x 60 and 4 x 100 of these 19 and 17 against 14
// and 14, 50 after 700 16 against 20.
bool prefer_tiles(const PromptArgs &a, int64_t units)
{
    const double keys = (double)a.Tk / a.S, seen = a.causal ? keys - 0.5 * a.Tq / a.S : keys;
    const double gflop = 4e-9 * a.D * a.Hq * a.Tq * (seen > 0 ? seen : 0), tiles = keys / 64;
    const double rows_us = gflop * (a.kv_f16 ? 1e3 / 75 : 1e3 / 45) + 0.008 * units * a.Hkv;
    const double tiles_us = a.kv_f16 ? (a.D <= 64 ? 4 + 1.1 * tiles : 4 + 2 * tiles) : (a.D <= 64 ? 6 + 1.7 * tiles : 10 + 3 * tiles);
    return rows_us > tiles_us;
}

// Of a packed batch's planes: how many keys (a tile may reach 63 beyond the last) and tiles there are, ...
Planes planes_for(int64_t S, int64_t Tk) { return {nullptr, nullptr, nullptr, Tk + kTile, Tk / kTile + S}; }
// ... their bytes, ...
int64_t plane_bytes(const Planes &p, int64_t Hkv, int64_t D)
{
    const int64_t n = Hkv * (p.count * (plane_key_bytes(padded(D)) + 8) + p.slots * 8);
    return (n + 255) & ~(int64_t)255;
}
// ... and where they are.
void place_planes(Planes &p, int64_t Hkv, int64_t D, char *at)
{
    p.keys = at;
    p.key_shifts = (int32_t *)(at + p.count * Hkv * plane_key_bytes(padded(D)));
    p.shifts = p.key_shifts + 2 * p.count * Hkv;
}

// Where blocks of 128 rows are few, their keys make parts of at least
// kPartTiles tiles for the average sequence, up to 512 blocks for long ones
// (2048 x 12 x 64 FP32, 204 blocks: 68 -> 60 us), up to 320 for shorter (1500 x
// 12 x 64, 144 blocks: 55 -> 46; with 200 to 256 blocks of 1000 keys two parts
// cost more than they gave: x 32/8 x 128 FP16 43 -> 53 us; and so did parts of
// four tiles: 4 x 300 x 12 x 64 FP16 after 100 each 16 -> 25 us).
constexpr int64_t kTileBlocks = 512, kPartTiles = 8;
int tile_parts(int64_t S, int64_t Tk, int64_t blocks)
{
    const int64_t most = (Tk / S + kPartTiles * kTile - 1) / (kPartTiles * kTile);
    const int64_t want = (Tk / S >= 24 * kTile ? kTileBlocks : 320) / blocks;
    return (int)(want <= 1 || most <= 1 ? 1 : most < want ? most : want);
}

// Whether a tile block has eight waves, by the number of blocks of 128 rows.
bool eight_tile_waves(const PromptArgs &a, int64_t blocks)
{
    // Eight waves multiply and make weights at the same time; four give more
    // and shorter blocks.  Two blocks of four to a CU and not more: four
    // (1024 x 32/8 x 128 FP16 52 -> 43 us, FP32 77 -> 66; 8192: 903 -> 955 and
    // 1321 -> 1572).  Where two of them fit a CU's LDS together, also for up
    // to four and for short sequences, whose blocks are mostly beginning and
    // end (eight against four: 2 x 4000 x 12 x 64 FP16 138 / 125, 16 x 1000 of
    // these 105 / 91, 200 x 40 92 / 49, 8 x 750 x 32/8 x 128 136 / 128, 6 x
    // 1400 218 / 229, 4 x 2000 275 / 287, FP32 4 x 4000 x 32/8 x 64 778 / 814;
    // where they do not fit, 8 x 750 x 32/8 x 128 FP32 189 / 227).
    const bool together = a.kv_f16 || a.D <= 64;
    return blocks > 512 && (!together || (blocks > 1024 && a.Tk / a.S > 1100));
}

// How many parts the shared keys of a decode make in tiles.
int decode_tile_parts(int64_t B, int64_t Hq, int64_t Hkv, int64_t keys, int page_log2)
{
    const int64_t blocks = (B * (Hq / Hkv) + 127) / 128 * Hkv, tiles = (keys + kTile - 1) / kTile;
    int64_t parts = 256 / blocks;  // one block to a CU, and room for the sequences' own keys beside it
    if (parts > (tiles + 3) / 4) parts = (tiles + 3) / 4;
    if (parts < 1) parts = 1;
    // A part's page ids (and two tiles' more, by rounding) fit the block's list.
    const int64_t room = ((int64_t)kPageIds - 2) << page_log2, per = room / kTile - 2;
    const int64_t least = (tiles + per - 1) / per;
    return (int)(parts > least ? parts : least);
}

// Which kernel takes the keys that all sequences share: estimates in
// microseconds, of this one by its groups of 16 rows, of attention_tile.hip's
// by its blocks of 128.  Measured, this against that, FP16 pages: 32 x 32/8 x
// 128 behind 320 / 1280 / 5120 / 20480 keys 22 / 33 / 50 / 117 against 29 / 30 /
// 33 / 45 us; 12 of these behind 1280 / 5120 18 / 35 against 24 / 26; 10 x 16/2
// x 128 behind 5120 / 20480 18 / 34 against 20 / 25; 16 x 14/2 x 64 behind 1280 /
// 5120 / 20480 12 / 16 / 29 against 15 / 16 / 18.
bool prefer_tiles(int64_t rows, int64_t Hkv, int64_t D, int64_t keys)
{
    const double k = 1e-3 * (double)keys * Hkv, groups = (double)ceil_div(rows, kRows), blocks = (double)ceil_div(rows, 128);
    return D <= 64 ? 0.06 * groups * k > 3 + 0.1 * blocks * k : 0.13 * groups * k > 8 + 0.13 * blocks * k;
}

// `tiles`: the pages allow the other kernel.
DecodeParts decode_parts(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t W, int lg, int64_t shared_pages, bool tiles)
{
    DecodeParts c = {};
    const int64_t g = Hq / Hkv, unit = 4 * wave_step(D);
    const int64_t n_shared = B > 1 ? shared_pages << lg : 0, n_own = (W << lg) - n_shared;
    c.shared_groups = (int)ceil_div(B * g, kRows);
    c.own_groups = (int)ceil_div(g, kRows);
    c.own_from = (int)n_shared;
    if (n_shared) {
        if (tiles && prefer_tiles(B * g, Hkv, D, n_shared)) c.tiles = decode_tile_parts(B, Hq, Hkv, n_shared, lg);
        else c.shared = key_parts(n_shared, unit, c.shared_groups * Hkv, kDecodeBlocks);
    }
    if (n_own > 0) c.own = key_parts(n_own, unit, B * c.own_groups * Hkv, kDecodeBlocks);
    // Tiles always leave their rows in slots: beside a single part, an empty one.
    if (c.shared + c.own == 0 && c.tiles <= 1) c.own = 1;
    c.eight = c.tiles == 0 && c.shared == 0 && c.own == 1 && eight_waves(n_own, D);
    c.to.slots = c.tiles + c.shared + c.own;
    c.to.dim = padded(D);
    return c;
}

}  // namespace

size_t attention_prompt_workspace(int64_t S, int64_t Tk, int64_t Hkv, int64_t D, bool kv_f16)
{
    // Whatever the rows are, blocks of kRows of them and parts make no more
    // than kPromptBlocks, and blocks of 128 and parts no more than kTileBlocks.
    const size_t rows = prompt_parts(S, Tk, 1, D) > 1 ? partial_bytes(kPromptBlocks * kRows / 2, 2, padded(D)) : 0;
    const size_t tiles = (tile_parts(S, Tk, 1) > 1 ? partial_bytes(kTileBlocks * 128 / 2, 2, padded(D)) : 0) +
                         (kv_f16 ? 0 : plane_bytes(planes_for(S, Tk), Hkv, D));
    return rows > tiles ? rows : tiles;
}

PromptPlan plan_prompt(const PromptArgs &a, void *workspace)
{
    PromptPlan p = {};
    const int g = a.Hq / a.Hkv;
    const int64_t units = (int64_t)a.Tq * g / kRows + a.S, rows = (int64_t)a.Tq * a.Hq;
    p.error = hipErrorInvalidConfiguration;
    if (units > 0x7FFFFFFF || rows > 0x7FFFFFFF) return p;
    p.wide = wide(a.k.data, a.k.tok | a.k.head, a.D, a.kv_f16) && wide(a.v.data, a.v.tok | a.v.head, a.D, a.kv_f16);
    const bool can = a.Tk > 0 && (!a.kv_f16 || (p.wide && a.k.tok < ((int64_t)1 << 25) && a.v.tok < ((int64_t)1 << 25)));
    p.tiles = can && prefer_tiles(a, units);
    p.to.dim = padded(a.D);
    if (p.tiles) {
        const int64_t blocks = ((int64_t)a.Tq * g / 128 + a.S) * a.Hkv;
        char *ws = (char *)workspace;
        if (!a.kv_f16) {
            p.planes = planes_for(a.S, a.Tk);
            if (!grid_ok(p.planes.slots, 256) || a.Hkv > 65535) return p;
            place_planes(p.planes, a.Hkv, a.D, ws);
            ws += plane_bytes(p.planes, a.Hkv, a.D);
        }
        p.eight = eight_tile_waves(a, blocks);
        p.blocks = ((int64_t)a.Tq * g / (p.eight ? 8 * kWaveRows : 4 * kWaveRows) + a.S) * a.Hkv;
        p.to.slots = tile_parts(a.S, a.Tk, blocks);
        place_partials(p.to, rows, ws);
    } else {
        p.blocks = units * a.Hkv;
        p.to.slots = prompt_parts(a.S, a.Tk, p.blocks, a.D);
        p.eight = eight_waves(ceil_div(a.Tk, (int64_t)a.S * p.to.slots), a.D);
        place_partials(p.to, rows, workspace);
    }
    if (grid_ok(p.blocks, p.eight ? 512 : 256) && join_ok(p.to, rows)) p.error = hipSuccess;
    return p;
}

size_t attention_decode_workspace(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t W, int lg, int64_t shared_pages,
                                  bool kv_f16)
{
    if (Hkv == 0) return 0;
    const size_t a = partial_bytes(B * Hq, decode_parts(B, Hq, Hkv, D, W, lg, shared_pages, false).to.slots, padded(D));
    if (!kv_f16) return a;
    const size_t b = partial_bytes(B * Hq, decode_parts(B, Hq, Hkv, D, W, lg, shared_pages, true).to.slots, padded(D));
    return a > b ? a : b;
}

DecodePlan plan_decode(const DecodeArgs &a, void *workspace)
{
    DecodePlan p = {};
    const int64_t rows = (int64_t)a.B * a.Hq;
    p.error = hipErrorInvalidConfiguration;
    if (a.Hkv > 65535 || rows > 0x7FFFFFFF) return p;
    p.wide = wide(a.k.data, a.k.page | a.k.head | a.k.tok, a.D, a.kv_f16) &&
             wide(a.v.data, a.v.page | a.v.head | a.v.tok, a.D, a.kv_f16);
    const bool tiles = a.kv_f16 && p.wide && a.k.tok < ((int64_t)1 << 31) && a.v.tok < ((int64_t)1 << 31);
    p.parts = decode_parts(a.B, a.Hq, a.Hkv, a.D, a.W, a.page_log2, a.shared_pages, tiles);
    const DecodeParts &c = p.parts;
    const int64_t own = (int64_t)a.B * c.own_groups * c.own;
    if (c.tiles) {
        p.tile_blocks = ceil_div((int64_t)a.B * (a.Hq / a.Hkv), 128) * a.Hkv * c.tiles;
        p.blocks = p.tile_blocks + own * a.Hkv;
    } else {
        p.blocks = (int64_t)c.shared * c.shared_groups + own;
    }
    place_partials(p.parts.to, rows, workspace);
    if (grid_ok(p.blocks, c.eight ? 512 : 256) && join_ok(c.to, rows)) p.error = hipSuccess;
    return p;
}

}  // namespace cfp32
