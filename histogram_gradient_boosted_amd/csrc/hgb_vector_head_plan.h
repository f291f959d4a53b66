// Launch plans of the head's losses (cross entropy and distillation over a
// vocabulary) and of the gate: sizes in, tiles, splits and workspace layouts
// out.  Plain C++, compiled and tested on the host alone.
#pragma once

#include "hgb_vector_plan.h"

namespace hgb {

constexpr int64_t kHeadMaxRows = 1 << 24;
constexpr int64_t kHeadMaxVocab = 1 << 24;
constexpr int64_t kHeadMaxDim = 32768;
constexpr int64_t kHeadMaxStride = 1 << 20;   // of rows that are read in place: a tile's 256 rows lie within 2^30 bytes
constexpr int kDistillMaxTop = 256;
constexpr int kHeadCus = 256;                 // splits are made for this many CUs

constexpr int kTileRows = 256;    // of the largest tile
constexpr int kTileCols = 256;
constexpr int kTileFew = 32;      // of the tile for no more rows than that
constexpr int kStepBytes = 128;   // of a row that one step of a product's sum takes

constexpr int kRateBlocks = 256;
constexpr int kRateWords = 2 + kRateBlocks;   // behind the rates: their unit, one over it, the blocks' largest

// Of the logits' gradient that is held at a time, for up to two planes (a third
// takes half as much again: in pieces of as many bytes 4,096 x 262,144 x 512
// took 8.2 ms for 6.7); at least a tile's tokens of every row.
constexpr int64_t kPieceBytes = (int64_t)1 << 30;
// Planes of the logits' gradient beside a 32-bit dtable of 16-bit inputs, each
// what the ones before it left: together they hold 24 bits.  Two of bf16 would
// hold 17, and dtable's error would be 1.75 times that of one from 32-bit
// values (2.6e-6 and 1.5e-6 for 4,096 x 262,144 x 512).
constexpr int kPlanesBf16 = 3, kPlanesF16 = 2;
constexpr int64_t kStatBytes = (int64_t)1 << 29;    // of the forward pass's partial sums

// The tiles of a product: rows x columns of a block of four waves, side by side
// in `wn` columns; how many such blocks a CU holds, by its LDS and by its
// registers (the kernels are built for that many); and how much of the largest
// tile's rate their products reach, in 16 and in 32 bits (the products of
// 32-bit values take eight times as long, and hide the rest).
struct Tile {
    int bm, bn, wn, per_cu;
    float rate16, rate32;
};
constexpr Tile kTiles[] = {{256, 256, 2, 1, 1.0f, 1.0f}, {128, 128, 2, 2, 0.75f, 0.95f}, {256, 64, 1, 1, 0.5f, 0.9f}, {32, 256, 4, 1, 0.3f, 0.5f}};
enum { kTileLarge, kTileMiddle, kTileNarrow, kTileLow };
constexpr int tile_blocks(int bm, int bn)
{
    for (const Tile& t : kTiles)
        if (t.bm == bm && t.bn == bn) return t.per_cu;
    return 0;
}

// A product's launch: C [m][n], summed over k in steps, in `splits` shares of
// the steps.
struct ProductPlan {
    int tile = kTileLarge;
    int bm = kTileRows, bn = kTileCols;
    int64_t tiles_m = 1, tiles_n = 1;
    int splits = 1;
    int64_t blocks() const { return tiles_m * tiles_n * splits; }
};

// The tile whose blocks, in whole rounds of the CUs, take the least time for
// their steps and as much as `ends` steps for their first loads and last
// stores.  `split`: a sum may be shared by as many blocks as fill the CUs once,
// of four steps at least.  The narrow tile is not for the logits, and rows that
// fit the low one take it.
inline ProductPlan plan_product(int64_t m, int64_t n, int64_t steps, int size, bool logits, bool split)
{
    ProductPlan best;
    double least = 0;
    const double ends = size == 4 ? 0.5 : 3;
    for (int t = 0; t < 4; ++t) {
        const Tile& tile = kTiles[t];
        if ((t == kTileNarrow && logits) || (t == kTileLow) != (m <= kTileFew)) continue;
        ProductPlan p;
        p.tile = t;
        p.bm = tile.bm;
        p.bn = tile.bn;
        p.tiles_m = vec_ceil(m, p.bm);
        p.tiles_n = vec_ceil(n, p.bn);
        const int64_t room = (int64_t)kHeadCus * tile.per_cu;
        if (split) p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(room / (p.tiles_m * p.tiles_n), steps / 4));
        const double rounds = (double)vec_ceil(p.blocks(), room) * tile.per_cu;
        const double time = rounds * p.bm * p.bn * ((double)steps / p.splits / (size == 4 ? tile.rate32 : tile.rate16) + ends);
        if (least == 0 || time < least) {
            least = time;
            best = p;
        }
    }
    return best;
}

// Whether rows can be read in place: each starts at 16 bytes and ends with them.
inline bool in_place(const void* p, int64_t stride, int64_t dim, int size)
{
    return (uintptr_t)p % 16 == 0 && stride * size % 16 == 0 && dim * size % 16 == 0 && stride <= kHeadMaxStride;
}

// Workspace of the forward pass: copies of x and table (where needed) | each
// row's partial maxima and sums | the targets' logits.
struct HeadPlan {
    bool copy_x = false, copy_table = false;
    int64_t dp = 0;            // values of a copied row
    int64_t piece = 0;         // rows of a launch
    ProductPlan z;
    int64_t parts = 0;         // partial pairs of a row
    int64_t off_x = 0, off_table = 0, off_part = 0, off_hit = 0, bytes = 0;
};

inline HeadPlan plan_head(bool copy_x, bool copy_table, int size, int64_t n, int64_t vocab, int64_t dim)
{
    HeadPlan p;
    p.copy_x = copy_x;
    p.copy_table = copy_table;
    p.dp = vec_up(dim, 16 / size);
    const int64_t most = vec_ceil(vocab, 64);   // partial pairs of a row, whatever the tile
    p.piece = std::min(n, std::max<int64_t>(kTileRows, kStatBytes / (8 * most) / kTileRows * kTileRows));
    p.z = plan_product(p.piece, vocab, vec_ceil(dim * size, kStepBytes), size, true, false);
    p.parts = p.z.tiles_n * kTiles[p.z.tile].wn;
    p.off_table = copy_x ? vec_up(n * p.dp * size, 256) : 0;
    p.off_part = p.off_table + (copy_table ? vec_up(vocab * p.dp * size, 256) : 0);
    p.off_hit = p.off_part + vec_up(p.parts * p.piece * 8, 256);
    p.bytes = p.off_hit + vec_up(n * 4, 256);
    return p;
}

// Workspace of the gradients: x, rows without a gradient cleared | a copy of
// table (where needed) | rates | the logits' gradient, a piece of the
// vocabulary | dx in 32 bits, by shares | dtable's piece by shares (where split).
struct HeadGradPlan {
    bool copy_table = false;
    int64_t dp = 0;
    int64_t piece = 0;         // tokens of a piece, whole tiles
    int64_t pieces = 0;
    int planes = 1;            // of the logits' gradient
    int64_t stride = 0;        // values of a row of the logits' gradient
    int64_t plane = 0;         // values of a plane
    int64_t width = 0;         // floats of a partial row
    ProductPlan z, dx, dw;     // of a whole piece
    int64_t off_table = 0, off_rate = 0, off_z = 0, off_dx = 0, off_dw = 0, bytes = 0;
};

inline HeadGradPlan plan_head_grad(bool copy_table, int size, int dtable_size, int64_t n, int64_t vocab, int64_t dim,
                                   int wide = kPlanesF16)   // planes beside a wider dtable
{
    HeadGradPlan p;
    p.copy_table = copy_table;
    p.dp = vec_up(dim, 16 / size);
    p.planes = dtable_size > size ? wide : 1;
    const int64_t whole = vec_up(vocab, kTileCols);
    const int64_t room = kPieceBytes / (n * size * std::min(p.planes, 2));
    p.piece = std::min(whole, std::max<int64_t>(kTileCols, room / kTileCols * kTileCols));
    p.pieces = vec_ceil(vocab, p.piece);
    // rows a large power of two apart would share the channels of L2 and memory
    p.stride = p.piece + 128 / size;
    p.plane = n * p.stride;
    p.width = vec_up(dim, 4);
    const int step = kStepBytes / size;
    p.z = plan_product(n, p.piece, vec_ceil(dim, step), size, true, false);
    p.dx = plan_product(n, dim, std::min(p.piece, vocab) / step, size, false, true);
    p.dw = plan_product(std::min(p.piece, vocab), dim, vec_ceil(n, step) * p.planes, size, false, true);
    p.off_table = vec_up(n * p.dp * size, 256);
    p.off_rate = p.off_table + (copy_table ? vec_up(vocab * p.dp * size, 256) : 0);
    p.off_z = p.off_rate + vec_up((n + kRateWords) * 4, 256);
    p.off_dx = p.off_z + vec_up(p.plane * p.planes * size, 256);
    p.off_dw = p.off_dx + vec_up(p.dx.splits * n * p.width * 4, 256);
    p.bytes = p.off_dw + (p.dw.splits > 1 ? vec_up(p.dw.splits * p.piece * p.width * 4, 256) : 0);
    return p;
}

// The gate: a row over 2^log_group lanes, `values` experts in each.
struct GatePlan {
    int values = 8;
    int log_group = 0;
    int per_block = 1;   // rows of a block of 256 threads
};

// LDS of a block: the rows' choices; then of each of its four waves the worths
// of its rows' groups and whether they are kept, or the keys and worths of an
// exact choice.
constexpr int gate_list_bytes(int rows, int top) { return (rows * top * 4 + 7) / 8 * 8; }
inline int gate_wave_bytes(const GatePlan& p, int experts, int groups, bool exact)
{
    return std::max(groups > 1 ? p.per_block / 4 * groups * 8 : 0, exact ? (experts + groups) * 8 : 0);
}
inline int gate_lds(const GatePlan& p, int experts, int groups, int top, bool exact)
{
    return gate_list_bytes(p.per_block, top) + 4 * gate_wave_bytes(p, experts, groups, exact);
}

inline GatePlan plan_gate(int experts)
{
    GatePlan p;
    p.values = experts > 128 ? 16 : 8;
    while ((p.values << p.log_group) < experts) ++p.log_group;
    p.per_block = 256 >> p.log_group;
    return p;
}

}  // namespace hgb
