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

constexpr int kTileRows = 256;    // of a product's tile, and
constexpr int kTileFew = 32;      // where there are no more rows than that
constexpr int kTileCols = 256;
constexpr int kTileNarrow = 64;   // columns, where there are no more than that
constexpr int kStepBytes = 128;   // of a row that one step of a product's sum takes

constexpr int64_t kPieceBytes = (int64_t)1 << 30;   // of the logits' gradient that is held at a time
constexpr int64_t kStatBytes = (int64_t)1 << 28;    // of the forward pass's partial sums

// A product's launch: C [m][n], summed over k in steps, in `splits` shares of
// the steps.
struct ProductPlan {
    int bm = kTileRows, bn = kTileCols;
    int64_t tiles_m = 1, tiles_n = 1;
    int splits = 1;
    int64_t blocks() const { return tiles_m * tiles_n * splits; }
};

inline ProductPlan plan_product(int64_t m, int64_t n, int64_t steps, bool narrow, bool split)
{
    ProductPlan p;
    p.bm = m <= kTileFew ? kTileFew : kTileRows;
    p.bn = narrow && n <= kTileNarrow && p.bm == kTileRows ? kTileNarrow : kTileCols;
    p.tiles_m = vec_ceil(m, p.bm);
    p.tiles_n = vec_ceil(n, p.bn);
    // as many shares as fill the CUs once, of four steps at least
    if (split)
        p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(kHeadCus / (p.tiles_m * p.tiles_n), steps / 4));
    return p;
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

constexpr int tile_parts(int bm) { return bm == kTileRows ? 2 : 4; }   // waves side by side in a tile's columns

inline HeadPlan plan_head(bool copy_x, bool copy_table, int size, int64_t n, int64_t vocab, int64_t dim)
{
    HeadPlan p;
    p.copy_x = copy_x;
    p.copy_table = copy_table;
    p.dp = vec_up(dim, 16 / size);
    const int bm = n <= kTileFew ? kTileFew : kTileRows;
    p.parts = vec_ceil(vocab, kTileCols) * tile_parts(bm);
    p.piece = std::min(n, std::max<int64_t>(kTileRows, kStatBytes / (8 * p.parts) / kTileRows * kTileRows));
    p.z = plan_product(p.piece, vocab, 1, false, false);
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
    int planes = 1;            // of the logits' gradient: 2 beside a 32-bit dtable of 16-bit inputs
    int64_t stride = 0;        // values of a row of the logits' gradient
    int64_t plane = 0;         // values of a plane
    int64_t width = 0;         // floats of a partial row
    ProductPlan z, dx, dw;     // of a whole piece
    int64_t off_table = 0, off_rate = 0, off_z = 0, off_dx = 0, off_dw = 0, bytes = 0;
};

inline HeadGradPlan plan_head_grad(bool copy_table, int size, int dtable_size, int64_t n, int64_t vocab, int64_t dim)
{
    HeadGradPlan p;
    p.copy_table = copy_table;
    p.dp = vec_up(dim, 16 / size);
    p.planes = dtable_size > size ? 2 : 1;
    const int64_t whole = vec_up(vocab, kTileCols);
    p.piece = std::min(whole, std::max<int64_t>(kTileCols, kPieceBytes / (n * size * p.planes) / kTileCols * kTileCols));
    p.pieces = vec_ceil(vocab, p.piece);
    // rows a large power of two apart would share the channels of L2 and memory
    p.stride = p.piece + 128 / size;
    p.plane = n * p.stride;
    p.width = vec_up(dim, 4);
    const int step = kStepBytes / size;
    p.z = plan_product(n, p.piece, 1, false, false);
    p.dx = plan_product(n, dim, p.piece / step, true, true);
    p.dw = plan_product(p.piece, dim, vec_ceil(n, step) * p.planes, true, true);
    p.off_table = vec_up(n * p.dp * size, 256);
    p.off_rate = p.off_table + (copy_table ? vec_up(vocab * p.dp * size, 256) : 0);
    p.off_z = p.off_rate + vec_up((n + 2) * 4, 256);
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
