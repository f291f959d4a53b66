// Launch plans of the vector verbs (embedding, layer norm, routing): sizes in,
// launch shapes and workspace layouts out.  Plain C++, like hgb_plan.h: no HIP
// header, so it is compiled and tested on the host alone.
#pragma once

#include <algorithm>
#include <cstdint>

namespace hgb {

constexpr int64_t kVecMaxDim = 1 << 20;
constexpr int64_t kVecMaxRows = 2147483647;      // rows, tokens and routed slots are int32
constexpr int64_t kVecMaxVocab = 2147483646;     // the key of a dropped token is `vocab`
constexpr int kRouteMaxExperts = 1023;           // one digit holds every expert and the dropped slots' key
constexpr int kRouteMaxTop = 64;

inline int64_t vec_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
inline int64_t vec_ceil(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int vec_bits(int64_t v)   // bits of the values [0, v]
{
    int b = 1;
    while (v >> b) ++b;
    return b;
}
inline int vec_pow2(int64_t v)   // the smallest power of two >= v
{
    int p = 1;
    while (p < v) p *= 2;
    return p;
}

// Stable sort of n keys in [0, limit], least significant digit first.
// Up to kSortSmall keys one block sorts in LDS, all passes in one launch.
// Above that, each pass scatters from `blocks` equal shares of the keys, a
// share being `tiles` tiles of `items` keys a thread taken one after the other.
// Where each block's keys go follows from the digits of all keys: up to
// kSortSelf blocks each counts them itself, beyond that a launch of its own
// counts each share (`count`), and a block sums the counts before it.
constexpr int kSortThreads = 1024;
constexpr int kSortItems = 8;
constexpr int kSortSmall = 4 * kSortThreads;
constexpr int kSortBits = 10;        // of a digit at most, and
constexpr int kSortManyBits = 8;     // where more than kSortFew blocks' counts are summed
constexpr int kSortFew = 32;
constexpr int kSortSelf = 8;
constexpr int kSortMaxBlocks = 512;

struct SortPlan {
    int64_t n = 0;
    int passes = 0;
    int key_bits = 0;    // of a key
    int bits = 0;        // of every digit (the last may have fewer: pass())
    int radix = 0;       // digits' values: 2^bits
    int row = 4;         // words of a share's counts: the radix, at least a 16-byte load
    bool small = false;
    bool count = false;
    int items = 1;       // keys a thread holds of a tile: 1, 4 or kSortItems
    int blocks = 1;
    int tiles = 1;

    void digits(int b)
    {
        bits = b;
        radix = 1 << b;
        row = std::max(radix, 4);
    }
    SortPlan pass(int k) const   // as pass k takes it, whose digits begin at bit k * bits
    {
        SortPlan p = *this;
        p.digits(std::min(bits, key_bits - k * bits));
        return p;
    }
};

inline SortPlan plan_sort(int64_t n, int64_t limit, bool one_pass)
{
    SortPlan p;
    p.n = n;
    p.small = n <= kSortSmall;
    if (p.small) {
        p.items = n <= kSortThreads ? 1 : 4;
    } else {
        // few keys a thread while that gives no CU two blocks
        p.items = n <= 256 * kSortThreads ? 1 : n <= 1024 * kSortThreads ? 4 : kSortItems;
        const int64_t tiles = vec_ceil(n, (int64_t)p.items * kSortThreads);
        p.tiles = (int)vec_ceil(tiles, kSortMaxBlocks);
        p.blocks = (int)vec_ceil(tiles, p.tiles);
        p.count = p.blocks > kSortSelf;
    }
    p.key_bits = vec_bits(limit);
    const int most = one_pass || p.blocks <= kSortFew ? kSortBits : kSortManyBits;
    p.passes = (int)vec_ceil(p.key_bits, most);
    p.digits((int)vec_ceil(p.key_bits, p.passes));
    return p;
}

// Keys that pass through LDS on their way out, so that a digit's keys of a tile
// are stored side by side; with one key a thread the runs are too short.
constexpr int scatter_pair_words(int items) { return items > 1 ? 2 * items * kSortThreads : 0; }

// LDS words in which the one-block sort exchanges its pairs between passes:
// the launch and the kernel lay the rest out behind them.
constexpr int small_pair_words(const SortPlan& p, int items, int threads) { return p.passes > 1 ? 2 * items * threads : 0; }

// One vector of V values a thread, for rows of `dim`: 256 threads take `per`
// whole rows where a row has at most 256 vectors, else one of its `slices` (the
// grid's y: no division, and no branch that would part the kernel's loads of
// its arguments).  Threads that idle: at most a sixteenth for rows of up to 25
// vectors and a third for up to 128, where groups of 2^k lanes leave up to a
// half; but a half just above 128 and 256 vectors, as those do (129 50%, 150
// 41%, 257 50%).  Embedding 100,000 rows, fp32 to bf16: 1,024 values 78 us, 1,040
// 84; 2,048 values 160, 2,056 211.
struct RowMap {
    int vecs = 1;
    int per = 1;
    int slices = 1;
    int magic = 0;   // thread / vecs = thread * magic >> 16
};

inline RowMap plan_rows(int64_t dim, int V)
{
    RowMap m;
    m.vecs = (int)vec_ceil(dim, V);
    m.per = std::max(1, 256 / m.vecs);
    m.slices = (int)vec_ceil(m.vecs, 256);
    m.magic = m.vecs <= 256 ? 65536 / m.vecs + 1 : 0;
    return m;
}

inline int64_t row_blocks(const RowMap& m, int64_t rows) { return vec_ceil(rows, m.per); }

// A dimension of a grid holds fewer than 2^32 threads.  Blocks of 256 threads
// beyond kGridBlocks go on in the grid's z: block b is (b % kGridBlocks, b /
// kGridBlocks), and a part-filled last layer's blocks find no work.
constexpr int kGridLog = 23;
constexpr int64_t kGridBlocks = (int64_t)1 << kGridLog;
struct GridSpan {
    unsigned x = 1, z = 1;
};
inline GridSpan span_blocks(int64_t blocks)
{
    GridSpan g;
    g.x = (unsigned)std::min(blocks, kGridBlocks);
    g.z = (unsigned)vec_ceil(blocks, kGridBlocks);
    return g;
}

// The embedding's gradient: the sort, then chunks of sorted positions.
// Workspace: counts | pairs A | pairs B | partial sums (two rows a chunk) |
// how each chunk ends.
struct EmbedPlan {
    SortPlan sort;
    int chunk = 1;             // sorted positions a group of lanes sums
    int64_t chunks = 0;
    int64_t part_stride = 0;   // floats of a partial row
    int64_t off_a = 0, off_b = 0, off_part = 0, off_ends = 0, bytes = 0;
};

constexpr int kEmbedChunk = 256;         // largest chunk
constexpr int kEmbedFew = 32;
constexpr int64_t kEmbedWaves = 8192;    // chunks are halved until this many waves run (32 a CU), below
                                        // 32 tokens a quarter, below 16 a sixteenth

inline EmbedPlan plan_embed(int64_t n, int64_t vocab, int64_t dim)
{
    EmbedPlan p;
    p.sort = plan_sort(n, vocab, false);
    // The narrowest lanes' values (4) decide, so that the plan and the
    // workspace do not depend on the types.
    const int64_t vecs = vec_ceil(dim, 4);
    // a handful of tokens is one chunk: nothing to join
    p.chunk = n <= kEmbedFew ? kEmbedFew : kEmbedChunk;
    auto fewer = [&](int least, int64_t waves) {
        while (p.chunk > least && vec_ceil(n, p.chunk) * vecs / 64 < waves) p.chunk /= 2;
    };
    if (n > kEmbedFew) {
        fewer(32, kEmbedWaves);
        fewer(16, kEmbedWaves / 4);
        fewer(8, kEmbedWaves / 16);
    }
    p.chunks = vec_ceil(n, p.chunk);
    p.part_stride = vec_up(dim, 4);
    p.off_a = p.sort.count ? vec_up((int64_t)p.sort.blocks * p.sort.row * 4, 256) : 0;
    p.off_b = p.off_a + vec_up(n * 8, 256);
    p.off_part = p.off_b + (p.sort.small ? 0 : vec_up(n * 8, 256));
    p.off_ends = p.off_part + vec_up(p.chunks * 2 * p.part_stride * 4, 256);
    p.bytes = p.off_ends + vec_up(p.chunks * 4, 256);
    return p;
}

// The routing's sort: counts only.
inline int64_t route_workspace(int64_t slots, int experts)
{
    const SortPlan p = plan_sort(slots, experts, true);
    return p.count ? vec_up((int64_t)p.blocks * p.row * 4, 256) : 0;
}

// The layer norm's launch: `values` of a row in each lane's registers, a row
// over 2^log_group lanes of a wave (waves = 1) or over all `waves` of a block.
// `values` = 0: the row is too wide for registers and is read again.
constexpr int kNormThreads = 512;      // of a block whose waves take a row each
constexpr int kNormMaxDim = 16384;     // 16 values a lane, 16 waves (32 spill: a block of 16 waves has 128 registers a lane)
constexpr int kNormParts = 256;        // blocks of the backward pass: one a CU
constexpr int norm_threads(int waves) { return waves > 1 ? 64 * waves : kNormThreads; }

// Threads of a block of the backward pass: with 32 values a lane the registers
// hold three waves on a SIMD.
constexpr int norm_grad_threads(int values, int waves) { return waves == 1 && values == 32 ? 768 : norm_threads(waves); }

struct NormPlan {
    int values = 0;
    int waves = 1;
    int log_group = 6;
    int per_block = 1;   // rows of a block at a time
};

inline NormPlan plan_norm(int64_t dim)
{
    NormPlan p;
    if (dim > kNormMaxDim) return p;
    p.waves = dim <= 2048 ? 1 : dim <= 8192 ? 4 : 16;
    const int64_t lane = vec_ceil(dim, 64 * p.waves);   // values a lane
    p.values = lane <= 8 ? 8 : lane <= 16 ? 16 : 32;
    if (dim <= 512) {
        p.log_group = 0;
        while ((8 << p.log_group) < dim) ++p.log_group;
    }
    p.per_block = p.waves > 1 ? 1 : kNormThreads >> p.log_group;
    return p;
}

// Partial rows of the parameters' gradients, [2][dim] floats each: of the wide
// rows' kernel (shares of 16 rows and more), and the register kernel's blocks.
inline int norm_parts(int64_t rows) { return (int)std::min<int64_t>(kNormParts, std::max<int64_t>(1, vec_ceil(rows, 16))); }
inline int norm_blocks(int64_t rows, const NormPlan& p)
{
    const int64_t each = p.waves > 1 ? 1 : norm_grad_threads(p.values, 1) >> p.log_group;   // rows of a block at a time
    const int64_t steps = std::max<int64_t>(1, vec_ceil(rows, each));
    // Two blocks a CU fit with four waves, and with 8 values a lane, where their
    // sums are worth it from 8 rows a wave on: 100,000 rows of 512 bf16 values
    // take 55 us with two and 62 with one, 22,888 of 242 14.8 and 14.2.
    const bool two = p.waves == 4 || (p.values == 8 && steps >= 8 * 2 * kNormParts);
    return (int)std::min<int64_t>(two ? 2 * kNormParts : kNormParts, steps);
}
inline int64_t norm_workspace(int64_t rows, int64_t dim)
{
    return vec_up((int64_t)std::max(norm_parts(rows), norm_blocks(rows, plan_norm(dim))) * dim * 2 * 4, 256);
}

}  // namespace hgb
