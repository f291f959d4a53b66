// Device kernels of the vector verbs (gfx950).  Internal header: included by
// hgb_vectors.hip only.
//
// Rows are vectors of `dim` values of T (float, __bf16, _Float16); sums and
// statistics are 32-bit floats, rounded once when they are stored.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "hgb_ctx.h"
#include "hgb_vector_plan.h"

namespace hgb {

// Values a lane takes of a row at a time: 16 bytes of the narrower type.
template <typename T, typename U = T>
constexpr int kVals = sizeof(T) < 4 || sizeof(U) < 4 ? 8 : 4;

// V values as one load or store; rows may start at any element (gfx950
// serves global accesses of any alignment).
template <typename T, int V>
struct Vals {
    typedef T type __attribute__((ext_vector_type(V), aligned(sizeof(T))));
};

// `left` of the values lie in the row, the others are zeros.  WHOLE: all do or
// none, which spares the code for a part: a row's last vector then ends where
// the row does and shares values with the one before it (both store the same).
// STREAM: past the caches, for rows that a large call reads once.
template <int V, bool WHOLE = false, bool STREAM = false, typename T>
__device__ inline typename Vals<T, V>::type load_raw(const T* p, int64_t left)
{
    typedef typename Vals<T, V>::type Vec;
    Vec v{};
    if (WHOLE ? left > 0 : left >= V) {
        v = STREAM ? __builtin_nontemporal_load((const Vec*)p) : *(const Vec*)p;
    } else if (!WHOLE) {
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = k < left ? p[k] : (T)0.0f;
    }
    return v;
}

template <int V, bool WHOLE = false, typename T>
__device__ inline void load_vals(float (&r)[V], const T* p, int64_t left)
{
    const typename Vals<T, V>::type v = load_raw<V, WHOLE>(p, left);
#pragma unroll
    for (int k = 0; k < V; ++k) r[k] = (float)v[k];
}

// `stream`: past the caches, for large calls.
template <int V, bool WHOLE = false, typename T>
__device__ inline void store_raw(const typename Vals<T, V>::type& v, T* p, int64_t left, bool stream)
{
    typedef typename Vals<T, V>::type Vec;
    if (WHOLE ? left > 0 : left >= V) {
        if (stream) {
            // the empty asm keeps the two stores apart: made one, they lose the hint
            asm volatile("");
            __builtin_nontemporal_store(v, (Vec*)p);
            asm volatile("");
        } else {
            *(Vec*)p = v;
        }
    } else if (!WHOLE) {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k < left) p[k] = v[k];
    }
}

template <int V, bool WHOLE = false, typename T>
__device__ inline void store_vals(const float (&r)[V], T* p, int64_t left, bool stream = false)
{
    typename Vals<T, V>::type v;
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = (T)r[k];
    store_raw<V, WHOLE>(v, p, left, stream);
}

// A block's number in a grid of span_blocks.
__device__ inline uint32_t block_number() { return (blockIdx.z << kGridLog) + blockIdx.x; }

// A thread's place among rows of `dim` (plan_rows): its row, the first column
// of its vector (the last vector is moved back to end with the row) and
// whether it has one.
struct RowPlace {
    uint32_t r;
    int c;
    bool in;
};

template <int V>
__device__ inline RowPlace row_place(const RowMap& m, uint32_t rows, int dim)
{
    const int t = threadIdx.x, q = (t * m.magic) >> 16, j = (int)blockIdx.y * 256 + t - q * m.vecs;
    RowPlace p;
    p.r = block_number() * (uint32_t)m.per + (uint32_t)q;
    p.c = dim < V ? 0 : min(j * V, dim - V);
    p.in = q < m.per && j < m.vecs && p.r < rows;
    return p;
}

// x plus the value of the lane that CTRL names in its row of 16.
template <int CTRL>
__device__ inline float dpp_add(float x)
{
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}

// Sums over aligned groups of 2^log_group lanes; every lane of a group gets
// its sum, the same bits.  Moves between lanes in the vector unit: no trip
// through LDS as a shuffle makes.
__device__ inline float group_sum(float x, int log_group)
{
    if (log_group > 0) x = dpp_add<0xb1>(x);    // lanes 1, 0, 3, 2 of a quad
    if (log_group > 1) x = dpp_add<0x4e>(x);    // lanes 2, 3, 0, 1
    if (log_group > 2) x = dpp_add<0x141>(x);   // the other quad of eight, mirrored
    if (log_group > 3) x = dpp_add<0x140>(x);   // the other eight of sixteen
    if (log_group > 4) {
        const uint32_t u = __float_as_uint(x);
        const auto v = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        x = __uint_as_float(v[0]) + __uint_as_float(v[1]);
    }
    if (log_group > 5) {
        const uint32_t u = __float_as_uint(x);
        const auto v = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        x = __uint_as_float(v[0]) + __uint_as_float(v[1]);
    }
    return x;
}

// ---------------------------------------------------------------------------
// Stable sort by key
// ---------------------------------------------------------------------------

// What a sort reads and writes.  A key is a token or expert below `limit`;
// every other value, and `pad`, sorts last under the key `limit`.
struct SortIn {
    const int32_t* tokens;   // the first pass's input
    const uint2* from;       // a later pass's input (key, index)
    int64_t n;
    int64_t limit;
    int32_t pad;
    uint32_t flag;           // raised for a value that is neither a key nor pad
    uint32_t* err;
};

struct SortOut {
    uint2* to;               // (key, index), or
    int32_t* order;          // index by place (-1: none),
    int32_t* position;       // place by index (-1: none)
    int32_t* offsets;        // and the first place of each key
};

template <bool FIRST>
__device__ inline uint2 sort_load(const SortIn& in, int64_t i, bool* bad)
{
    if (!FIRST) return in.from[i];
    const int32_t t = in.tokens[i];
    const bool live = t != in.pad && t >= 0 && t < in.limit;
    if (!live && t != in.pad) *bad = true;
    return make_uint2(live ? (uint32_t)t : (uint32_t)in.limit, (uint32_t)i);
}

__device__ inline void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Ranks of a tile's digits.  Item i of lane l of wave w is element
// w * 64 * ITEMS + i * 64 + l, so that a wave meets its elements in order.
// rank[i]: the elements of the same digit before it in its wave; on return
// count[w * radix + d] holds the digit's elements in the waves before w and
// total[d] those of the whole tile.
// WAVES: the block's, where the compiler may know and the registers suffice.
template <int ITEMS, int WAVES = 0>
__device__ inline void tile_ranks(const uint32_t (&digit)[ITEMS], int live, int bits, int radix, uint32_t* count,
                                  uint32_t* total, uint32_t (&rank)[ITEMS])
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, waves = WAVES ? WAVES : blockDim.x >> 6;
    for (int i = threadIdx.x; i < waves * radix; i += blockDim.x) count[i] = 0;
    __syncthreads();
    uint32_t* mine = count + w * radix;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int at = w * 64 * ITEMS + i * 64 + lane;
        const bool in = at < live;
        // the lanes with this lane's digit, a bit at a time
        const uint64_t lanes = __ballot(in);
        uint32_t lo = (uint32_t)lanes, hi = (uint32_t)(lanes >> 32);
#pragma unroll
        for (int b = 0; b < kSortBits; ++b)
            if (b < bits) {
                const uint32_t one = (uint32_t)((int32_t)(digit[i] << (31 - b)) >> 31);   // the bit, 32 times
                const uint64_t m = __ballot(one != 0);
                lo &= ~((uint32_t)m ^ one);
                hi &= ~((uint32_t)(m >> 32) ^ one);
            }
        const int before = __builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0));
        if (in) rank[i] = mine[digit[i]] + before;
        wave_order();
        if (in && before == 0) mine[digit[i]] = rank[i] + __popc(lo) + __popc(hi);
        wave_order();
    }
    __syncthreads();
    for (int d = threadIdx.x; d < radix; d += blockDim.x) {
        uint32_t sum = 0;
        if (WAVES) {   // all loads before the first store
            uint32_t c[WAVES ? WAVES : 1];
#pragma unroll
            for (int k = 0; k < WAVES; ++k) c[k] = count[k * radix + d];
#pragma unroll
            for (int k = 0; k < WAVES; ++k) {
                count[k * radix + d] = sum;
                sum += c[k];
            }
        } else {
            for (int k = 0; k < waves; ++k) {
                const uint32_t c = count[k * radix + d];
                count[k * radix + d] = sum;
                sum += c;
            }
        }
        total[d] = sum;
    }
    __syncthreads();
}

// Exclusive sums of v[0, radix) in place, radix <= the block's threads;
// `tmp` holds a word per wave.
template <int WAVES = 0>
__device__ inline void block_scan(uint32_t* v, int radix, uint32_t* tmp)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, waves = WAVES ? WAVES : blockDim.x >> 6;
    const uint32_t own = (int)threadIdx.x < radix ? v[threadIdx.x] : 0;
    uint32_t x = own;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t y = __shfl_up(x, d, 64);
        if (lane >= d) x += y;
    }
    if (lane == 63) tmp[w] = x;
    __syncthreads();
    uint32_t before = 0;
    for (int k = 0; k < waves; ++k)
        if (k < w) before += tmp[k];
    if ((int)threadIdx.x < radix) v[threadIdx.x] = before + x - own;
    __syncthreads();
}

// Zeros to `rows` rows of `cols` elements, by the blocks that call it.
struct ZeroFill {
    void* out = nullptr;
    int64_t rows = 0, cols = 0, stride = 0;   // elements
    int elem = 4;                             // bytes
    bool stream = false;                      // past the caches
};

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

__device__ inline void zero_row(char* p, int64_t bytes, int64_t first, int64_t step, bool stream)
{
    const int64_t whole = bytes / 16;
    if (stream)
        for (int64_t i = first; i < whole; i += step) __builtin_nontemporal_store(u32x4_any{0, 0, 0, 0}, (u32x4_any*)(p + 16 * i));
    else
        for (int64_t i = first; i < whole; i += step) *(u32x4_any*)(p + 16 * i) = u32x4_any{0, 0, 0, 0};
    for (int64_t i = whole * 8 + first; i < bytes / 2; i += step) ((uint16_t*)p)[i] = 0;
}

__device__ inline void zero_fill(const ZeroFill& z, int block, int blocks)
{
    if (z.stride == z.cols) {
        zero_row((char*)z.out, z.rows * z.cols * z.elem, (int64_t)block * blockDim.x + threadIdx.x,
                 (int64_t)blocks * blockDim.x, z.stream);
        return;
    }
    for (int64_t r = block; r < z.rows; r += blocks)
        zero_row((char*)z.out + r * z.stride * z.elem, z.cols * z.elem, threadIdx.x, blockDim.x, z.stream);
}

// One block sorts up to kSortSmall keys, all passes in LDS; the other blocks
// write the zeros.  LDS: pairs [ITEMS * threads] where there are several passes
// (small_pair_words), counts [waves][radix], totals [radix], scan words.
template <int ITEMS>
__global__ __launch_bounds__(kSortThreads) void k_sort_small(SortIn in, SortOut out, SortPlan p, ZeroFill z)
{
    if (blockIdx.x > 0) {
        zero_fill(z, blockIdx.x - 1, gridDim.x - 1);
        return;
    }
    extern __shared__ uint32_t lds[];
    const int waves = blockDim.x >> 6;
    uint2* pairs = (uint2*)lds;
    uint32_t* count = lds + small_pair_words(p, ITEMS, blockDim.x);
    uint32_t* total = count + waves * p.radix;
    uint32_t* tmp = total + p.radix;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, first = w * 64 * ITEMS + lane;
    const int n = (int)in.n;
    uint2 kv[ITEMS];
    uint32_t digit[ITEMS], rank[ITEMS];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        kv[i] = make_uint2(0, 0);
        if (first + i * 64 < n) kv[i] = sort_load<true>(in, first + i * 64, &bad);
    }
    if (bad) atomicOr(in.err, in.flag);
    for (int pass = 0; pass < p.passes; ++pass) {
        const int shift = pass * p.bits;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) digit[i] = (kv[i].x >> shift) & (p.radix - 1);
        tile_ranks<ITEMS>(digit, n, p.bits, p.radix, count, total, rank);
        block_scan(total, p.radix, tmp);
        const bool last = pass == p.passes - 1;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            if (first + i * 64 < n) {
                const int at = (int)(total[digit[i]] + count[w * p.radix + digit[i]] + rank[i]);
                if (!last) {
                    pairs[at] = kv[i];
                } else if (out.to) {
                    out.to[at] = kv[i];
                } else {
                    const bool live = kv[i].x < (uint32_t)in.limit;
                    out.order[at] = live ? (int32_t)kv[i].y : -1;
                    out.position[kv[i].y] = live ? at : -1;
                }
            }
        if (last) {
            if (out.offsets)
                for (int d = threadIdx.x; d <= in.limit; d += blockDim.x) out.offsets[d] = (int32_t)total[d];
            break;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            if (first + i * 64 < n) kv[i] = pairs[first + i * 64];
    }
}

// hist[digit of key i] += 1 for the keys [begin, end), by the whole block.
// Eight keys a thread are loaded before they are counted.
template <bool FIRST>
__device__ inline bool count_digits(const SortIn& in, const SortPlan& p, int shift, int64_t begin, int64_t end,
                                    uint32_t* hist)
{
    bool bad = false;
    for (int64_t i = begin + threadIdx.x; i < end; i += 8 * kSortThreads) {
        uint32_t key[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) key[u] = i + u * kSortThreads < end ? sort_load<FIRST>(in, i + u * kSortThreads, &bad).x : 0;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (i + u * kSortThreads < end) atomicAdd(&hist[(key[u] >> shift) & (p.radix - 1)], 1u);
    }
    return bad;
}

// counts[block][digit] of one pass, rows of p.row; blocks past p.blocks write the zeros.
template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void k_sort_count(SortIn in, SortPlan p, int shift, uint32_t* counts,
                                                             ZeroFill z)
{
    if ((int)blockIdx.x >= p.blocks) {
        zero_fill(z, blockIdx.x - p.blocks, gridDim.x - p.blocks);
        return;
    }
    extern __shared__ uint32_t lds[];
    for (int d = threadIdx.x; d < p.row; d += blockDim.x) lds[d] = 0;
    __syncthreads();
    const int64_t share = (int64_t)p.tiles * p.items * kSortThreads, begin = blockIdx.x * share;
    if (count_digits<FIRST>(in, p, shift, begin, begin + share < in.n ? begin + share : in.n, lds)) atomicOr(in.err, in.flag);
    __syncthreads();
    for (int d = threadIdx.x; d < p.row; d += blockDim.x) counts[(int64_t)blockIdx.x * p.row + d] = lds[d];
}

// The pass's scatter: each block finds where its digits' keys begin (from the
// shares' counts, at most kSortMaxBlocks rows of them and read from L2, or by
// counting all keys itself) instead of a scan in a launch of its own, then
// ranks its tiles in order.  Blocks past p.blocks write the zeros.  3,670,016
// keys by 128 digits: 27 us, of which 5 for the counts, 6 for the ranks, 4 to
// pass through LDS and out (38 us with the pairs stored from their lanes and
// the counts read a word at a time).
template <bool FIRST, int ITEMS>
__global__ __launch_bounds__(kSortThreads, 8) void k_sort_scatter(SortIn in, SortOut out, SortPlan p, int shift,
                                                                  const uint32_t* counts, ZeroFill z)
{
    if ((int)blockIdx.x >= p.blocks) {
        zero_fill(z, blockIdx.x - p.blocks, gridDim.x - p.blocks);
        return;
    }
    extern __shared__ uint32_t lds[];
    constexpr int kTile = ITEMS * kSortThreads;
    const int waves = blockDim.x >> 6;
    uint2* pairs = (uint2*)lds;                        // [kTile], where ITEMS > 1
    uint32_t* count = lds + scatter_pair_words(ITEMS);  // [waves][radix]
    uint32_t* total = count + waves * p.radix;         // [radix]
    uint32_t* base = total + p.radix;                  // [radix]
    uint32_t* tmp = base + p.radix;                    // [waves]
    // base[d] = keys of smaller digits + keys of digit d in earlier blocks
    if ((int)threadIdx.x < p.radix) total[threadIdx.x] = base[threadIdx.x] = 0;
    __syncthreads();
    if (p.count) {
        // four digits a thread, eight shares at a time
        const int quads = p.row / 4, d = (threadIdx.x & (quads - 1)) * 4, g = threadIdx.x / quads, groups = blockDim.x / quads;
        uint32_t all[4] = {0, 0, 0, 0}, before[4] = {0, 0, 0, 0};
        for (int b = g; b < p.blocks; b += 8 * groups) {
            uint4 c[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int k = b + u * groups;
                c[u] = k < p.blocks ? *(const uint4*)(counts + (int64_t)k * p.row + d) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const uint32_t v[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
                const bool earlier = b + u * groups < (int)blockIdx.x;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    all[k] += v[k];
                    before[k] += earlier ? v[k] : 0;
                }
            }
        }
        if (g < p.blocks)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (d + k < p.radix) {
                    atomicAdd(&total[d + k], all[k]);
                    atomicAdd(&base[d + k], before[k]);
                }
        __syncthreads();
    } else {
        const int64_t begin = (int64_t)blockIdx.x * p.tiles * kTile;
        bool bad = count_digits<FIRST>(in, p, shift, 0, begin, base);
        bad |= count_digits<FIRST>(in, p, shift, begin, in.n, total);
        if (bad && blockIdx.x == 0) atomicOr(in.err, in.flag);
        __syncthreads();
        if ((int)threadIdx.x < p.radix) total[threadIdx.x] += base[threadIdx.x];
        __syncthreads();
    }
    block_scan<ITEMS == 1 ? kSortThreads / 64 : 0>(total, p.radix, tmp);
    if (out.offsets && blockIdx.x == 0)
        for (int k = threadIdx.x; k <= in.limit; k += blockDim.x) out.offsets[k] = (int32_t)total[k];
    if ((int)threadIdx.x < p.radix) base[threadIdx.x] += total[threadIdx.x];
    __syncthreads();
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, first = w * 64 * ITEMS + lane;
    for (int t = 0; t < p.tiles; ++t) {
        const int64_t begin = ((int64_t)blockIdx.x * p.tiles + t) * kTile;
        if (begin >= in.n) break;
        const int live = in.n - begin < kTile ? (int)(in.n - begin) : kTile;
        uint2 kv[ITEMS];
        uint32_t digit[ITEMS], rank[ITEMS];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            kv[i] = make_uint2(0, 0);
            if (first + i * 64 < live) kv[i] = sort_load<FIRST>(in, begin + first + i * 64, &bad);
            digit[i] = (kv[i].x >> shift) & (p.radix - 1);
        }
        tile_ranks<ITEMS, ITEMS == 1 ? kSortThreads / 64 : 0>(digit, live, p.bits, p.radix, count, total, rank);
        if (ITEMS == 1) {
            if (first < live) {
                const int64_t at = base[digit[0]] + count[w * p.radix + digit[0]] + rank[0];
                const bool keep = kv[0].x < (uint32_t)in.limit;
                if (out.to) {
                    out.to[at] = kv[0];
                } else {
                    out.order[at] = keep ? (int32_t)kv[0].y : -1;
                    out.position[kv[0].y] = keep ? (int32_t)at : -1;
                }
            }
            __syncthreads();
            if ((int)threadIdx.x < p.radix) base[threadIdx.x] += total[threadIdx.x];
            continue;
        }
        // in LDS at their place in the tile: total becomes the digits' first
        // places there, and base what leads from such a place to the output's
        const uint32_t keys = (int)threadIdx.x < p.radix ? total[threadIdx.x] : 0;
        block_scan<ITEMS == 1 ? kSortThreads / 64 : 0>(total, p.radix, tmp);
        if ((int)threadIdx.x < p.radix) base[threadIdx.x] -= total[threadIdx.x];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            if (first + i * 64 < live) {
                const uint32_t at = total[digit[i]] + count[w * p.radix + digit[i]] + rank[i];
                pairs[at] = kv[i];
                if (!out.to) out.position[kv[i].y] = kv[i].x < (uint32_t)in.limit ? (int32_t)(base[digit[i]] + at) : -1;
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int at = i * kSortThreads + threadIdx.x;
            if (at < live) {
                const uint2 v = pairs[at];
                const uint32_t to = base[(v.x >> shift) & (p.radix - 1)] + at;
                if (out.to) out.to[to] = v;
                else out.order[to] = v.x < (uint32_t)in.limit ? (int32_t)v.y : -1;
            }
        }
        __syncthreads();
        if ((int)threadIdx.x < p.radix) base[threadIdx.x] += total[threadIdx.x] + keys;
    }
}

// ---------------------------------------------------------------------------
// Embedding
// ---------------------------------------------------------------------------

// out[i] = scale * table[token i], a vector a thread.  Bound by the bytes
// written (the table's rows come from L2): 3,670,016 rows of 64 bf16 values in
// 81 us, 5.8 TB/s (a fill: 84 us).  Four tokens a thread 90 us: more
// instructions before the first store, and blocks less in order.
template <typename T, typename U>
__global__ __launch_bounds__(256) void k_embed(const T* __restrict__ table, int64_t table_stride, int vocab, int dim,
                                               const int32_t* __restrict__ tokens, int n, int32_t pad, float scale,
                                               U* __restrict__ out, int64_t out_stride, RowMap m, bool stream,
                                               uint32_t* err)
{
    constexpr int V = kVals<T, U>;
    const RowPlace at = row_place<V>(m, n, dim);
    if (!at.in) return;
    const int32_t t = tokens[at.r];
    const bool live = t != pad && (uint32_t)t < (uint32_t)vocab;
    if (!live && t != pad && at.c == 0) atomicOr(err, kVecErrToken);
    const T* from = table + (uint64_t)(live ? (uint32_t)t : 0) * (uint64_t)table_stride + at.c;
    U* to = out + (uint64_t)at.r * (uint64_t)out_stride + at.c;
    auto copy = [&](auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        float v[V];
        load_vals<V, WHOLE>(v, from, live ? dim : 0);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = live ? v[k] * scale : 0.0f;
        store_vals<V, WHOLE>(v, to, dim, stream);
    };
    if (dim >= V) copy(std::true_type());
    else copy(std::false_type());
}

__global__ __launch_bounds__(256) void k_zero_rows(ZeroFill z) { zero_fill(z, blockIdx.x, gridDim.x); }

// Sums of the gradient's rows over each run of equal keys.  The threads of a
// row's vectors walk one chunk of sorted positions; a run that lies in its chunk is
// finished there, and a run that crosses a border leaves its part in the
// chunk's partial rows: row 0 a run that began before the chunk, row 1 one
// that begins in it and goes on.  ends[chunk] tells k_embed_join: the key of a
// run that begins in the chunk and goes on, kChunkWhole where one run fills the
// chunk and goes on at both ends, else kChunkNone.  The order of the sums
// depends on the tokens alone.  Bound by the gradient's rows, 128 bytes each in the measured case, in
// the tokens' order: 3,670,016 rows of 64 bf16 values in 104 us, 4.7 TB/s (with a
// quarter of the waves 108, those through the caches 114; a large copy: 4.9 TB/s).
constexpr uint32_t kChunkNone = 0xffffffffu, kChunkWhole = 0xfffffffeu;   // no key is that large

template <typename T, typename U>
__global__ __launch_bounds__(256) void k_embed_sum(const uint2* __restrict__ pairs, int64_t n, const T* __restrict__ grad,
                                                   int64_t grad_stride, int64_t dim, int64_t vocab, float scale,
                                                   U* __restrict__ out, int64_t out_stride, float* __restrict__ part,
                                                   int64_t part_stride, uint32_t* __restrict__ ends, int chunk,
                                                   int64_t chunks, RowMap m, bool stream)
{
    constexpr int V = kVals<T, U>;
    const RowPlace at = row_place<V>(m, (uint32_t)chunks, (int)dim);
    if (!at.in) return;
    const int64_t id = at.r, c = at.c, begin = id * chunk, end = begin + chunk < n ? begin + chunk : n;
    const uint32_t none = 0xffffffffu;
    const uint32_t prev = begin > 0 ? pairs[begin - 1].x : none, next = end < n ? pairs[end].x : none;
    // STEP rows in flight; fewer where a row is shorter than a vector and its
    // values are loaded one by one
    auto walk = [&](auto step, auto past) {
        constexpr int STEP = decltype(step)::value;
        constexpr bool WHOLE = STEP == 8, STREAM = decltype(past)::value;
        uint32_t cur = pairs[begin].x;
        bool head = cur == prev;
        float acc[V];
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = 0.0f;
        auto flush = [&](bool open) {
            if (cur >= (uint32_t)vocab) return;
            if (head || open) {
                store_vals<V, WHOLE>(acc, part + (id * 2 + (head ? 0 : 1)) * part_stride + c, dim);
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k) acc[k] *= scale;
                store_vals<V, WHOLE>(acc, out + (int64_t)cur * out_stride + c, dim);
            }
        };
        uint2 ahead[STEP];   // the next step's pairs
#pragma unroll
        for (int u = 0; u < STEP; ++u) ahead[u] = pairs[begin + u < end ? begin + u : end - 1];
        for (int64_t j = begin; j < end; j += STEP) {
            uint2 kv[STEP];
            typename Vals<T, V>::type v[STEP];
#pragma unroll
            for (int u = 0; u < STEP; ++u) kv[u] = ahead[u];
            // a dropped token's row is not read: its sum, which no one stores, takes row 0
#pragma unroll
            for (int u = 0; u < STEP; ++u)
                v[u] = load_raw<V, WHOLE, STREAM>(
                    grad + (kv[u].x < (uint32_t)vocab ? (uint64_t)kv[u].y : 0) * (uint64_t)grad_stride + c, dim);
#pragma unroll
            for (int u = 0; u < STEP; ++u) ahead[u] = pairs[j + STEP + u < end ? j + STEP + u : end - 1];
#pragma unroll
            for (int u = 0; u < STEP; ++u) {
                if (j + u >= end) break;
                if (kv[u].x != cur) {
                    flush(false);
                    cur = kv[u].x;
                    head = false;
#pragma unroll
                    for (int k = 0; k < V; ++k) acc[k] = 0.0f;
                }
#pragma unroll
                for (int k = 0; k < V; ++k) acc[k] += (float)v[u][k];
            }
        }
        flush(cur == next);
        if (c == 0) ends[id] = cur != next || cur >= (uint32_t)vocab ? kChunkNone : head ? kChunkWhole : cur;
    };
    if (dim < V) walk(std::integral_constant<int, 4>(), std::false_type());
    else if (stream) walk(std::integral_constant<int, 8>(), std::true_type());
    else walk(std::integral_constant<int, 8>(), std::false_type());
}

// Runs that cross chunk borders: the partial row 1 of the chunk where the run
// begins plus row 0 of each chunk it goes on in.  A block takes `own` chunks (up
// to 64, which it sees) and 64 columns: the lanes of a partial row's columns sum
// a short run, the whole block a long one, joined in a fixed order.  Bound by its
// chain of loads that wait for one another: 5.5 us for 626 chunks, 8.5 for
// 57,344.  (A wave a chunk that looks for its run among the keys took 5.3 and 19.)
constexpr int kJoinChunks = 64;
constexpr int kJoinLong = 16;

template <typename U>
__global__ __launch_bounds__(256) void k_embed_join(const uint32_t* __restrict__ ends, int dim, float scale,
                                                    U* __restrict__ out, int64_t out_stride, const float* __restrict__ part,
                                                    int64_t part_stride, int chunks, int own, int log_cols)
{
    __shared__ int first[kJoinChunks], last[kJoinChunks], count;   // of the runs that begin here
    __shared__ uint32_t key[kJoinChunks];
    __shared__ float4 sums[4][16];
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if (w == 0) {
        const int base = blockIdx.x * own, id = base + lane;
        const uint32_t e = id < chunks ? ends[id] : kChunkNone;
        const bool begins = e < kChunkWhole && lane < own;
        const uint64_t begin = __ballot(begins), whole = __ballot(e == kChunkWhole);
        // a run ends in the first chunk after it that is not whole
        const uint64_t after = lane < 63 ? whole >> (lane + 1) : 0;
        const int len = __ffsll((unsigned long long)~after) - 1;   // whole chunks that follow
        int more = 0;
        if (__any(begins && lane + len == 63)) {   // beyond what the block sees, 256 at a glance
            for (int n = 256; n == 256; more += n) {
                const int at = base + kJoinChunks + more + lane * 4;
                n = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) n += n == k && at + k < chunks && ends[at + k] == kChunkWhole;
                const uint64_t part_full = ~__ballot(n == 4);
                const int full = part_full ? __ffsll((unsigned long long)part_full) - 1 : 64;   // lanes before the first with another
                n = full == 64 ? 256 : full * 4 + __shfl(n, full, 64);
            }
        }
        if (begins) {
            const int at = __builtin_amdgcn_mbcnt_hi((uint32_t)(begin >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)begin, 0));
            first[at] = id;
            last[at] = id + len + 1 + (lane + len == 63 ? more : 0);
            key[at] = e;
        }
        if (lane == 0) count = __popcll(begin);
    }
    __syncthreads();
    // 2^log_cols lanes hold a row's columns, four each
    const int cols = 1 << log_cols, group = threadIdx.x >> log_cols, groups = 256 >> log_cols;
    const int c = blockIdx.y * 64 + (lane & (cols - 1)) * 4;
    const bool in = c < dim;   // part rows are padded to four floats
    auto sum = [&](int from, int to, int step, int begin) {
        float4 a = make_float4(0, 0, 0, 0);
        if (in)
#pragma unroll 8
            for (int k = from; k <= to; k += step) {
                const float4 v = *(const float4*)(part + ((int64_t)k * 2 + (k == begin ? 1 : 0)) * part_stride + c);
                a.x += v.x;
                a.y += v.y;
                a.z += v.z;
                a.w += v.w;
            }
        return a;
    };
    auto store = [&](const float4& a, uint32_t k) {
        const float r[4] = {a.x * scale, a.y * scale, a.z * scale, a.w * scale};
        if (in) store_vals<4>(r, out + (int64_t)k * out_stride + c, dim - c);
    };
    for (int i = group; i < count; i += groups)
        if (last[i] - first[i] <= kJoinLong) store(sum(first[i], last[i], 1, first[i]), key[i]);
    for (int i = 0; i < count; ++i) {
        if (last[i] - first[i] <= kJoinLong) continue;
        float4 a = sum(first[i] + group, last[i], groups, first[i]);
        for (int d = cols; d < 64; d *= 2) {
            a.x += __shfl_xor(a.x, d, 64);
            a.y += __shfl_xor(a.y, d, 64);
            a.z += __shfl_xor(a.z, d, 64);
            a.w += __shfl_xor(a.w, d, 64);
        }
        __syncthreads();
        if (lane < cols) sums[w][lane] = a;
        __syncthreads();
        if ((int)threadIdx.x < cols) {
            float4 t = sums[0][lane];
            for (int k = 1; k < 4; ++k) {
                t.x += sums[k][lane].x;
                t.y += sums[k][lane].y;
                t.z += sums[k][lane].z;
                t.w += sums[k][lane].w;
            }
            store(t, key[i]);
        }
    }
}

// ---------------------------------------------------------------------------
// Layer norm
// ---------------------------------------------------------------------------

// A parameter's value c as float: type 0 float, 1 bf16, 2 f16.
__device__ inline float param(const void* p, int type, int64_t c)
{
    return type == 0 ? ((const float*)p)[c] : type == 1 ? (float)((const __bf16*)p)[c] : (float)((const _Float16*)p)[c];
}

__device__ inline void set_param(void* p, int type, int64_t c, float v)
{
    if (type == 0) ((float*)p)[c] = v;
    else if (type == 1) ((__bf16*)p)[c] = (__bf16)v;
    else ((_Float16*)p)[c] = (_Float16)v;
}

__device__ inline float wave_sum(float x) { return group_sum(x, 6); }

__device__ inline float block_sum(float x, float* tmp)   // 256 threads; tmp: four floats
{
    x = wave_sum(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = x;
    __syncthreads();
    return tmp[0] + tmp[1] + (tmp[2] + tmp[3]);
}

// The columns of a row that a lane holds: K runs of V values, c(k) =
// (k * span + lane) * V, where `span` lanes share the row: a part of a wave, a
// wave (WPR = 1), or WPR waves, which are the whole block then.  With more than
// 8 values a lane a row is longer than half of its columns (plan_norm), so that
// only the upper half of the runs can pass its end.  TAIL says how a row ends:
// with a vector (kEven), inside one, which is moved back then so that it ends
// with the row and shares values with the one before (kBack: both compute the
// same, and the sums over the row leave the shared values of the last one out),
// or it is shorter than a vector (kPart).
constexpr int kEven = 0, kBack = 1, kPart = 2;

template <typename T, int NV, int WPR>
struct NormShape {
    static constexpr int V = kVals<T>, K = NV / V, kThreads = norm_threads(WPR);
    static constexpr int kFull = NV > 8 ? K / 2 : 0;   // runs that lie in every row
    static_assert(NV % V == 0, "whole vectors");
};

// Run k of a lane: how many values from its column on lie in the row (any
// positive number where TAIL is not kPart), its first column, and the first of
// its values that counts in sums over the row.
template <typename S, int TAIL>
struct NormRun {
    int left, c, own;
    __device__ NormRun(int k, int span, int lane, int dim)
    {
        const int at = (k * span + lane) * S::V;
        const bool full = k < S::kFull;
        left = full ? S::V : dim - at;
        c = TAIL == kBack && !full ? min(at, dim - S::V) : at;
        own = at - c;
    }
    // value i counts
    __device__ bool counts(int i) const { return TAIL == kPart ? i < left : left > 0 && (TAIL == kEven || i >= own); }
};

// The row of a lane's span: the same for the whole wave unless several rows
// share one (8 values a lane), and known to be, so that it stays in scalar
// registers and the loads take a scalar base.
template <int NV>
__device__ inline int64_t norm_row(int64_t first, int span_index)
{
    return first + (NV > 8 ? __builtin_amdgcn_readfirstlane(span_index) : span_index);
}

// v, as a value of which the compiler knows nothing: what was computed from
// it before does not stay in registers.
template <typename R>
__device__ inline R anew(R v)
{
    typedef uint32_t Words __attribute__((ext_vector_type(sizeof(R) / 4)));
    Words u = __builtin_bit_cast(Words, v);
    asm volatile("" : "+v"(u));
    return __builtin_bit_cast(R, u);
}

// Sums of N values over the lanes that share a row; every lane gets them.
// `tmp` ([2][N][WPR] floats) is used by turns, so that one barrier a sum is
// enough.
template <int N, int WPR>
__device__ inline void row_sums(float (&x)[N], int log_group, float* tmp, int& turn)
{
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = group_sum(x[i], log_group);
    if (WPR > 1) {
        float* t = tmp + turn * N * WPR;
        turn ^= 1;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) t[i * WPR + (threadIdx.x >> 6)] = x[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = 0.0f;
#pragma unroll
            for (int k = 0; k < WPR; ++k) x[i] += t[i * WPR + k];
        }
    }
}

// V values of a parameter from column c on; `other` where there is none.
template <int V, bool WHOLE>
__device__ inline void load_param(float (&r)[V], const void* p, int type, int64_t c, int64_t left, float other)
{
    if (!p || left <= 0) {
#pragma unroll
        for (int k = 0; k < V; ++k) r[k] = other;
    } else if (type == 0) {
        load_vals<V, WHOLE>(r, (const float*)p + c, left);
    } else if (type == 1) {
        load_vals<V, WHOLE>(r, (const __bf16*)p + c, left);
    } else {
        load_vals<V, WHOLE>(r, (const _Float16*)p + c, left);
    }
}

// V values of a parameter's gradient.
template <int V, bool WHOLE>
__device__ inline void store_param(const float (&r)[V], void* p, int type, int64_t c, int64_t left)
{
    if (!p) return;
    if (type == 0) store_vals<V, WHOLE>(r, (float*)p + c, left);
    else if (type == 1) store_vals<V, WHOLE>(r, (__bf16*)p + c, left);
    else store_vals<V, WHOLE>(r, (_Float16*)p + c, left);
}

// mean = sum x / dim, rstd = 1 / sqrt(sum (x - mean)^2 / dim + eps), y = (x -
// mean) rstd weight + bias.  Bound by bytes: the row stays in registers between
// its three uses, so x is read once, and the parameters stay there from row to
// row.  A wave takes a row of up to 2,048 values: its sums need no barrier.
// 32,768 rows of 1,792 bf16 values: 44 us, 5.3 TB/s (a large copy: 4.9); a
// block a row that read the row three times took 235 us.
template <typename T, int NV, int WPR, int TAIL>
__global__ __launch_bounds__(norm_threads(WPR)) void k_norm(
    const T* __restrict__ x, int64_t x_stride, int64_t rows, int dim, const void* __restrict__ weight,
    const void* __restrict__ bias, int wtype, float eps, T* __restrict__ y, int64_t y_stride, float* __restrict__ mean,
    float* __restrict__ rstd, int log_group, bool stream)
{
    using S = NormShape<T, NV, WPR>;
    constexpr int V = S::V, K = S::K;
    constexpr bool WHOLE = TAIL != kPart;
    __shared__ float tmp[2 * WPR];
    int turn = 0;
    if (NV > 8) log_group = 6;   // known to the compiler: the columns are fixed offsets then
    const int span = WPR > 1 ? S::kThreads : 1 << log_group, lane = threadIdx.x & (span - 1);
    const int per = S::kThreads / span;   // rows a block takes at a time
    float w[K][V], b[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const NormRun<S, TAIL> run(k, span, lane, dim);
        load_param<V, WHOLE>(w[k], weight, wtype, run.c, run.left, 1.0f);
        load_param<V, WHOLE>(b[k], bias, wtype, run.c, run.left, 0.0f);
    }
    for (int64_t r = norm_row<NV>((int64_t)blockIdx.x * per, threadIdx.x / span); r < rows; r += (int64_t)gridDim.x * per) {
        const T* p = x + r * x_stride;
        float v[K][V], s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const NormRun<S, TAIL> run(k, span, lane, dim);
            load_vals<V, WHOLE>(v[k], p + run.c, run.left);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const NormRun<S, TAIL> run(k, span, lane, dim);
#pragma unroll
            for (int i = 0; i < V; ++i) s[0] += TAIL != kBack || k < S::kFull || run.counts(i) ? v[k][i] : 0.0f;
        }
        row_sums<1, WPR>(s, log_group, tmp, turn);
        const float m = s[0] / (float)dim;
        s[0] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const NormRun<S, TAIL> run(k, span, lane, dim);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[k][i] -= m;
                if (k < S::kFull || run.counts(i)) s[0] = fmaf(v[k][i], v[k][i], s[0]);
            }
        }
        row_sums<1, WPR>(s, log_group, tmp, turn);
        const float q = 1.0f / sqrtf(s[0] / (float)dim + eps);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const NormRun<S, TAIL> run(k, span, lane, dim);
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] = fmaf(v[k][i] * q, w[k][i], b[k][i]);
            store_vals<V, WHOLE>(v[k], y + r * y_stride + run.c, run.left, stream);
        }
        if (lane == 0) {
            mean[r] = m;
            rstd[r] = q;
        }
    }
}

// dx by rows, and the parameters' gradients over the block's rows in the same
// pass: a lane keeps the sums of its columns in registers, the block's waves
// join theirs through LDS at the end (a fixed tree), and part
// [blocks][2][dim] holds the blocks' sums for k_norm_join.  A block alone stores
// the gradients itself.  Bound by bytes,
// each read and written once.  32,768 rows of 1,792 bf16 values: 74 us, 4.8
// TB/s, and 5 us for k_norm_join.  On the way: 298 us as passes of their own
// for dx and for the sums, 120 in one pass, 94 with the next row ahead but both
// forms of a row in registers, 78 with one form and two waves on a SIMD.
template <typename T, int NV, int WPR, int TAIL>
__global__ __launch_bounds__(norm_grad_threads(NV, WPR)) void k_norm_grad(
    const T* __restrict__ grad, int64_t grad_stride, const T* __restrict__ x, int64_t x_stride, int64_t rows, int dim,
    const float* __restrict__ mean, const float* __restrict__ rstd, const void* __restrict__ weight, int wtype,
    T* __restrict__ dx, int64_t dx_stride, float* __restrict__ part, void* __restrict__ dweight, void* __restrict__ dbias,
    int log_group, bool stream)
{
    using S = NormShape<T, NV, WPR>;
    constexpr int V = S::V, K = S::K, THREADS = norm_grad_threads(NV, WPR), WAVES = THREADS / 64;
    // with 32 values a lane the weights are in LDS: a third wave on a SIMD is
    // worth more than their registers
    constexpr bool FAR = NV == 32, WHOLE = TAIL != kPart;
    __shared__ float tmp[2 * 2 * WPR];
    __shared__ float sums[WPR > 1 ? 1 : WAVES / 2][WPR > 1 ? 1 : 64 * NV];
    __shared__ __align__(16) float far[FAR ? 64 * WPR * NV : 1];
    int turn = 0;
    if (NV > 8) log_group = 6;
    const int span = WPR > 1 ? THREADS : 1 << log_group, lane = threadIdx.x & (span - 1);
    const int per = THREADS / span;
    float w[K][V], dw[K][V], db[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const NormRun<S, TAIL> run(k, span, lane, dim);
        if (!FAR || (int)threadIdx.x < span) load_param<V, WHOLE>(w[k], weight, wtype, run.c, run.left, 1.0f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (FAR && (int)threadIdx.x < span) far[(k * span + lane) * V + i] = w[k][i];
            dw[k][i] = db[k][i] = 0.0f;
        }
    }
    if (FAR) __syncthreads();
    auto weights = [&](float (&v)[V], int k) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = FAR ? far[(k * span + lane) * V + i] : w[k][i];
    };
    // The next row is on its way while a row is summed: with three waves on a
    // SIMD (the sums take the registers) nothing else hides its latency.  A row
    // is held as it was loaded and converted twice, for the same reason.  Where
    // the registers do not reach for that (32 values of 32 bits; the 128 a lane
    // of a block of 16 waves), rows come one at a time, to more waves.
    constexpr bool AHEAD = WPR < 16 && (sizeof(T) < 4 || NV < 32);
    using Raw = typename Vals<T, V>::type;
    Raw next_g[K], next_x[K];
    float next_m, next_q;
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const NormRun<S, TAIL> run(k, span, lane, dim);
            next_g[k] = load_raw<V, WHOLE>(grad + r * grad_stride + run.c, run.left);
            next_x[k] = load_raw<V, WHOLE>(x + r * x_stride + run.c, run.left);
        }
        next_m = mean[r];
        next_q = rstd[r];
    };
    const int64_t step = (int64_t)gridDim.x * per;
    int64_t r = norm_row<NV>((int64_t)blockIdx.x * per, threadIdx.x / span);
    if (AHEAD && r < rows) fetch(r);
    for (; r < rows; r += step) {
        if (!AHEAD) fetch(r);
        Raw g[K], p[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            g[k] = next_g[k];
            p[k] = next_x[k];
        }
        const float m = next_m, q = next_q;
        if (AHEAD && r + step < rows) fetch(r + step);
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const NormRun<S, TAIL> run(k, span, lane, dim);
            float wk[V];
            weights(wk, k);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float h = ((float)p[k][i] - m) * q;
                // past the row's end g is 0, and h too: not a mean or rstd that may be infinite
                if (k >= S::kFull && !(TAIL == kBack ? run.left > 0 : run.counts(i))) h = 0.0f;
                const float u = (float)g[k][i], v = TAIL != kBack || k < S::kFull || i >= run.own ? u * wk[i] : 0.0f;
                dw[k][i] = fmaf(u, h, dw[k][i]);
                db[k][i] += u;
                s[0] += v;
                s[1] = fmaf(v, h, s[1]);
                // added here and now: put off to the loop's end, which the compiler
                // does, u and h of the whole row stay in registers
                asm volatile("" : "+v"(dw[k][i]), "+v"(db[k][i]));
            }
        }
        row_sums<2, WPR>(s, log_group, tmp, turn);
        const float a = s[0] / (float)dim, b = s[1] / (float)dim;
        if (sizeof(T) < 4) {
            // the row's values are converted anew from here on
#pragma unroll
            for (int k = 0; k < K; ++k) {
                g[k] = anew(g[k]);
                p[k] = anew(p[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const NormRun<S, TAIL> run(k, span, lane, dim);
            float v[V];
            weights(v, k);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = q * fmaf(((float)p[k][i] - m) * q, -b, (float)g[k][i] * v[i] - a);
            store_vals<V, WHOLE>(v, dx + r * dx_stride + run.c, run.left, stream);
        }
    }
    if (!part) return;
    if (WPR == 1) {
        const int wave = threadIdx.x >> 6, l = threadIdx.x & 63;
        for (int d = span; d < 64; d *= 2)
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    dw[k][i] += __shfl_xor(dw[k][i], d, 64);
                    db[k][i] += __shfl_xor(db[k][i], d, 64);
                }
        // waves [half, waves) add theirs to the first waves - half
        auto join = [&](float (&v)[K][V], int waves, int half) {
            if (wave >= half && wave < waves)
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int i = 0; i < V; ++i) sums[wave - half][(k * V + i) * 64 + l] = v[k][i];
            __syncthreads();
            if (wave < waves - half)
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int i = 0; i < V; ++i) v[k][i] += sums[wave][(k * V + i) * 64 + l];
            __syncthreads();
        };
#pragma unroll
        for (int waves = WAVES; waves > 1; waves = (waves + 1) / 2) {
            join(dw, waves, (waves + 1) / 2);
            join(db, waves, (waves + 1) / 2);
        }
        if ((int)threadIdx.x >= span) return;
    }
    float* to = part + (int64_t)blockIdx.x * 2 * dim;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const NormRun<S, TAIL> run(k, span, lane, dim);
        if (gridDim.x == 1) {
            store_param<V, WHOLE>(dw[k], dweight, wtype, run.c, run.left);
            store_param<V, WHOLE>(db[k], dbias, wtype, run.c, run.left);
            continue;
        }
        store_vals<V, WHOLE>(dw[k], to + run.c, run.left);
        store_vals<V, WHOLE>(db[k], to + dim + run.c, run.left);
    }
}

// Rows that registers do not hold (dim above kNormMaxDim): one row a block,
// read again for each of its sums (from the cache).
template <typename T>
__global__ __launch_bounds__(256) void k_norm_wide(const T* __restrict__ x, int64_t x_stride, int64_t rows, int64_t dim,
                                                   const void* __restrict__ weight, const void* __restrict__ bias,
                                                   int wtype, float eps, T* __restrict__ y, int64_t y_stride,
                                                   float* __restrict__ mean, float* __restrict__ rstd)
{
    __shared__ float tmp[4];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T* p = x + r * x_stride;
        float s = 0.0f;
        for (int64_t c = threadIdx.x; c < dim; c += 256) s += (float)p[c];
        const float m = block_sum(s, tmp) / (float)dim;
        s = 0.0f;
        for (int64_t c = threadIdx.x; c < dim; c += 256) {
            const float d = (float)p[c] - m;
            s = fmaf(d, d, s);
        }
        const float q = 1.0f / sqrtf(block_sum(s, tmp) / (float)dim + eps);
        for (int64_t c = threadIdx.x; c < dim; c += 256) {
            float v = ((float)p[c] - m) * q;
            if (weight) v *= param(weight, wtype, c);
            if (bias) v += param(bias, wtype, c);
            y[r * y_stride + c] = (T)v;
        }
        if (threadIdx.x == 0) {
            mean[r] = m;
            rstd[r] = q;
        }
    }
}

template <typename T>
__global__ __launch_bounds__(256) void k_norm_wide_dx(const T* __restrict__ grad, int64_t grad_stride,
                                                      const T* __restrict__ x, int64_t x_stride, int64_t rows,
                                                      int64_t dim, const float* __restrict__ mean,
                                                      const float* __restrict__ rstd, const void* __restrict__ weight,
                                                      int wtype, T* __restrict__ dx, int64_t dx_stride)
{
    __shared__ float tmp[4];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T* g = grad + r * grad_stride;
        const T* p = x + r * x_stride;
        const float m = mean[r], q = rstd[r];
        float a = 0.0f, b = 0.0f;
        for (int64_t c = threadIdx.x; c < dim; c += 256) {
            const float v = (float)g[c] * (weight ? param(weight, wtype, c) : 1.0f);
            a += v;
            b = fmaf(v, ((float)p[c] - m) * q, b);
        }
        a = block_sum(a, tmp) / (float)dim;
        b = block_sum(b, tmp) / (float)dim;
        for (int64_t c = threadIdx.x; c < dim; c += 256) {
            const float v = (float)g[c] * (weight ? param(weight, wtype, c) : 1.0f);
            dx[r * dx_stride + c] = (T)(q * (v - a - ((float)p[c] - m) * q * b));
        }
    }
}

// Partial sums of the parameters' gradients over one share of the rows: part
// [parts][2][dim].
template <typename T>
__global__ __launch_bounds__(256) void k_norm_wide_params(const T* __restrict__ grad, int64_t grad_stride,
                                                          const T* __restrict__ x, int64_t x_stride, int64_t rows,
                                                          int64_t dim, const float* __restrict__ mean,
                                                          const float* __restrict__ rstd, float* __restrict__ part)
{
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= dim) return;
    float w = 0.0f, b = 0.0f;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const float g = (float)grad[r * grad_stride + c];
        w = fmaf(g, ((float)x[r * x_stride + c] - mean[r]) * rstd[r], w);
        b += g;
    }
    part[((int64_t)blockIdx.y * 2) * dim + c] = w;
    part[((int64_t)blockIdx.y * 2 + 1) * dim + c] = b;
}

// The parameters' gradients from the blocks' sums: 16 columns a block, 16
// threads a column, each over every 16th part, joined by a fixed tree.
__global__ __launch_bounds__(256) void k_norm_join(const float* __restrict__ part, int parts, int64_t dim,
                                                   void* __restrict__ dweight, void* __restrict__ dbias, int wtype)
{
    __shared__ float sums[16][17];
    const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
    const int64_t c = (int64_t)blockIdx.x * 16 + col;
    void* out = blockIdx.y == 0 ? dweight : dbias;
    if (!out) return;
    float s = 0.0f;
    if (c < dim) {
#pragma unroll 8
        for (int k = row; k < parts; k += 16) s += part[((int64_t)k * 2 + blockIdx.y) * dim + c];
    }
    sums[row][col] = s;
    __syncthreads();
    for (int half = 8; half > 0; half /= 2) {
        if (row < half) sums[row][col] += sums[row + half][col];
        __syncthreads();
    }
    if (row == 0 && c < dim) set_param(out, wtype, c, sums[0][col]);
}

// ---------------------------------------------------------------------------
// Rows sorted by expert, and back
// ---------------------------------------------------------------------------

// Rows to their slots' places, a vector a thread.  It also zeroes the places of
// its number range that lie past the last routed slot.  Bound by bytes: 32,768
// rows of 1,024 bf16 values, four places each, in 51 us, 6.5 TB/s.
template <typename T>
__global__ __launch_bounds__(256) void k_route_gather(const T* __restrict__ x, int64_t x_stride, int64_t rows, int top,
                                                      int dim, const int32_t* __restrict__ position,
                                                      const int32_t* __restrict__ routed, T* __restrict__ out,
                                                      int64_t out_stride, RowMap m, bool stream)
{
    constexpr int V = kVals<T>;
    const RowPlace p = row_place<V>(m, (uint32_t)rows, dim);
    if (!p.in) return;
    const int64_t slots = rows * top, used = *routed, first = (int64_t)p.r * top;
    auto copy = [&](auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        const typename Vals<T, V>::type v = load_raw<V, WHOLE>(x + p.r * x_stride + p.c, dim);
        for (int k = 0; k < top; ++k) {
            const int64_t at = position[first + k];
            if (at >= 0 && at < slots) store_raw<V, WHOLE>(v, out + at * out_stride + p.c, dim, stream);
            if (first + k >= used)
                store_raw<V, WHOLE>(typename Vals<T, V>::type{}, out + (first + k) * out_stride + p.c, dim, stream);
        }
    };
    if (dim >= V) copy(std::true_type());
    else copy(std::false_type());
}

// out[r] = sum over k of weight[r][k] * y[position[r][k]], in the order of k,
// a vector a thread, four rows of y in flight.  Bound by bytes: 32,768 rows of
// 1,024 bf16 values, four each, in 55 us, 6.1 TB/s (y through the caches: 59).
template <typename T>
__global__ __launch_bounds__(256) void k_route_combine(const T* __restrict__ y, int64_t y_stride, int64_t rows, int top,
                                                       int dim, const int32_t* __restrict__ position,
                                                       const float* __restrict__ weight, T* __restrict__ out,
                                                       int64_t out_stride, RowMap m, bool stream)
{
    constexpr int V = kVals<T>, STEP = 4;
    const RowPlace p = row_place<V>(m, (uint32_t)rows, dim);
    if (!p.in) return;
    const int64_t slots = rows * top, first = (int64_t)p.r * top;
    auto sum = [&](auto whole, auto past) {
        constexpr bool WHOLE = decltype(whole)::value, STREAM = decltype(past)::value;
        float acc[V];
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = 0.0f;
        for (int k = 0; k < top; k += STEP) {
            typename Vals<T, V>::type v[STEP];
            float w[STEP];
#pragma unroll
            for (int u = 0; u < STEP; ++u) {
                const int64_t at = k + u < top ? position[first + k + u] : -1;
                const bool live = at >= 0 && at < slots;
                w[u] = live && weight ? weight[first + k + u] : live;
                v[u] = live ? load_raw<V, WHOLE, STREAM>(y + at * y_stride + p.c, dim) : typename Vals<T, V>::type{};
            }
#pragma unroll
            for (int u = 0; u < STEP; ++u)
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = fmaf(w[u], (float)v[u][i], acc[i]);
        }
        store_vals<V, WHOLE>(acc, out + p.r * out_stride + p.c, dim, STREAM);
    };
    if (dim < V) sum(std::false_type(), std::false_type());
    else if (stream) sum(std::true_type(), std::true_type());
    else sum(std::true_type(), std::false_type());
}

// dy[position[r][k]] = weight[r][k] * grad[r]; dweight[r][k] = <grad[r], y[position[r][k]]>.
// A wave takes a slot, or several where a row has few vectors (WAVE false), four
// vectors of each row in flight; a row's slots are neighbours, so that its
// gradient comes from the cache after the first.  Places past the last routed
// slot are zeroed as in k_route_gather.  Bound by bytes: 32,768 rows of 1,024
// bf16 values, four slots each, in 94 us, 6.4 TB/s (y through the caches 106, and
// a wave a row 116; 7 and 45 for 186 rows of 3,304 values, six slots each).
template <typename T, bool WAVE>
__global__ __launch_bounds__(256) void k_route_combine_grad(const T* __restrict__ grad, int64_t grad_stride,
                                                            const T* __restrict__ y, int64_t y_stride, int64_t rows,
                                                            int top, int dim, const int32_t* __restrict__ position,
                                                            const int32_t* __restrict__ routed,
                                                            const float* __restrict__ weight, T* __restrict__ dy,
                                                            int64_t dy_stride, float* __restrict__ dweight, int log_group,
                                                            bool stream)
{
    constexpr int V = kVals<T>, STEP = WAVE ? 4 : 1;
    if (WAVE) log_group = 6;
    const int lane = threadIdx.x & ((1 << log_group) - 1), group = threadIdx.x >> log_group;
    const uint32_t slots = (uint32_t)(rows * top);
    const uint32_t s = block_number() * (256u >> log_group) + (WAVE ? __builtin_amdgcn_readfirstlane(group) : group);
    if (s >= slots) return;
    const uint32_t r = s / (uint32_t)top, used = (uint32_t)*routed, at = (uint32_t)position[s];
    const bool live = at < slots;   // -1 is not
    const float w = weight ? weight[s] : 1.0f;
    const T* g_row = grad + (int64_t)r * grad_stride;
    const T* y_row = y + (live ? (int64_t)at : 0) * y_stride;
    T* to = dy + (live ? (int64_t)at : 0) * dy_stride;
    T* zero = dy + (int64_t)s * dy_stride;
    typedef typename Vals<T, V>::type Vec;
    float dot = 0.0f;
    auto slot = [&](auto whole, auto past) {
        constexpr bool WHOLE = decltype(whole)::value, STREAM = decltype(past)::value;
        for (int first = lane * V; first < dim; first += (STEP * V) << log_group) {
            Vec g[STEP], v[STEP];
            int c[STEP];
#pragma unroll
            for (int u = 0; u < STEP; ++u) {
                const int from = first + ((u * V) << log_group);
                c[u] = WHOLE ? min(from, dim - V) : from;
                g[u] = load_raw<V, WHOLE>(g_row + c[u], live ? dim - from : 0);
                v[u] = load_raw<V, WHOLE, STREAM>(y_row + c[u], live && dweight ? dim - from : 0);
            }
#pragma unroll
            for (int u = 0; u < STEP; ++u) {
                const int from = first + ((u * V) << log_group);
                float out[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    // values shared with the vector before count there
                    if (c[u] + i >= from) dot = fmaf((float)g[u][i], (float)v[u][i], dot);
                    out[i] = (float)g[u][i] * w;
                }
                if (live) store_vals<V, WHOLE>(out, to + c[u], dim - from, STREAM);
                if (s >= used) store_raw<V, WHOLE>(Vec{}, zero + c[u], dim - from, STREAM);
            }
        }
    };
    if (dim < V) slot(std::false_type(), std::false_type());
    else if (stream) slot(std::true_type(), std::true_type());
    else slot(std::true_type(), std::false_type());
    if (dweight) {
        dot = group_sum(dot, log_group);
        if (lane == 0) dweight[s] = dot;
    }
}

}  // namespace hgb
