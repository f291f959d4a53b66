// Device kernels of the vector verbs (gfx950).  Internal header: included by
// hgb_vectors.hip only.
//
// Rows are vectors of `dim` values of T (float, __bf16, _Float16); sums and
// statistics are 32-bit floats, rounded once when they are stored.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

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

template <int V, typename T>
__device__ inline void load_vals(float (&r)[V], const T* p, int64_t left)
{
    if (left >= V) {
        const typename Vals<T, V>::type v = *(const typename Vals<T, V>::type*)p;
#pragma unroll
        for (int k = 0; k < V; ++k) r[k] = (float)v[k];
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) r[k] = k < left ? (float)p[k] : 0.0f;
    }
}

template <int V, typename T>
__device__ inline void store_vals(const float (&r)[V], T* p, int64_t left)
{
    if (left >= V) {
        typename Vals<T, V>::type v;
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = (T)r[k];
        *(typename Vals<T, V>::type*)p = v;
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k < left) p[k] = (T)r[k];
    }
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
template <int ITEMS>
__device__ inline void tile_ranks(const uint32_t (&digit)[ITEMS], int live, int bits, int radix, uint32_t* count,
                                  uint32_t* total, uint32_t (&rank)[ITEMS])
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, waves = blockDim.x >> 6;
    for (int i = threadIdx.x; i < waves * radix; i += blockDim.x) count[i] = 0;
    __syncthreads();
    uint32_t* mine = count + w * radix;
    const uint64_t below = (1ull << lane) - 1;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int at = w * 64 * ITEMS + i * 64 + lane;
        const bool in = at < live;
        uint64_t same = __ballot(in);
        for (int b = 0; b < bits; ++b) {
            const bool one = (digit[i] >> b) & 1;
            const uint64_t m = __ballot(one);
            same &= one ? m : ~m;
        }
        const int before = __popcll(same & below);
        if (in) rank[i] = mine[digit[i]] + before;
        wave_order();
        if (in && before == 0) mine[digit[i]] = rank[i] + __popcll(same);
        wave_order();
    }
    __syncthreads();
    for (int d = threadIdx.x; d < radix; d += blockDim.x) {
        uint32_t sum = 0;
        for (int k = 0; k < waves; ++k) {
            const uint32_t c = count[k * radix + d];
            count[k * radix + d] = sum;
            sum += c;
        }
        total[d] = sum;
    }
    __syncthreads();
}

// Exclusive sums of v[0, radix) in place, radix <= the block's threads;
// `tmp` holds a word per wave.
__device__ inline void block_scan(uint32_t* v, int radix, uint32_t* tmp)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, waves = blockDim.x >> 6;
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
};

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

__device__ inline void zero_row(char* p, int64_t bytes, int64_t first, int64_t step)
{
    const int64_t whole = bytes / 16;
    for (int64_t i = first; i < whole; i += step) *(u32x4_any*)(p + 16 * i) = u32x4_any{0, 0, 0, 0};
    for (int64_t i = whole * 8 + first; i < bytes / 2; i += step) ((uint16_t*)p)[i] = 0;
}

__device__ inline void zero_fill(const ZeroFill& z, int block, int blocks)
{
    if (z.stride == z.cols) {
        zero_row((char*)z.out, z.rows * z.cols * z.elem, (int64_t)block * blockDim.x + threadIdx.x,
                 (int64_t)blocks * blockDim.x);
        return;
    }
    for (int64_t r = block; r < z.rows; r += blocks)
        zero_row((char*)z.out + r * z.stride * z.elem, z.cols * z.elem, threadIdx.x, blockDim.x);
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

// counts[block][digit] of one pass; blocks past p.blocks write the zeros.
template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void k_sort_count(SortIn in, SortPlan p, int shift, uint32_t* counts,
                                                             ZeroFill z)
{
    if ((int)blockIdx.x >= p.blocks) {
        zero_fill(z, blockIdx.x - p.blocks, gridDim.x - p.blocks);
        return;
    }
    extern __shared__ uint32_t lds[];
    for (int d = threadIdx.x; d < p.radix; d += blockDim.x) lds[d] = 0;
    __syncthreads();
    const int64_t begin = (int64_t)blockIdx.x * p.tiles * kSortTile;
    const int64_t end = begin + (int64_t)p.tiles * kSortTile < in.n ? begin + (int64_t)p.tiles * kSortTile : in.n;
    bool bad = false;
    for (int64_t i = begin + threadIdx.x; i < end; i += blockDim.x)
        atomicAdd(&lds[(sort_load<FIRST>(in, i, &bad).x >> shift) & (p.radix - 1)], 1u);
    if (bad) atomicOr(in.err, in.flag);
    __syncthreads();
    for (int d = threadIdx.x; d < p.radix; d += blockDim.x) counts[(int64_t)blockIdx.x * p.radix + d] = lds[d];
}

// The pass's scatter: each block sums the counts before it (there are at most
// kSortMaxBlocks rows of them, read from L2) instead of a scan in a launch of
// its own, then ranks its tiles in order.
template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void k_sort_scatter(SortIn in, SortOut out, SortPlan p, int shift,
                                                               const uint32_t* counts)
{
    extern __shared__ uint32_t lds[];
    const int waves = blockDim.x >> 6;
    uint32_t* count = lds;                        // [waves][radix]
    uint32_t* total = count + waves * p.radix;    // [radix]
    uint32_t* base = total + p.radix;             // [radix]
    uint32_t* tmp = base + p.radix;               // [waves]
    // base[d] = keys of smaller digits + keys of digit d in earlier blocks
    {
        const int d = threadIdx.x & (p.radix - 1), g = threadIdx.x / p.radix, groups = blockDim.x / p.radix;
        uint32_t all = 0, before = 0;
        for (int b = g; b < p.blocks; b += groups) {
            const uint32_t c = counts[(int64_t)b * p.radix + d];
            all += c;
            if (b < (int)blockIdx.x) before += c;
        }
        if (g == 0) total[d] = base[d] = 0;
        __syncthreads();
        atomicAdd(&total[d], all);
        atomicAdd(&base[d], before);
        __syncthreads();
        block_scan(total, p.radix, tmp);
        if (out.offsets && blockIdx.x == 0)
            for (int k = threadIdx.x; k <= in.limit; k += blockDim.x) out.offsets[k] = (int32_t)total[k];
        if (g == 0) base[d] += total[d];
        __syncthreads();
    }
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, first = w * 64 * kSortItems + lane;
    for (int t = 0; t < p.tiles; ++t) {
        const int64_t begin = ((int64_t)blockIdx.x * p.tiles + t) * kSortTile;
        if (begin >= in.n) break;
        const int live = in.n - begin < kSortTile ? (int)(in.n - begin) : kSortTile;
        uint2 kv[kSortItems];
        uint32_t digit[kSortItems], rank[kSortItems];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            kv[i] = make_uint2(0, 0);
            if (first + i * 64 < live) kv[i] = sort_load<FIRST>(in, begin + first + i * 64, &bad);
            digit[i] = (kv[i].x >> shift) & (p.radix - 1);
        }
        tile_ranks<kSortItems>(digit, live, p.bits, p.radix, count, total, rank);
#pragma unroll
        for (int i = 0; i < kSortItems; ++i)
            if (first + i * 64 < live) {
                const int64_t at = base[digit[i]] + count[w * p.radix + digit[i]] + rank[i];
                if (out.to) {
                    out.to[at] = kv[i];
                } else {
                    const bool keep = kv[i].x < (uint32_t)in.limit;
                    out.order[at] = keep ? (int32_t)kv[i].y : -1;
                    out.position[kv[i].y] = keep ? (int32_t)at : -1;
                }
            }
        __syncthreads();
        if ((int)threadIdx.x < p.radix) base[threadIdx.x] += total[threadIdx.x];
    }
}

// ---------------------------------------------------------------------------
// Embedding
// ---------------------------------------------------------------------------

// out[i] = scale * table[token i]; a group of lanes takes ROWS tokens.
template <typename T, typename U, int ROWS>
__global__ __launch_bounds__(256) void k_embed(const T* __restrict__ table, int64_t table_stride, int64_t vocab,
                                               int64_t dim, const int32_t* __restrict__ tokens, int64_t n, int32_t pad,
                                               float scale, U* __restrict__ out, int64_t out_stride, int log_group,
                                               uint32_t* err)
{
    constexpr int V = kVals<T, U>;
    const int groups = 256 >> log_group, g = threadIdx.x >> log_group, lane = threadIdx.x & ((1 << log_group) - 1);
    const int64_t first = (int64_t)blockIdx.x * groups * ROWS + g;
    int32_t t[ROWS];
    bool bad = false;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t i = first + (int64_t)r * groups;
        t[r] = i < n ? tokens[i] : pad;
        const bool live = t[r] != pad && t[r] >= 0 && t[r] < vocab;
        if (!live && t[r] != pad) bad = true;
        if (!live) t[r] = -1;
    }
    if (bad && lane == 0) atomicOr(err, kVecErrToken);
    for (int64_t c = (int64_t)lane * V; c < dim; c += (int64_t)V << log_group) {
        float v[ROWS][V];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (t[r] >= 0) {
                load_vals<V>(v[r], table + t[r] * table_stride + c, dim - c);
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k) v[r][k] = 0.0f;
            }
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int64_t i = first + (int64_t)r * groups;
#pragma unroll
            for (int k = 0; k < V; ++k) v[r][k] = t[r] >= 0 ? v[r][k] * scale : 0.0f;
            if (i < n) store_vals<V>(v[r], out + i * out_stride + c, dim - c);
        }
    }
}

__global__ __launch_bounds__(256) void k_zero_rows(ZeroFill z) { zero_fill(z, blockIdx.x, gridDim.x); }

// Sums of the gradient's rows over each run of equal keys.  A group of lanes
// walks one chunk of sorted positions; a run that lies in its chunk is
// finished there, and a run that crosses a border leaves its part in the
// chunk's partial rows: row 0 a run that began before the chunk, row 1 one
// that begins in it and goes on.
template <typename T, typename U>
__global__ __launch_bounds__(256) void k_embed_sum(const uint2* __restrict__ pairs, int64_t n, const T* __restrict__ grad,
                                                   int64_t grad_stride, int64_t dim, int64_t vocab, float scale,
                                                   U* __restrict__ out, int64_t out_stride, float* __restrict__ part,
                                                   int64_t part_stride, int chunk, int log_group)
{
    constexpr int V = kVals<T, U>, STEP = 8;
    const int lane = threadIdx.x & ((1 << log_group) - 1);
    const int64_t id = (int64_t)blockIdx.x * (256 >> log_group) + (threadIdx.x >> log_group);
    const int64_t c = ((int64_t)blockIdx.y << log_group) * V + (int64_t)lane * V;
    const int64_t begin = id * chunk, end = begin + chunk < n ? begin + chunk : n;
    if (begin >= n || c >= dim) return;
    const uint32_t none = 0xffffffffu;
    const uint32_t prev = begin > 0 ? pairs[begin - 1].x : none, next = end < n ? pairs[end].x : none;
    uint32_t cur = pairs[begin].x;
    bool head = cur == prev;
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.0f;
    auto flush = [&](bool open) {
        if (cur >= (uint32_t)vocab) return;
        if (head || open) {
            float* p = part + (id * 2 + (head ? 0 : 1)) * part_stride + c;
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (c + k < dim) p[k] = acc[k];
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] *= scale;
            store_vals<V>(acc, out + (int64_t)cur * out_stride + c, dim - c);
        }
    };
    for (int64_t j = begin; j < end; j += STEP) {
        uint2 kv[STEP];
        float v[STEP][V];
#pragma unroll
        for (int u = 0; u < STEP; ++u) kv[u] = pairs[j + u < end ? j + u : end - 1];
#pragma unroll
        for (int u = 0; u < STEP; ++u)
            if (kv[u].x < (uint32_t)vocab) load_vals<V>(v[u], grad + (int64_t)kv[u].y * grad_stride + c, dim - c);
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
            if (cur < (uint32_t)vocab) {
#pragma unroll
                for (int k = 0; k < V; ++k) acc[k] += v[u][k];
            }
        }
    }
    flush(cur == next);
}

// Runs that cross chunk borders: the partial row of the chunk where the run
// begins plus row 0 of each chunk it goes on in.  A block takes kJoinChunks
// chunks and 64 columns: a wave sums a short run, the whole block a long one
// (16 rows at a time, joined in a fixed order).
constexpr int kJoinChunks = 16;
constexpr int kJoinLong = 32;

template <typename U>
__global__ __launch_bounds__(256) void k_embed_join(const uint2* __restrict__ pairs, int64_t n, int64_t dim, int64_t vocab,
                                                    float scale, U* __restrict__ out, int64_t out_stride,
                                                    const float* __restrict__ part, int64_t part_stride, int chunk,
                                                    int64_t chunks)
{
    __shared__ int64_t last[kJoinChunks];   // the run's last chunk; -1: no run to join here
    __shared__ uint32_t key[kJoinChunks];
    __shared__ float4 sums[4][16];
    const int64_t base = (int64_t)blockIdx.x * kJoinChunks;
    if (threadIdx.x < kJoinChunks) {
        const int64_t id = base + threadIdx.x;
        int64_t e = -1;
        uint32_t k = 0;
        if (id + 1 < chunks) {
            const int64_t begin = id * chunk, end = begin + chunk;
            k = pairs[end - 1].x;
            const bool open = pairs[end].x == k;
            const bool whole = pairs[begin].x == k && begin > 0 && pairs[begin - 1].x == k;
            if (open && !whole && k < (uint32_t)vocab) {
                // the last chunk that begins with the run: doubling, then halving
                int64_t lo = id + 1, step = 1;
                while (lo + step < chunks && pairs[(lo + step) * chunk].x == k) {
                    lo += step;
                    step *= 2;
                }
                for (; step > 0; step /= 2)
                    if (lo + step < chunks && pairs[(lo + step) * chunk].x == k) lo += step;
                e = lo;
            }
        }
        last[threadIdx.x] = e;
        key[threadIdx.x] = k;
    }
    __syncthreads();
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, row = lane >> 4;
    const int64_t c = (int64_t)blockIdx.y * 64 + (lane & 15) * 4;
    const bool in = c < dim;   // part rows are padded to four floats
    for (int s = 0; s < kJoinChunks; ++s) {
        const int64_t e = last[s], id = base + s;
        if (e < 0) continue;
        const bool whole_block = e - id > kJoinLong;
        if (!whole_block && (s & 3) != w) continue;
        const int rows = whole_block ? 16 : 4;
        float4 a = make_float4(0, 0, 0, 0);
        if (in)
            for (int64_t k = id + (whole_block ? w * 4 + row : row); k <= e; k += rows) {
                const float4 v = *(const float4*)(part + (k * 2 + (k == id ? 1 : 0)) * part_stride + c);
                a.x += v.x;
                a.y += v.y;
                a.z += v.z;
                a.w += v.w;
            }
#pragma unroll
        for (int d = 16; d < 64; d *= 2) {
            a.x += __shfl_xor(a.x, d, 64);
            a.y += __shfl_xor(a.y, d, 64);
            a.z += __shfl_xor(a.z, d, 64);
            a.w += __shfl_xor(a.w, d, 64);
        }
        if (whole_block) {
            __syncthreads();
            if (lane < 16) sums[w][lane] = a;
            __syncthreads();
            if (w != 0) continue;
            a = make_float4(0, 0, 0, 0);
            for (int k = 0; k < 4; ++k) {
                const float4 v = sums[k][lane & 15];
                a.x += v.x;
                a.y += v.y;
                a.z += v.z;
                a.w += v.w;
            }
        }
        if (lane < 16 && in) {
            const float r[4] = {a.x * scale, a.y * scale, a.z * scale, a.w * scale};
            store_vals<4>(r, out + (int64_t)key[s] * out_stride + c, dim - c);
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

__device__ inline float wave_sum(float x)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d, 64);
    return x;
}

__device__ inline float block_sum(float x, float* tmp)   // 256 threads; tmp: four floats
{
    x = wave_sum(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = x;
    __syncthreads();
    return tmp[0] + tmp[1] + (tmp[2] + tmp[3]);
}

// One row a block, read again for each of its three sums (from the cache).
template <typename T>
__global__ __launch_bounds__(256) void k_norm(const T* __restrict__ x, int64_t x_stride, int64_t rows, int64_t dim,
                                              const void* __restrict__ weight, const void* __restrict__ bias, int wtype,
                                              float eps, T* __restrict__ y, int64_t y_stride, float* __restrict__ mean,
                                              float* __restrict__ rstd)
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
__global__ __launch_bounds__(256) void k_norm_dx(const T* __restrict__ grad, int64_t grad_stride, const T* __restrict__ x,
                                                 int64_t x_stride, int64_t rows, int64_t dim,
                                                 const float* __restrict__ mean, const float* __restrict__ rstd,
                                                 const void* __restrict__ weight, int wtype, T* __restrict__ dx,
                                                 int64_t dx_stride)
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
__global__ __launch_bounds__(256) void k_norm_params(const T* __restrict__ grad, int64_t grad_stride,
                                                     const T* __restrict__ x, int64_t x_stride, int64_t rows, int64_t dim,
                                                     const float* __restrict__ mean, const float* __restrict__ rstd,
                                                     float* __restrict__ part)
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

__global__ __launch_bounds__(256) void k_norm_join(const float* __restrict__ part, int parts, int64_t dim,
                                                   void* __restrict__ dweight, void* __restrict__ dbias, int wtype)
{
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= dim) return;
    void* out = blockIdx.y == 0 ? dweight : dbias;
    if (!out) return;
    float s = 0.0f;
    for (int k = 0; k < parts; ++k) s += part[((int64_t)k * 2 + blockIdx.y) * dim + c];
    set_param(out, wtype, c, s);
}

// ---------------------------------------------------------------------------
// Rows sorted by expert, and back
// ---------------------------------------------------------------------------

// Rows to their slots' places; a group of lanes takes one row.  It also
// zeroes the places of its number range that lie past the last routed slot.
template <typename T>
__global__ __launch_bounds__(256) void k_route_gather(const T* __restrict__ x, int64_t x_stride, int64_t rows, int top,
                                                      int64_t dim, const int32_t* __restrict__ position,
                                                      const int32_t* __restrict__ routed, T* __restrict__ out,
                                                      int64_t out_stride, int log_group)
{
    constexpr int V = kVals<T>;
    const int lane = threadIdx.x & ((1 << log_group) - 1);
    const int64_t r = (int64_t)blockIdx.x * (256 >> log_group) + (threadIdx.x >> log_group);
    if (r >= rows) return;
    const int64_t slots = rows * top, used = *routed;
    for (int64_t c = (int64_t)lane * V; c < dim; c += (int64_t)V << log_group) {
        float v[V], zero[V];
        load_vals<V>(v, x + r * x_stride + c, dim - c);
#pragma unroll
        for (int k = 0; k < V; ++k) zero[k] = 0.0f;
        for (int k = 0; k < top; ++k) {
            const int64_t at = position[r * top + k];
            if (at >= 0 && at < slots) store_vals<V>(v, out + at * out_stride + c, dim - c);
            if (r * top + k >= used) store_vals<V>(zero, out + (r * top + k) * out_stride + c, dim - c);
        }
    }
}

// out[r] = sum over k of weight[r][k] * y[position[r][k]], in the order of k.
template <typename T>
__global__ __launch_bounds__(256) void k_route_combine(const T* __restrict__ y, int64_t y_stride, int64_t rows, int top,
                                                       int64_t dim, const int32_t* __restrict__ position,
                                                       const float* __restrict__ weight, T* __restrict__ out,
                                                       int64_t out_stride, int log_group)
{
    constexpr int V = kVals<T>;
    const int lane = threadIdx.x & ((1 << log_group) - 1);
    const int64_t r = (int64_t)blockIdx.x * (256 >> log_group) + (threadIdx.x >> log_group);
    if (r >= rows) return;
    const int64_t slots = rows * top;
    for (int64_t c = (int64_t)lane * V; c < dim; c += (int64_t)V << log_group) {
        float acc[V], v[V];
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = 0.0f;
        for (int k = 0; k < top; ++k) {
            const int64_t at = position[r * top + k];
            if (at < 0 || at >= slots) continue;
            const float w = weight ? weight[r * top + k] : 1.0f;
            load_vals<V>(v, y + at * y_stride + c, dim - c);
#pragma unroll
            for (int u = 0; u < V; ++u) acc[u] = fmaf(w, v[u], acc[u]);
        }
        store_vals<V>(acc, out + r * out_stride + c, dim - c);
    }
}

// dy[position[r][k]] = weight[r][k] * grad[r]; dweight[r][k] = <grad[r], y[position[r][k]]>.
// A wave takes one row; places past the last routed slot are zeroed as in
// k_route_gather.
template <typename T>
__global__ __launch_bounds__(256) void k_route_combine_grad(const T* __restrict__ grad, int64_t grad_stride,
                                                            const T* __restrict__ y, int64_t y_stride, int64_t rows,
                                                            int top, int64_t dim, const int32_t* __restrict__ position,
                                                            const int32_t* __restrict__ routed,
                                                            const float* __restrict__ weight, T* __restrict__ dy,
                                                            int64_t dy_stride, float* __restrict__ dweight)
{
    constexpr int V = kVals<T>;
    const int lane = threadIdx.x & 63;
    const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (r >= rows) return;
    const int64_t slots = rows * top, used = *routed;
    for (int k = 0; k < top; ++k) {
        const int64_t s = r * top + k, at = position[s];
        const bool live = at >= 0 && at < slots;
        const float w = weight ? weight[s] : 1.0f;
        float dot = 0.0f;
        if (live)
            for (int64_t c = lane * V; c < dim; c += 64 * V) {
                float g[V], v[V];
                load_vals<V>(g, grad + r * grad_stride + c, dim - c);
                if (dweight) {
                    load_vals<V>(v, y + at * y_stride + c, dim - c);
#pragma unroll
                    for (int u = 0; u < V; ++u) dot = fmaf(g[u], v[u], dot);
                }
#pragma unroll
                for (int u = 0; u < V; ++u) g[u] *= w;
                store_vals<V>(g, dy + at * dy_stride + c, dim - c);
            }
        if (dweight) {
            dot = wave_sum(dot);
            if (lane == 0) dweight[s] = dot;
        }
        if (s >= used)
            for (int64_t c = lane * V; c < dim; c += 64 * V) {
                float zero[V];
#pragma unroll
                for (int u = 0; u < V; ++u) zero[u] = 0.0f;
                store_vals<V>(zero, dy + s * dy_stride + c, dim - c);
            }
    }
}

}  // namespace hgb
