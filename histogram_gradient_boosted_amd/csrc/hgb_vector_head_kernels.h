// Device kernels of the head's losses: cross entropy and distillation over a
// vocabulary (gfx950).  Internal header: included by hgb_vector_head.hip only.
//
// All three large sums are products of two matrices,
//   z = x table^T          [rows][tokens], summed over the vectors' values
//   dx = dz table          [rows][values], summed over the tokens
//   dtable = dz^T x        [tokens][values], summed over the rows
// and one kernel makes them; what it does with its tile of the result differs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "hgb_ctx.h"
#include "hgb_vector_head_plan.h"
#include "hgb_vector_rows.h"

namespace hgb {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// A value that all lanes have, for the compiler to keep as one.
__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A factor of a product, rows of 16-byte chunks.  Along the rows ("by k"
// false): row m holds the values that are summed; by k: row k holds the value
// k of every m.
struct Factor {
    const void* p;
    int64_t stride;   // of a row, in values
    int64_t rows;
    int64_t cols;     // of the rows that may be read
    int64_t plane;    // values between planes
};

struct ProductArgs {
    Factor a, b;
    int m, n;            // C's size
    int k_steps;         // steps of a plane's sum
    int planes;          // of a; the sum runs over all of them with the same b
    int splits;
    int tiles_m, tiles_n;
    int first;           // row of x, or token, that C's first row or column stands for

    // z and dz
    float scale;         // of the logits (the softmax's sums: times log2(e))
    int limit;           // C's columns beyond this are no tokens
    const int32_t* target;
    float2* part;        // [n_part][m]: maxima and sums
    float* hit;          // the targets' logits
    const float* lse;
    const float* rate;
    const float* unit;   // what dz is multiplied by
    void* dz;
    int64_t dz_stride, dz_plane;   // from dz to the plane of what its rounding left, and on to the next; 0: none

    // sums
    float* sum;          // [splits][m][sum_stride]
    int64_t sum_stride;
    int add;             // to what is there
    void* out;           // C itself, [m][out_stride], values of out_type
    int64_t out_stride;
    int out_type;
    const float* factor;   // of C, or null
};

// The planes that dz has where it has more than one.
template <typename T>
constexpr int kPlanes = std::is_same<T, __bf16>::value ? kPlanesBf16 : kPlanesF16;

// What becomes of C: the logits' maxima and sums by rows and parts of 64 to 128
// tokens; the logits' gradient dz; a sum in 32 bits, by shares; or C itself.
enum { kStats, kGrad, kSum, kOut };

template <typename T>
struct Frag {
    typedef T vec __attribute__((ext_vector_type(8)));
    typedef vec type;
};
template <>
struct Frag<float> {
    typedef float type __attribute__((ext_vector_type(4)));
};

typedef float Acc __attribute__((ext_vector_type(16)));
typedef int Rsrc __attribute__((ext_vector_type(4)));
typedef short Short4 __attribute__((ext_vector_type(4)));

__device__ inline Acc mma(const Frag<__bf16>::type& a, const Frag<__bf16>::type& b, const Acc& c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ inline Acc mma(const Frag<_Float16>::type& a, const Frag<_Float16>::type& b, const Acc& c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ inline Acc mma(const Frag<float>::type& a, const Frag<float>::type& b, Acc c)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
    return c;
}

// 64 lanes' 16 bytes each, from memory to consecutive places in LDS.  An
// offset past the descriptor's bytes gives zeros.  m0, which holds the place in
// LDS, is the asm's own: an output of the s_mov (as a clobber it gives a
// warning, being a reserved register).
__device__ __forceinline__ void load_lds(uint32_t lds, uint32_t offset, const Rsrc& r)
{
    uint32_t m0;
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds"
                 : "={m0}"(m0)
                 : "s"(lds), "v"(offset), "s"(r)
                 : "memory");
}

constexpr uint32_t kNowhere = 0x80000000u;

// The place of a 16-byte chunk in a row of the tile that is summed along its
// rows (128 bytes): with it the 16 lanes of a part of a 16-byte read meet every
// bank once.
__device__ inline int along_place(int row, int chunk) { return chunk ^ ((row >> 1) & 7); }

// And in row k of a tile of R values a row: the four (32-bit values: two) rows
// that 32 (64) lanes read at a time lie in different banks.
template <typename T, int R>
__device__ inline int by_k_place(int k, int chunk)
{
    constexpr int bytes = R * (int)sizeof(T);
    if (sizeof(T) == 4) return bytes >= 256 ? chunk ^ (((k >> 2) & 1) << 3) : chunk;
    return bytes >= 256 ? chunk ^ ((k & 3) << 2) : bytes == 128 ? chunk ^ (((k >> 1) & 1) << 2) : chunk;
}

// Loads a factor's tiles of R rows (by k: columns), a step at a time: a wave's N
// loads of a step one by one, then next().
template <typename T, int R, int WAVES, bool BY_K>
struct Loader {
    static constexpr int N = R / 8 / WAVES;   // loads of a wave
    static constexpr int SIZE = sizeof(T), STEP = kStepBytes / SIZE;
    uint32_t offset[N];
    int head[N];         // the first value of the lane's chunk: in the step, by k in the tile
    const char* base;    // of the step
    int bytes;           // from there to the end of the step's rows
    int live;            // values of the rows from the step (by k: the tile) on
    int step;            // bytes from a step to the next
    int rows;            // by k: from the step on

    __device__ __forceinline__ void init(const Factor& f, int wave, int lane)
    {
        // a tile's rows behind the last may wrap round 2^32: only what is in the
        // factor is read, and those rows' results are not stored
        const uint32_t stride = (uint32_t)(f.stride * SIZE);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = (wave * N + i) * 1024 + lane * 16, width = BY_K ? R * SIZE : kStepBytes;
            const int row = at / width, place = at % width / 16;
            const int chunk = BY_K ? by_k_place<T, R>(row, place) : along_place(row, place);
            offset[i] = (uint32_t)row * stride + (uint32_t)chunk * 16;
            head[i] = chunk * (16 / SIZE);
        }
        step = BY_K ? (int)(STEP * stride) : kStepBytes;
    }

    // to the tile from row (column) `first` on, at step k of a plane
    __device__ __forceinline__ void begin(const Factor& f, int first, int plane, int k)
    {
        const int row = BY_K ? k * STEP : first, col = BY_K ? first : k * STEP, stride = (int)f.stride;
        base = (const char*)f.p + (plane * f.plane + (int64_t)row * stride + col) * SIZE;
        live = (int)f.cols - col;
        rows = (int)f.rows - row;
        bytes = ((min(rows, BY_K ? STEP : R) - 1) * stride + live) * SIZE;
    }

    // the wave's load i to its place from `lds` on
    __device__ __forceinline__ void load(int i, uint32_t lds) const
    {
        const uint64_t b = (uint64_t)base;
        const Rsrc r = {uniform((int)(uint32_t)b), uniform((int)((uint32_t)(b >> 32) & 0xffffu)), uniform(bytes), 0x00027000};
        load_lds(lds + i * 1024, head[i] < live ? offset[i] : kNowhere, r);
    }

    __device__ __forceinline__ void next()
    {
        base += step;
        if (BY_K) {
            rows -= STEP;
            bytes = (min(rows, STEP) - 1) * (step / STEP) + live * SIZE;
        } else {
            live -= STEP;
            bytes -= kStepBytes;
        }
    }

    // from here on zeros
    __device__ __forceinline__ void stop() { bytes = live = 0; }
};

// Lane's part of 32 rows (columns) of a tile in LDS, sub-step s of the step.
template <typename T, int R, bool BY_K>
__device__ __forceinline__ typename Frag<T>::type fragment(const char* tile, int block, int s, int lane)
{
    typename Frag<T>::type v;
    if (!BY_K) {
        const int row = block * 32 + (lane & 31);
        v = *(const typename Frag<T>::type*)(tile + row * kStepBytes + along_place(row, 2 * s + (lane >> 5)) * 16);
    } else if constexpr (sizeof(T) == 4) {
        const int m = block * 32 + (lane & 31), k = 8 * s + 4 * (lane >> 5);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = *(const float*)(tile + (k + e) * R * 4 + by_k_place<T, R>(k + e, m / 4) * 16 + m % 4 * 4);
    } else {
        // a read gives a lane the four values of its column from four rows k
        // that its sixteen lanes point at, four lanes a row
        const int m = block * 32 + ((lane >> 4) & 1) * 16 + (lane & 3) * 4, k = 16 * s + (lane >> 5) * 8 + ((lane >> 2) & 3);
        typedef __attribute__((address_space(3))) Short4 LdsShort4;
        union {
            Short4 half[2];
            typename Frag<T>::type whole;
        } u;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const char* p = tile + (k + 4 * e) * R * 2 + by_k_place<T, R>(k + 4 * e, m / 8) * 16 + m % 8 * 2;
            u.half[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsShort4*)p);
        }
        v = u.whole;
    }
    return v;
}

__device__ inline float swap_halves(float x)
{
    const uint32_t u = __float_as_uint(x);
    const auto v = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __uint_as_float((threadIdx.x & 32) ? v[0] : v[1]);
}

// 32 rows of W * 32 columns of a wave's, as the matrix instructions leave them
// (a lane has a row's values, four side by side), to memory by whole rows:
// through the wave's own part of LDS, so that a store takes runs of 64 bytes
// and more.  Stored straight from the registers, 8 bytes here and there, the
// logits' gradient of 8,192 x 32,768 took twice as long as its product.
// LEFT: what the rounding to T left goes `plane` values further on.
// ADD: to what is there.  Of the columns `cols` are stored, 16 bytes at a time
// where they are all of them and rows start at 16 bytes (`whole`).
constexpr int strip_bytes(int bm, int bn) { return bm * bn >= 256 * 256 ? 8192 : 4096; }   // of a wave
constexpr int strip_width(int bytes, int tn, int size, bool left)   // W
{
    return tn >= 2 && 32 * 64 * size * (left ? 2 : 1) <= bytes ? 2 : 1;
}

template <bool LEFT = false, bool ADD = false, int W, typename T>
__device__ __forceinline__ void store_strip(const float (&v)[W][16], char* strip, int lane, int rows, int cols, bool whole, T* out,
                                            int64_t stride, int64_t plane = 0)
{
    constexpr int V = 16 / sizeof(T), CHUNKS = W * 32 / V, ROW = CHUNKS * 16, PLANE = 32 * ROW, AT_ONCE = 64 / CHUNKS;
    // (rows of 256 bytes: chunk by row; shorter ones: so that the rows of 256 bytes differ)
    auto place = [](int row, int chunk) { return row * ROW + (chunk ^ ((CHUNKS >= 16 ? row : row / (16 / CHUNKS)) & (CHUNKS - 1))) * 16; };
    typedef T Four __attribute__((ext_vector_type(4)));
    typedef T Chunk __attribute__((ext_vector_type(V)));
    const int row = lane & 31, half = lane >> 5;
    wave_order();
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int col = j * 32 + q * 8 + half * 4;
            char* to = strip + place(row, col / V) + col % V * (int)sizeof(T);
            Four f;
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = (T)v[j][4 * q + e];
            *(Four*)to = f;
            if (LEFT) {
                Four rest;
#pragma unroll
                for (int e = 0; e < 4; ++e) rest[e] = (T)(v[j][4 * q + e] - (float)f[e]);
                *(Four*)(to + PLANE) = rest;
            }
        }
    wave_order();
    const int first = lane / CHUNKS, chunk = lane % CHUNKS;
    auto store = [&](const char* from, T* to) {
        to += first * stride + chunk * V;
        if (whole && rows >= 32) {
            Chunk old[ADD ? 32 / AT_ONCE : 1];
            if (ADD) {   // all loads, then all stores: a load waits for the stores before it
                T* p = to;
#pragma unroll
                for (int k = 0; k < 32 / AT_ONCE; ++k) {
                    old[ADD ? k : 0] = *(const Chunk*)p;
                    p += AT_ONCE * stride;
                    asm volatile("" : "+v"(p));   // one pointer, moved on, for all rows
                }
            }
#pragma unroll
            for (int k = 0; k < 32 / AT_ONCE; ++k) {
                Chunk c = *(const Chunk*)(from + place(k * AT_ONCE + first, chunk));
                if (ADD) c += old[ADD ? k : 0];
                *(Chunk*)to = c;
                to += AT_ONCE * stride;
                asm volatile("" : "+v"(to));
            }
        } else {
            for (int k = 0; k < 32 / AT_ONCE; ++k) {
                const int r = k * AT_ONCE + first;
                if (r < rows)
                    for (int e = 0; e < V; ++e)
                        if (chunk * V + e < cols) {
                            const T x = *(const T*)(from + place(r, chunk) + e * (int)sizeof(T));
                            to[e] = ADD ? to[e] + x : x;
                        }
                to += AT_ONCE * stride;
            }
        }
    };
    store(strip, out);
    if (LEFT) store(strip + PLANE, out + plane);
}

// The arguments once more, for use off the inner loop: behind a pointer that
// the compiler cannot follow, so that it does not keep them all in registers
// (it had put the loop's own out to lanes of vector registers).
__device__ __forceinline__ const ProductArgs& cold_args()
{
    typedef const __attribute__((address_space(4))) ProductArgs* Constant;
    Constant p = (Constant)__builtin_amdgcn_kernarg_segment_ptr();   // the kernel's only argument
    asm volatile("" : "+s"(p));
    return *(const ProductArgs*)p;
}

// An item of work: a tile of C and a share of its steps, one at least (the
// launch sees to that: no more shares than steps).
struct Item {
    int m, n, split;
    int t0, t1;
};

__device__ inline Item item_at(const ProductArgs& g, uint32_t at)
{
    // eight rows of tiles at a time, so that neighbours share rows and columns
    const uint32_t tiles = (uint32_t)g.tiles_m * (uint32_t)g.tiles_n;
    const uint32_t split = at / tiles, tile = at - split * tiles, width = 8 * (uint32_t)g.tiles_n, band = tile / width;
    const uint32_t first = band * 8, rows = min(8u, (uint32_t)g.tiles_m - first), in = tile - band * width, n = in / rows;
    const int steps = g.k_steps * g.planes;
    const uint64_t t0 = (uint64_t)steps * split, t1 = t0 + steps;
    return {uniform((int)(first + in - n * rows)), uniform((int)n), uniform((int)split),
            uniform(g.splits == 1 ? 0 : (int)(t0 / (uint32_t)g.splits)), uniform(g.splits == 1 ? steps : (int)(t1 / (uint32_t)g.splits))};
}

// A lane's row of partial maxima and sums (in units of log2), of the wave's
// TN * 32 columns, of which `left` are tokens.  Per value: a maximum (of three),
// an fma, an exponential (four times an instruction's time) and a sum.
// RARE: some are no tokens, or the scale is not positive (`sign` is its sign).
template <bool RARE, int TN>
__device__ __forceinline__ float2 row_stats(const Acc (&acc)[TN], float scale, float sign, int left)
{
    const int quad = (threadIdx.x & 32) / 8;
    auto value = [&](int j, int r) {
        if (!RARE) return acc[j][r];
        return j * 32 + 8 * (r / 4) + quad + r % 4 < left ? acc[j][r] * sign : -INFINITY;
    };
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, value(j, r));
    top = fmaxf(top, swap_halves(top));
    top *= scale;
    const float from = top == -INFINITY ? 0.0f : top;   // 2^-infinity is 0 from anywhere
    float sum[4] = {};
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) sum[r % 4] += __builtin_amdgcn_exp2f(__builtin_fmaf(value(j, r), scale, -from));
    float all = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    all += swap_halves(all);
    return make_float2(top, all);   // of no tokens (-infinity, 0), which joins nothing
}

// Blocks of a product's tile that a CU holds at a time.
constexpr int product_lds(int bm, int bn, int waves, bool strips)
{
    return 2 * (bm + bn) * kStepBytes + (strips ? waves * strip_bytes(bm, bn) : 0);
}
constexpr int product_blocks(int bm, int bn, int waves, bool strips) { return kLdsBytes / product_lds(bm, bn, waves, strips); }

// One product: C = a b over the tiles.  A block of WM x WN waves makes tiles of
// BM x BN, each wave BM / WM x BN / WN of them in blocks of 32 x 32.  Steps of
// 128 bytes of the summed values go through two halves of LDS: one is filled
// while the other is multiplied.  A block takes its tiles one after the other
// as one run of steps, so that a tile's first steps are loaded while the one
// before is finished.
//
// Four waves of 128 x 128 read the least of LDS for their products (8 KB each
// for 16 matrix instructions, half of what LDS gives in that time; eight waves
// of 128 x 64 would take three quarters, beside a quarter for the loads), and
// their 256 results a lane leave 256 registers for all else: one wave a SIMD
// (12 to 164 bytes a lane go to scratch where a tile of logits, dz or C itself
// is finished, none between the products).  Tiles of 128 x 128 have two.
// Bound by the matrix instructions (64% of the time at 8,192^3 bf16, 1.20
// PFLOP/s; the rest are waits at the step's barrier and for fragments), and for
// short sums by the tiles' ends: 16,384 x 32,768 logits of 1,024 values 0.99 ms
// (1.11 PFLOP/s), of 512 0.57 (0.97).
template <typename T, int BM, int BN, int WM, int WN, bool A_BY_K, bool B_BY_K, int WHAT>
__global__ __launch_bounds__(64 * WM * WN, tile_blocks(BM, BN) * WM * WN / 4) void k_product(const ProductArgs args)
{
    constexpr int WAVES = WM * WN, TM = BM / WM / 32, TN = BN / WN / 32;
    constexpr int STAGE = (BM + BN) * kStepBytes, STRIP = strip_bytes(BM, BN);
    extern __shared__ __align__(16) char smem[];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;

    // Blocks go round the 8 XCDs: each XCD has a run of the items, which its
    // blocks take in turn, so that those in flight share its L2.
    const uint32_t total = (uint32_t)args.tiles_m * (uint32_t)args.tiles_n * (uint32_t)args.splits;
    const uint32_t xcds = min(8u, gridDim.x), xcd = blockIdx.x % 8, per = total / xcds, more = total % xcds;
    const uint32_t turn = uniform((gridDim.x - xcd + 7) / 8), end = uniform((xcd + 1) * per + min(xcd + 1, more));
    uint32_t at = uniform(xcd * per + min(xcd, more) + blockIdx.x / 8);   // the item that is multiplied, and
    uint32_t ahead = at;                                                  // the one that is loaded
    if (at >= end) return;

    Loader<T, BM, WAVES, A_BY_K> la;
    Loader<T, BN, WAVES, B_BY_K> lb;
    la.init(args.a, wave, lane);
    lb.init(args.b, wave, lane);
    const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem;
    const uint32_t lds_a = lds + wave * (la.N * 1024), lds_b = lds + BM * kStepBytes + wave * (lb.N * 1024);
    constexpr int LOADS = la.N + lb.N, FIRST = LOADS / 2;
    auto load = [&](int i, uint32_t half) {   // one of a step's loads
        if (i < la.N) la.load(i, lds_a + half);
        else lb.load(i - la.N, lds_b + half);
    };
    int to_load = 1, to_wrap = 1;   // steps that are left of the item ahead, and of the plane
    ahead -= turn;
    auto next = [&] {
        if (to_load == 0) return;
        --to_load;
        if (--to_wrap != 0) {
            la.next();
            lb.next();
        } else {   // the next plane, or the next item
            if (to_load == 0 && (ahead += turn, (int)(end - ahead) <= 0)) {
                la.stop();
                lb.stop();
                return;
            }
            const ProductArgs& g = cold_args();
            const Item w = item_at(g, ahead);
            if (to_load == 0) to_load = w.t1 - w.t0;
            const int t = w.t1 - to_load, plane = uniform(t / g.k_steps), k = t - plane * g.k_steps;
            la.begin(g.a, w.m * BM, plane, k);
            lb.begin(g.b, w.n * BN, 0, k);
            to_wrap = min(to_load, g.k_steps - k);
        }
    };

    // A step is four sub-steps; each sub-step's fragments are read while the
    // one before is multiplied.  Before the last sub-step every wave has read
    // its half of LDS and the other half's loads are in: one barrier a step,
    // after which the half just read is filled for the step after the next.
    // The loads take two sub-steps, the last of this step and the first of the
    // next: 64 KB at 64 bytes a cycle are 1,024 cycles, two sub-steps' products.
    // (All in the one: 1,120 against 1,097 us, 16,384 x 32,768 x 1,024.)
    Acc acc[TM][TN];
    typename Frag<T>::type fa[2][TM], fb[2][TN];
    int half = 0;
    auto read = [&](int i, int from, int s, int to) {   // one of a sub-step's fragments
        const char* tile = smem + from * STAGE;
        if (i < TM) fa[to][i] = fragment<T, BM, A_BY_K>(tile, wm * TM + i, s, lane);
        else fb[to][i - TM] = fragment<T, BN, B_BY_K>(tile + BM * kStepBytes, wn * TN + i - TM, s, lane);
    };
    auto sub_step = [&](auto which) {
        constexpr int s = decltype(which)::value, MMAS = TM * TN, READS = TM + TN;
        // between the products: the next fragments, and after the barrier the loads
#pragma unroll
        for (int n = 0; n < MMAS; ++n) {
            const int i = n / TN, j = n % TN;
            acc[i][j] = mma(fb[s & 1][j], fa[s & 1][i], acc[i][j]);
#pragma unroll
            for (int r = n * READS / MMAS; r < (n + 1) * READS / MMAS; ++r)
                read(r, s == 3 ? half ^ 1 : half, (s + 1) & 3, (s + 1) & 1);
            if (s == 3) {
#pragma unroll
                for (int l = n * FIRST / MMAS; l < (n + 1) * FIRST / MMAS; ++l) load(l, half * STAGE);
            }
            if (s == 0) {
#pragma unroll
                for (int l = n * (LOADS - FIRST) / MMAS; l < (n + 1) * (LOADS - FIRST) / MMAS; ++l)
                    load(FIRST + l, (half ^ 1) * STAGE);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    next();
#pragma unroll
    for (int i = 0; i < LOADS; ++i) load(i, 0);
    next();
#pragma unroll
    for (int i = 0; i < FIRST; ++i) load(i, STAGE);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(FIRST) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < TM + TN; ++i) read(i, 0, 0, 0);

    for (; at < end; at += turn) {
        // Value r of a 32 x 32 block's lane: row lane % 32, column
        // 8 (r / 4) + 4 (lane / 32) + r % 4.
        const int quad = (lane >> 5) * 4;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
        int t;
        {
            const ProductArgs& g = cold_args();
            const Item w = item_at(g, at);
            t = w.t1 - w.t0;
        }
        for (; t > 0; --t) {
            sub_step(std::integral_constant<int, 0>());
            next();
            sub_step(std::integral_constant<int, 1>());
            sub_step(std::integral_constant<int, 2>());
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            sub_step(std::integral_constant<int, 3>());
            half ^= 1;
        }

        const ProductArgs& g = cold_args();
        const Item w = item_at(g, at);
        const int m0 = w.m * BM + wm * TM * 32, n0 = w.n * BN + wn * TN * 32;
        if constexpr (WHAT == kStats || WHAT == kGrad) {
            const int left = g.limit - n0;
            // What the rows' lanes need, before the first store: a load waits for
            // the stores before it.
            int to[TM];   // the target's place from the wave's first column on
            float rate[TM], lse[TM];
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int row = m0 + i * 32 + (lane & 31);
                to[i] = row < g.m && g.target ? g.target[row] - g.first - n0 : -1;
                if (WHAT == kGrad) {
                    rate[i] = row < g.m ? g.rate[row] * g.unit[0] : 0.0f;
                    lse[i] = rate[i] != 0.0f ? g.lse[row] : 0.0f;
                }
            }
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int row = m0 + i * 32 + (lane & 31);
                if constexpr (WHAT == kStats) {
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        const int in = to[i] - j * 32;
                        if (!__ballot((uint32_t)in < 32u)) continue;   // few blocks hold a row's target
                        float v = 0.0f;
#pragma unroll
                        for (int r = 0; r < 16; ++r) v = in == 8 * (r / 4) + quad + r % 4 ? acc[i][j][r] : v;
                        if ((uint32_t)in < 32u && (in & 4) == quad && to[i] < left) g.hit[row] = v * g.scale;
                    }
                    float2 s;
                    if (left >= TN * 32 && g.scale > 0.0f) s = row_stats<false>(acc[i], g.scale, 1.0f, left);
                    else if (g.scale != 0.0f) s = row_stats<true>(acc[i], fabsf(g.scale), g.scale > 0.0f ? 1.0f : -1.0f, left);
                    else s = row_stats<true>(acc[i], 1.0f, 0.0f, left);
                    if (row < g.m && lane < 32) g.part[((int64_t)w.n * WN + wn) * g.m + row] = s;
                    __builtin_amdgcn_sched_barrier(0);
                } else {
                    T* out = (T*)g.dz + (int64_t)(m0 + i * 32) * g.dz_stride + n0;
                    char* strip = smem + 2 * STAGE + wave * STRIP;
                    // dz is rounded to T, its products' type: half a step of each
                    // value, and in dx of bf16 an error of 2.4e-3 where rounding
                    // the result alone leaves 1.7e-3.  More planes in dx too would
                    // double its steps; they are for a 32-bit dtable (kPlanes).
                    auto store = [&](auto left_over) {
                        constexpr bool LEFT = decltype(left_over)::value;
                        constexpr int W = strip_width(STRIP, TN, sizeof(T), LEFT);
#pragma unroll
                        for (int j = 0; j < TN; j += W) {
                            float v[W][16];
#pragma unroll
                            for (int h = 0; h < W; ++h) {
                                const int in = to[i] - (j + h) * 32;
#pragma unroll
                                for (int r = 0; r < 16; ++r)
                                    v[h][r] = rate[i] * __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j + h][r], g.scale, -lse[i]) * kLog2e);
                                if (__ballot((uint32_t)in < 32u)) {
#pragma unroll
                                    for (int r = 0; r < 16; ++r) v[h][r] -= in == 8 * (r / 4) + quad + r % 4 ? rate[i] : 0.0f;
                                }
                                if (left < (j + h + 1) * 32) {   // past the tokens
#pragma unroll
                                    for (int r = 0; r < 16; ++r)
                                        v[h][r] = (j + h) * 32 + 8 * (r / 4) + quad + r % 4 < left ? v[h][r] : 0.0f;
                                }
                            }
                            store_strip<LEFT>(v, strip, lane, g.m - m0 - i * 32, W * 32, true, out + j * 32, g.dz_stride, g.dz_plane);
                            if constexpr (LEFT && kPlanes<T> == 3) {
#pragma unroll
                                for (int h = 0; h < W; ++h)
#pragma unroll
                                    for (int r = 0; r < 16; ++r) {
                                        v[h][r] -= (float)(T)v[h][r];
                                        v[h][r] -= (float)(T)v[h][r];
                                    }
                                store_strip(v, strip, lane, g.m - m0 - i * 32, W * 32, true, out + 2 * g.dz_plane + j * 32, g.dz_stride);
                            }
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    };
                    if constexpr (sizeof(T) < 4) {
                        if (g.dz_plane) store(std::true_type());
                        else store(std::false_type());
                    } else {
                        store(std::false_type());
                    }
                }
            }
        } else {
            char* strip = smem + 2 * STAGE + wave * STRIP;
            auto store = [&](auto add, auto* out, int64_t stride, float factor) {
                using U = std::remove_reference_t<decltype(*out)>;
                constexpr int W = strip_width(STRIP, TN, sizeof(U), false);
                const bool aligned = ((uint64_t)out | (uint64_t)stride * sizeof(U)) % 16 == 0;
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; j += W) {
                        float v[W][16];
#pragma unroll
                        for (int h = 0; h < W; ++h)
#pragma unroll
                            for (int r = 0; r < 16; ++r) v[h][r] = acc[i][j + h][r] * factor;
                        const int row = m0 + i * 32, cols = g.n - n0 - j * 32;
                        store_strip<false, decltype(add)::value>(v, strip, lane, g.m - row, cols, aligned && cols >= W * 32,
                                                                 out + row * stride + n0 + j * 32, stride);
                        __builtin_amdgcn_sched_barrier(0);
                    }
            };
            if constexpr (WHAT == kSum) {
                float* sum = g.sum + (int64_t)w.split * g.m * g.sum_stride;
                if (g.add) store(std::true_type(), sum, g.sum_stride, 1.0f);
                else store(std::false_type(), sum, g.sum_stride, 1.0f);
            } else {
                const float factor = g.factor ? g.factor[0] : 1.0f;
                if (g.out_type == HGB_F32) store(std::false_type(), (float*)g.out, g.out_stride, factor);
                else store(std::false_type(), (T*)g.out, g.out_stride, factor);
            }
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing is on its way to LDS when the block ends
}

// Each row's rate, the factor of its logits' gradient (zero without one), and
// the blocks' largest finite one (from a rate that is not, no unit could be
// made for the other rows).
struct RateArgs {
    const float* grad;
    float scale;
    int64_t n;
    int32_t vocab;
    const int32_t* token;
    int top;               // tokens of a row
    int32_t pad;
    const void* teacher;   // or null
    int teacher_type;
    float* rate;           // [n], then kRateWords
    uint32_t* err;
};

__device__ inline float teacher_at(const void* p, int type, int64_t i)
{
    return type == HGB_F32 ? ((const float*)p)[i] : type == HGB_BF16 ? (float)((const __bf16*)p)[i] : (float)((const _Float16*)p)[i];
}

__global__ __launch_bounds__(256) void k_head_rate(const RateArgs a)
{
    __shared__ float most[4];
    float top = 0.0f;
    bool bad = false;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.n; i += (int64_t)gridDim.x * 256) {
        bool live = false;
        for (int k = 0; k < a.top; ++k) {
            const int32_t t = a.token[i * a.top + k];
            const bool in = t >= 0 && t < a.vocab && t != a.pad;
            if (!in && t != a.pad) bad = true;
            live = live || (in && (!a.teacher || teacher_at(a.teacher, a.teacher_type, i * a.top + k) != -INFINITY));
        }
        const float r = live ? a.grad[i] * a.scale : 0.0f;
        a.rate[i] = r;
        if (fabsf(r) < INFINITY) top = fmaxf(top, fabsf(r));
    }
    if (bad) atomicOr(a.err, kVecErrToken);
    for (int s = 32; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor(top, s));
    if ((threadIdx.x & 63) == 0) most[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0) a.rate[a.n + 2 + blockIdx.x] = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
}

// What the logits' gradient is multiplied by for its type, and one over it:
// fp16 holds values of 2^-24 to 2^16, and a rate times a probability is often
// less than the former, so the largest rate (of `blocks` blocks') is brought
// between 2^14 and 2^15 (below 2^-112 as near as 2^126 brings it, whose inverse
// is the least normal number).  Powers of two: exact.
__device__ inline void rate_unit(float* words, int blocks, bool half)
{
    float top = 0.0f;
    for (int i = threadIdx.x; i < blocks; i += 64) top = fmaxf(top, words[2 + i]);
    for (int s = 32; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor(top, s));
    if (threadIdx.x == 0) {
        int e = 0;   // top in [2^(e - 1), 2^e)
        if (half && top > 0.0f) (void)frexpf(top, &e);
        e = half ? min(126, 15 - e) : 0;   // -113 at least: top is below 2^128
        words[0] = ldexpf(1.0f, e);
        words[1] = ldexpf(1.0f, -e);
    }
}

// Rows copied to where they start at 16 bytes, with zeros behind their end,
// and instead of rows whose rate is zero.  With rates, the first wave makes
// their unit.
template <typename T>
__global__ __launch_bounds__(256) void k_head_copy(const T* x, int64_t stride, int64_t n, int dim, int dp, float* rate, int blocks,
                                                   T* out)
{
    if (rate && blockIdx.x == 0 && threadIdx.x < 64) rate_unit(rate + n, blocks, std::is_same<T, _Float16>::value);
    constexpr int V = 16 / sizeof(T);
    const int per = dp / V;
    const int64_t total = n * per;
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < total; at += (int64_t)gridDim.x * 256) {
        const int64_t row = at / per;
        const int c = (int)(at - row * per) * V;
        typename Vals<T, V>::type v{};
        if (!rate || rate[row] != 0.0f) v = load_raw<V>(x + row * stride + c, dim - c);
        *(typename Vals<T, V>::type*)(out + row * dp + c) = v;
    }
}

// A sum's shares added up: rows of zero rate are zero.  8 shares of 4,096 x 512:
// 14 us (67 MB, 5 TB/s).
template <typename T>
__global__ __launch_bounds__(256) void k_head_join(const float* sum, int64_t sum_stride, int splits, int64_t rows, int dim,
                                                   const float* rate, const float* factor, T* out, int64_t stride)
{
    const int per = (dim + 3) / 4;
    const int64_t total = rows * per;
    const float f = factor[0];
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < total; at += (int64_t)gridDim.x * 256) {
        const int64_t row = at / per;
        const int c = (int)(at - row * per) * 4;
        float v[4] = {};
        if (!rate || rate[row] != 0.0f)
#pragma unroll 8
            for (int s = 0; s < splits; ++s) {
                const float4 u = *(const float4*)(sum + ((int64_t)s * rows + row) * sum_stride + c);
                v[0] += u.x;
                v[1] += u.y;
                v[2] += u.z;
                v[3] += u.w;
            }
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= f;
        store_vals<4>(v, out + row * stride + c, dim - c);
    }
}

// Rows of `width` bytes, `stride` apart, set to zero.
__global__ __launch_bounds__(256) void k_head_zero(char* out, int64_t stride, int64_t rows, int64_t width)
{
    const int64_t per = width / 2, total = rows * per;
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < total; at += (int64_t)gridDim.x * 256)
        ((uint16_t*)(out + at / per * stride))[at % per] = 0;
}

// The rows' partial maxima and sums (of 2^z) joined: lse, and the loss of a
// target.  2^log_rows rows a block, the other threads side by side in parts.
// 16,384 rows of 256 parts: 13 us (2.5 TB/s).
struct LossArgs {
    const float2* part;
    int64_t parts, rows;
    int log_rows;
    const float* hit;       // targets' logits, times log2(e)
    const int32_t* target;  // null for a teacher's
    int32_t pad;
    int32_t vocab;
    float* loss;
    float* lse;
    uint32_t* err;
};

__device__ inline float2 stat_join(float2 a, float2 b)
{
    const float top = fmaxf(a.x, b.x), from = top == -INFINITY ? 0.0f : top;
    return make_float2(top, a.y * __builtin_amdgcn_exp2f(a.x - from) + b.y * __builtin_amdgcn_exp2f(b.x - from));
}

__global__ __launch_bounds__(256) void k_head_loss(const LossArgs a)
{
    __shared__ float2 got[256];
    const int rows = 1 << a.log_rows, slices = 256 >> a.log_rows;
    const int r = threadIdx.x & (rows - 1), slice = threadIdx.x >> a.log_rows;
    const int64_t row = (int64_t)blockIdx.x * rows + r;
    float2 s = make_float2(-INFINITY, 0.0f);
    if (row < a.rows)
        for (int64_t p = slice; p < a.parts; p += slices) s = stat_join(s, a.part[p * a.rows + row]);
    got[threadIdx.x] = s;
    __syncthreads();
    for (int step = slices / 2; step > 0; step /= 2) {
        if (slice < step) got[threadIdx.x] = stat_join(got[threadIdx.x], got[threadIdx.x + step * rows]);
        __syncthreads();
    }
    if (slice != 0 || row >= a.rows) return;
    s = got[r];
    const float lse2 = s.x + __builtin_amdgcn_logf(s.y);
    a.lse[row] = lse2 * kLn2;
    if (a.target) {
        const int32_t t = a.target[row];
        const bool live = t >= 0 && t < a.vocab && t != a.pad;
        if (!live && t != a.pad) atomicOr(a.err, kVecErrToken);
        a.loss[row] = live ? (lse2 - a.hit[row]) * kLn2 : 0.0f;
    }
}

// A teacher's slots of a row, a wave's lanes side by side: which are left, and
// their probabilities.
struct TeacherArgs {
    const int32_t* token;
    const void* teacher;
    int teacher_type;
    int top;
    int32_t vocab;
    float heat;
};

constexpr int kTeacherSlots = kDistillMaxTop / 64;

struct TeacherRow {
    int32_t token[kTeacherSlots];
    float t[kTeacherSlots];   // (teacher - max) / T
    float p[kTeacherSlots];
    float log_sum;
    bool some, bad;
};

__device__ inline float wave_max(float x)
{
    for (int s = 32; s > 0; s >>= 1) x = fmaxf(x, __shfl_xor(x, s));
    return x;
}

__device__ inline TeacherRow teacher_row(const TeacherArgs& a, int64_t row, int lane)
{
    TeacherRow w;
    w.bad = false;
    float top = -INFINITY;
    bool some = false;
#pragma unroll
    for (int i = 0; i < kTeacherSlots; ++i) {
        const int k = i * 64 + lane;
        w.token[i] = -1;
        w.t[i] = -INFINITY;
        if (k < a.top) {
            const int32_t t = a.token[row * a.top + k];
            if (t >= 0 && t < a.vocab) {
                w.token[i] = t;
                w.t[i] = teacher_at(a.teacher, a.teacher_type, row * a.top + k);
            } else if (t != -1) {
                w.bad = true;
            }
        }
        some = some || w.t[i] != -INFINITY;
        top = fmaxf(top, w.t[i]);
    }
    top = wave_max(top);
    w.some = __ballot(some) != 0;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kTeacherSlots; ++i) {
        w.t[i] = w.t[i] == -INFINITY ? -INFINITY : (w.t[i] - top) / a.heat;   // over T first, the largest values would be infinite
        w.p[i] = expf(w.t[i]);
        sum += w.p[i];
    }
    sum = group_sum(sum, 6);
    w.log_sum = logf(sum);
#pragma unroll
    for (int i = 0; i < kTeacherSlots; ++i) w.p[i] /= sum;
    return w;
}

// The student's logits at the teacher's tokens: a wave a slot.  Bound by the
// tokens' vectors, out of the caches: 8,192 rows of 64 slots of 2 KB 144 us (7.4
// TB/s).  Picked out of the logits' tiles instead they cost those 359 us more.
template <typename T>
__global__ __launch_bounds__(256) void k_distill_pick(const T* x, int64_t x_stride, const T* table, int64_t table_stride,
                                                      int64_t n, int dim, const TeacherArgs a, float* picked)
{
    constexpr int V = 16 / sizeof(T);
    const int lane = threadIdx.x & 63;
    const int64_t slots = n * a.top;
    for (int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); at < slots; at += (int64_t)gridDim.x * 4) {
        const int32_t t = a.token[at];
        const bool in = t >= 0 && t < a.vocab;
        float sum = 0.0f;
        if (in) {
            const T* px = x + at / a.top * x_stride;
            const T* pw = table + t * table_stride;
            for (int c = lane * V; c < dim; c += 64 * V) {
                float u[V], w[V];
                load_vals<V>(u, px + c, dim - c);
                load_vals<V>(w, pw + c, dim - c);
#pragma unroll
                for (int e = 0; e < V; ++e) sum = __builtin_fmaf(u[e], w[e], sum);
            }
        }
        sum = group_sum(sum, 6);
        if (lane == 0) picked[at] = in ? sum / a.heat : 0.0f;
    }
}

// loss = T^2 (lse + the sum of p (log p - z)): a wave a row.
__global__ __launch_bounds__(256) void k_distill_loss(int64_t n, const TeacherArgs a, const float* lse, const float* picked,
                                                      float* loss, uint32_t* err)
{
    const int lane = threadIdx.x & 63;
    for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < n; row += (int64_t)gridDim.x * 4) {
        const TeacherRow w = teacher_row(a, row, lane);
        if (w.bad) atomicOr(err, kVecErrToken);
        const float whole = lse[row];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kTeacherSlots; ++i)
            if (w.t[i] != -INFINITY) {   // p = 0 of a finite teacher's logit counts for nothing
                const float d = w.t[i] - w.log_sum + (whole - picked[row * a.top + i * 64 + lane]);
                sum += w.p[i] == 0.0f ? 0.0f : w.p[i] * d;
            }
        sum = group_sum(sum, 6);
        if (lane == 0) loss[row] = w.some ? a.heat * a.heat * sum : 0.0f;
    }
}

// The logits' gradient at the teacher's tokens in [first, first + width):
// rate (q - P), P the sum over the row's slots of the same token.  A wave a
// row; slots of one token store the same value.
template <typename T>
__global__ __launch_bounds__(256) void k_distill_dz(int64_t n, const TeacherArgs a, const float* lse, const float* picked,
                                                    const float* rate, const float* unit, int first, int width, T* dz,
                                                    int64_t dz_stride, int64_t dz_plane)
{
    const int lane = threadIdx.x & 63;
    for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < n; row += (int64_t)gridDim.x * 4) {
        const float r = rate[row] * unit[0];
        if (r == 0.0f) continue;   // the row's gradient is zeros already
        const TeacherRow w = teacher_row(a, row, lane);
        float p[kTeacherSlots] = {};
#pragma unroll
        for (int i = 0; i < kTeacherSlots; ++i) {
            if (i * 64 >= a.top) break;
            for (int l = 0; l < min(64, a.top - i * 64); ++l) {
                const int32_t t = __shfl(w.token[i], l);
                const float add = __shfl(w.p[i], l);
#pragma unroll
                for (int j = 0; j < kTeacherSlots; ++j) p[j] += t == w.token[j] ? add : 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < kTeacherSlots; ++i) {
            const int to = w.token[i] - first;
            if (w.token[i] < 0 || to < 0 || to >= width) continue;
            const float q = expf(picked[row * a.top + i * 64 + lane] - lse[row]);
            const float d = r * (q - p[i]);
            T* at = dz + row * dz_stride + to;
            *at = (T)d;
            if (dz_plane) {
                const float rest = d - (float)(T)d;
                at[dz_plane] = (T)rest;
                if (kPlanes<T> == 3) at[2 * dz_plane] = (T)(rest - (float)(T)rest);
            }
        }
    }
}

}  // namespace hgb
