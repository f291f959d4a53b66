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
    float scale;         // of the logits (kStats: times log2(e))
    int limit;           // C's columns beyond this are no tokens
    const int32_t* target;
    float2* part;        // [n_part][m]: maxima and sums
    float* hit;          // the targets' logits
    const float* lse;
    const float* rate;
    const float* unit;   // what dz is multiplied by
    void* dz;
    int64_t dz_stride, dz_plane;

    // sums
    float* sum;          // [splits][m][sum_stride]
    int64_t sum_stride;
    int add;             // to what is there
    void* out;           // C itself, [m][out_stride], values of out_type
    int64_t out_stride;
    int out_type;
    const float* factor;   // of C, or null
};

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
// offset past the descriptor's bytes gives zeros.
__device__ __forceinline__ void load_lds(uint32_t lds, uint32_t offset, const Rsrc& r)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(offset), "s"(r)
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

// Loads a factor's tile of R rows (by k: columns), a step at a time: a wave's N
// loads of a step one by one, then next().  Past the last step zeros are loaded.
template <typename T, int R, int WAVES, bool BY_K>
struct Loader {
    static constexpr int N = R / 8 / WAVES;   // loads of a wave
    static constexpr int SIZE = sizeof(T), STEP = kStepBytes / SIZE;
    uint32_t offset[N];
    int tail[2];       // along: the first value of the lane's chunk in the step, of even and odd loads
    const char* base;  // of the step
    int64_t left;      // bytes from there to the factor's end
    int64_t step, back;   // bytes from a step to the next, and from a plane's last step to the next plane's first
    int live;          // along: values of the rows from the step on
    int cols, k, steps, to_go;

    // the steps [t0, t1) of all the planes'
    __device__ __forceinline__ void init(const Factor& f, int64_t first, int wave, int lane, int k_steps, int64_t plane, int t0, int t1)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = (wave * N + i) * 1024 + lane * 16;
            if (BY_K) {
                constexpr int row_bytes = R * SIZE;
                const int kk = at / row_bytes, chunk = by_k_place<T, R>(kk, at % row_bytes / 16);
                const int64_t col = first + chunk * (16 / SIZE);
                offset[i] = col < f.cols ? (uint32_t)(kk * f.stride * SIZE + chunk * 16) : kNowhere;
            } else {
                const int row = at / kStepBytes, chunk = along_place(row, at % kStepBytes / 16);
                offset[i] = (uint32_t)(row * f.stride * SIZE + chunk * 16);
                tail[i & 1] = chunk * (16 / SIZE);
                static_assert(R / 8 % 2 == 0 && (N % 2 == 0 || N == 1), "chunks go by a load's parity");
            }
        }
        steps = k_steps;
        const int at_plane = uniform(t0 / k_steps);
        k = t0 - at_plane * k_steps;
        to_go = t1 - t0;
        step = BY_K ? STEP * f.stride * SIZE : kStepBytes;
        back = plane * SIZE - step * (k_steps - 1);
        const int64_t row = BY_K ? (int64_t)k * STEP : first, col = BY_K ? first : (int64_t)k * STEP;
        base = (const char*)f.p + (at_plane * plane + row * f.stride + col) * SIZE;
        left = ((f.rows - 1 - row) * f.stride + f.cols - col) * SIZE;
        cols = (int)f.cols;
        live = cols - k * STEP;
    }

    // the wave's load i to its place from `lds` on
    __device__ __forceinline__ void load(int i, uint32_t lds) const
    {
        const uint64_t b = (uint64_t)base;
        const uint32_t bytes = to_go > 0 ? (uint32_t)min(left, (int64_t)0x7ffffff0) : 0;
        const Rsrc r = {uniform((int)(uint32_t)b), uniform((int)((uint32_t)(b >> 32) & 0xffffu)), uniform((int)bytes), 0x00027000};
        load_lds(lds + i * 1024, BY_K || tail[i & 1] < live ? offset[i] : kNowhere, r);
    }

    __device__ __forceinline__ void next()
    {
        --to_go;
        if (++k == steps) {
            k = 0;
            base += back;
            left += step * (steps - 1);
            live = cols;
        } else {
            base += step;
            left -= step;
            live -= STEP;
        }
    }
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

// A wave's 32 rows of TN * 32 columns, as the matrix instructions leave them (a
// lane has a row's values, four side by side), to memory by whole rows: through
// the wave's own part of LDS, so that a store takes runs of 128 bytes and more.
// Stored straight from the registers, 8 bytes here and there, the logits'
// gradient of 8,192 x 32,768 took twice as long as its product.
template <typename T, int TN>
__device__ __forceinline__ void store_strip(const Acc (&acc)[TN], char* strip, int lane, int rows, T* out, int64_t stride)
{
    constexpr int V = 16 / sizeof(T), CHUNKS = TN * 32 / V, ROW = CHUNKS * 16;
    auto place = [](int row, int chunk) { return row * ROW + (chunk ^ (CHUNKS >= 16 ? row & (CHUNKS - 1) : (row >> 1) & 7)) * 16; };
    const int row = lane & 31, half = lane >> 5;
    wave_order();
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int col = j * 32 + q * 8 + half * 4;
            typedef T Four __attribute__((ext_vector_type(4)));
            Four v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = (T)acc[j][4 * q + e];
            *(Four*)(strip + place(row, col / V) + col % V * (int)sizeof(T)) = v;
        }
    wave_order();
#pragma unroll
    for (int k = 0; k < 32 * CHUNKS / 64; ++k) {
        const int at = k * 64 + lane, r = at / CHUNKS, chunk = at % CHUNKS;
        if (r < rows) *(uint4*)(out + r * stride + chunk * V) = *(const uint4*)(strip + place(r, chunk));
    }
}

// A block's tile of C.
struct TilePlace {
    int m, n, split;
};

// Blocks go round the 8 XCDs: each gets a run of tiles, eight rows of tiles at
// a time, so that the tiles in flight on one share rows and columns in its L2.
__device__ inline TilePlace tile_place(const ProductArgs& g)
{
    const uint32_t tiles = (uint32_t)g.tiles_m * (uint32_t)g.tiles_n, total = tiles * (uint32_t)g.splits;
    const uint32_t xcd = blockIdx.x & 7, per = total / 8, more = total % 8;
    const uint32_t at = xcd * per + min(xcd, more) + blockIdx.x / 8;
    const uint32_t tile = at % tiles, width = 8 * (uint32_t)g.tiles_n, band = tile / width, first = band * 8;
    const uint32_t rows = min(8u, (uint32_t)g.tiles_m - first), in = tile % width;
    return {uniform((int)(first + in % rows)), uniform((int)(in / rows)), uniform((int)(at / tiles))};
}

// One product: C = a b over the tiles.  A block of WM x WN waves makes a tile
// of BM x BN, each wave BM / WM x BN / WN of it in blocks of 32 x 32.  Steps of
// 128 bytes of the summed values go through two halves of LDS: one is filled
// while the other is multiplied.
template <typename T, int BM, int BN, int WM, int WN, bool A_BY_K, bool B_BY_K, int WHAT>
__global__ __launch_bounds__(64 * WM * WN) void k_product(const ProductArgs g)
{
    constexpr int WAVES = WM * WN, TM = BM / WM / 32, TN = BN / WN / 32;
    constexpr int STAGE = (BM + BN) * kStepBytes;
    constexpr bool LANE_IS_ROW = WHAT == kStats || WHAT == kGrad;   // else a lane holds a column's values
    extern __shared__ __align__(16) char smem[];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const TilePlace at = tile_place(g);
    const int64_t row0 = (int64_t)at.m * BM, col0 = (int64_t)at.n * BN;
    const int steps = g.k_steps * g.planes;
    const int t0 = uniform((int)((int64_t)steps * at.split / g.splits)), t1 = uniform((int)((int64_t)steps * (at.split + 1) / g.splits));

    Loader<T, BM, WAVES, A_BY_K> la;
    Loader<T, BN, WAVES, B_BY_K> lb;
    la.init(g.a, row0, wave, lane, g.k_steps, g.a.plane, t0, t1);
    lb.init(g.b, col0, wave, lane, g.k_steps, 0, t0, t1);
    const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem;
    const uint32_t lds_a = lds + wave * (la.N * 1024), lds_b = lds + BM * kStepBytes + wave * (lb.N * 1024);
    auto load = [&](int i, uint32_t half) {   // one of a step's loads
        if (i < la.N) la.load(i, lds_a + half);
        else lb.load(i - la.N, lds_b + half);
    };
    constexpr int LOADS = la.N + lb.N, FIRST = LOADS / 2;

    Acc acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    // A step is four sub-steps; each sub-step's fragments are read while the
    // one before is multiplied.  Before the last sub-step every wave has read
    // its half of LDS and the other half's loads are in: one barrier a step,
    // after which the half just read is filled for the step after the next.
    // The loads take two sub-steps, the last of this step and the first of the
    // next: 64 KB at 64 bytes a cycle are 1,024 cycles, two sub-steps' products.
    // (All in the one: 1,120 against 1,097 us, 16,384 x 32,768 x 1,024.)
    typename Frag<T>::type fa[2][TM], fb[2][TN];
    auto read = [&](int i, int half, int s, int to) {   // one of a sub-step's fragments
        const char* tile = smem + half * STAGE;
        if (i < TM) fa[to][i] = fragment<T, BM, A_BY_K>(tile, wm * TM + i, s, lane);
        else fb[to][i - TM] = fragment<T, BN, B_BY_K>(tile + BM * kStepBytes, wn * TN + i - TM, s, lane);
    };
    if (t0 < t1) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) load(i, 0);
        la.next();
        lb.next();
#pragma unroll
        for (int i = 0; i < FIRST; ++i) load(i, STAGE);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(FIRST) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
#pragma unroll
        for (int i = 0; i < TM + TN; ++i) read(i, 0, 0, 0);
    }
    for (int t = t0; t < t1; ++t) {
        const int half = (t - t0) & 1;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (s == 3) {
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
            }
            // between the sub-step's products: the next one's fragments, and after the barrier the loads
            constexpr int MMAS = TM * TN, READS = TM + TN;
#pragma unroll
            for (int n = 0; n < MMAS; ++n) {
                const int i = n / TN, j = n % TN;
                acc[i][j] = LANE_IS_ROW ? mma(fb[s & 1][j], fa[s & 1][i], acc[i][j]) : mma(fa[s & 1][i], fb[s & 1][j], acc[i][j]);
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
            if (s == 0) {
                la.next();
                lb.next();
            }
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // LDS is written to no longer

    // Value r of a 32 x 32 block's lane: the lane's row (column) is lane % 32,
    // the other place 8 (r / 4) + 4 (lane / 32) + r % 4.
    const int half = (lane >> 5) * 4;
    const int64_t m0 = row0 + wm * TM * 32, n0 = col0 + wn * TN * 32;
    if constexpr (WHAT == kStats) {
        const bool ragged = n0 + TN * 32 > g.limit;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int64_t row = m0 + i * 32 + (lane & 31);
            const bool live = row < g.m;
            if (g.target) {
                const int32_t target = live ? g.target[row] : -1;
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const int64_t to = (int64_t)target - n0 - j * 32;
                    if (__ballot((uint64_t)to < 32u)) {
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            if (to == 8 * (r / 4) + half + r % 4 && target < g.limit) g.hit[row] = acc[i][j][r] * g.scale;
                    }
                }
            }
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float v = acc[i][j][r] * g.scale;
                    if (ragged && n0 + j * 32 + 8 * (r / 4) + half + r % 4 >= g.limit) v = -INFINITY;
                    acc[i][j][r] = v;
                    top = fmaxf(top, v);
                }
            top = fmaxf(top, swap_halves(top));
            const float from = top == -INFINITY ? 0.0f : top;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) sum += __builtin_amdgcn_exp2f(acc[i][j][r] - from);
            sum += swap_halves(sum);
            if (live && lane < 32) g.part[((int64_t)at.n * WN + wn) * g.m + row] = make_float2(top, sum);
        }
    } else if constexpr (WHAT == kGrad) {
        const float unit = g.unit[0];
        __syncthreads();   // the tiles in LDS are read
        char* strip = smem + wave * (32 * TN * 32 * (int)sizeof(T));
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int64_t row = m0 + i * 32 + (lane & 31);
            const bool live = row < g.m;
            const float rate = live ? g.rate[row] * unit : 0.0f;
            const float lse = live ? g.lse[row] : 0.0f;
            const int64_t target = live && g.target ? (int64_t)g.target[row] - g.first : -1;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int64_t col = n0 + j * 32 + 8 * (r / 4) + half + r % 4;
                    const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][r], g.scale, -lse) * kLog2e);
                    const float d = rate * (col == target ? p - 1.0f : p);
                    acc[i][j][r] = rate != 0.0f && col < g.limit ? d : 0.0f;
                }
            T* to = (T*)g.dz + (m0 + i * 32) * g.dz_stride + n0;
            store_strip<T, TN>(acc[i], strip, lane, (int)min((int64_t)32, g.m - m0 - i * 32), to, g.dz_stride);
            if (g.dz_plane) {   // what the rounding left
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[i][j][r] -= (float)(T)acc[i][j][r];
                store_strip<T, TN>(acc[i], strip, lane, (int)min((int64_t)32, g.m - m0 - i * 32), to + g.dz_plane, g.dz_stride);
            }
        }
    } else {
        const float factor = WHAT == kOut && g.factor ? g.factor[0] : 1.0f;
        const int64_t col = n0 + (lane & 31);
        const int cols = (int)min((int64_t)(TN * 32), g.n - col);   // of the lane's, 32 apart
        auto store = [&](auto* out, int64_t stride, bool add) {
#pragma unroll
            for (int i = 0; i < TM; ++i) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int64_t row = m0 + i * 32 + 8 * (r / 4) + half + r % 4;
                    if (row < g.m) {
                        auto* to = out + row * stride + col;
#pragma unroll
                        for (int j = 0; j < TN; ++j)
                            if (j * 32 < cols) {
                                const float v = acc[i][j][r] * factor;
                                to[j * 32] = (std::remove_reference_t<decltype(*to)>)(add ? (float)to[j * 32] + v : v);
                            }
                    }
                    __builtin_amdgcn_sched_barrier(0);   // else all rows' addresses are made first
                }
            }
        };
        if constexpr (WHAT == kSum) store(g.sum + (int64_t)at.split * g.m * g.sum_stride, g.sum_stride, g.add);
        else if (g.out_type == HGB_F32) store((float*)g.out, g.out_stride, false);
        else store((T*)g.out, g.out_stride, false);
    }
}

// Rows copied to where they start at 16 bytes, with zeros behind their end,
// and instead of rows whose rate is zero.
template <typename T>
__global__ __launch_bounds__(256) void k_head_copy(const T* x, int64_t stride, int64_t n, int dim, int dp, const float* rate,
                                                   T* out)
{
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

// Each row's rate, the factor of its logits' gradient (zero without one), and
// what the gradient is multiplied by for its type: fp16 holds values of 2^-24
// to 2^16, and a rate times a probability is often less than the former, so
// the largest rate is brought between 2^14 and 2^15.  Powers of two: exact.
// One block.
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
    int half;              // fp16
    float* rate;           // [n], then the factor and one over it
    uint32_t* err;
};

__device__ inline float teacher_at(const void* p, int type, int64_t i)
{
    return type == HGB_F32 ? ((const float*)p)[i] : type == HGB_BF16 ? (float)((const __bf16*)p)[i] : (float)((const _Float16*)p)[i];
}

__global__ __launch_bounds__(1024) void k_head_rate(const RateArgs a)
{
    __shared__ float most[16];
    float top = 0.0f;
    bool bad = false;
    for (int64_t i = threadIdx.x; i < a.n; i += 1024) {
        bool live = false;
        for (int k = 0; k < a.top; ++k) {
            const int32_t t = a.token[i * a.top + k];
            const bool in = t >= 0 && t < a.vocab && t != a.pad;
            if (!in && t != a.pad) bad = true;
            live = live || (in && (!a.teacher || teacher_at(a.teacher, a.teacher_type, i * a.top + k) != -INFINITY));
        }
        const float r = live ? a.grad[i] * a.scale : 0.0f;
        a.rate[i] = r;
        top = fmaxf(top, fabsf(r));
    }
    if (bad) atomicOr(a.err, kVecErrToken);
    for (int s = 32; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor(top, s));
    if ((threadIdx.x & 63) == 0) most[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 0; w < 16; ++w) top = fmaxf(top, most[w]);
        int e = 0;   // top in [2^(e - 1), 2^e)
        if (a.half && top > 0.0f && top < INFINITY) (void)frexpf(top, &e);
        e = a.half ? max(-100, min(100, 15 - e)) : 0;
        a.rate[a.n] = ldexpf(1.0f, e);
        a.rate[a.n + 1] = ldexpf(1.0f, -e);
    }
}

// A sum's shares added up: rows of zero rate are zero.
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
    float t[kTeacherSlots];   // teacher / T - max
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
                w.t[i] = teacher_at(a.teacher, a.teacher_type, row * a.top + k) / a.heat;
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
        w.t[i] = w.t[i] == -INFINITY ? -INFINITY : w.t[i] - top;
        w.p[i] = expf(w.t[i]);
        sum += w.p[i];
    }
    sum = group_sum(sum, 6);
    w.log_sum = logf(sum);
#pragma unroll
    for (int i = 0; i < kTeacherSlots; ++i) w.p[i] /= sum;
    return w;
}

// The student's logits at the teacher's tokens: a wave a slot.
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
            if (dz_plane) at[dz_plane] = (T)(d - (float)(T)d);
        }
    }
}

}  // namespace hgb
