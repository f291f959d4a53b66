// Device kernels of the gate (gfx950): each row's experts, their shares, and
// the logits' gradient.  Internal header: included by hgb_vector_gate.hip only.
#pragma once

#include <float.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hgb_ctx.h"
#include "hgb_vector_head_plan.h"
#include "hgb_vector_rows.h"

namespace hgb {

struct GateArgs {
    const void* logits;
    int64_t stride;
    int64_t n;
    int experts;
    int score;          // hgb_score
    const float* bias;
    int groups, keep, best, per;   // per: a group's experts
    int top;
    int renormalise;
    float scale;
    int log_group;
    int wave_bytes;
    int32_t* chosen;
    float* share;
    uint32_t* err;
};

struct GateGradArgs {
    const float* grad;
    const void* logits;
    int64_t stride;
    int64_t n;
    int experts;
    int score;
    const int32_t* chosen;
    int top;
    int renormalise;
    float scale;
    int log_group;
    void* out;
    int64_t out_stride;
    uint32_t* err;
};

// A logit as the gate takes it: NaN and +infinity are masked, and reported.
__device__ inline float gate_logit(float l, bool* bad)
{
    if (l < INFINITY) return l;
    *bad = true;
    return -INFINITY;
}

// The largest over the 2^log_group lanes of a row, which every lane gets: moves
// in the vector unit, no trips through LDS as a shuffle makes.
template <int CTRL>
__device__ inline uint32_t dpp_max(uint32_t x)
{
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true));
}

__device__ inline uint32_t lanes_max(uint32_t x, int log_group)
{
    if (log_group > 0) x = dpp_max<0xb1>(x);    // lanes 1, 0, 3, 2 of a quad
    if (log_group > 1) x = dpp_max<0x4e>(x);    // lanes 2, 3, 0, 1
    if (log_group > 2) x = dpp_max<0x141>(x);   // the other quad of eight, mirrored
    if (log_group > 3) x = dpp_max<0x140>(x);   // the other eight of sixteen
    if (log_group > 4) {
        const auto v = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        x = max(v[0], v[1]);
    }
    if (log_group > 5) {
        const auto v = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        x = max(v[0], v[1]);
    }
    return x;
}

// Floats in the order of unsigned numbers; 0 is below all of them.
__device__ inline uint32_t ordered(float v)
{
    const uint32_t u = __float_as_uint(v);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ inline float unordered(uint32_t o)
{
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// The largest of a wave's, the first among equals.
__device__ __forceinline__ void wave_first(double* best, int* at)
{
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
        const double other = __shfl_xor(*best, s);
        const int where = __shfl_xor(*at, s);
        const bool take = other > *best || (other == *best && where < *at);
        *best = take ? other : *best;
        *at = take ? where : *at;
    }
}

// The chosen experts of one row in order into list[0 .. top), by keys in 64
// bits and by a whole wave: key[experts] and worth[groups] in LDS are its own.
// Returns how many.  2 us a row of 256 experts, 8 of them in order, one row of
// the wave after the other: the last wave of a call may run it.
template <typename T>
__device__ __forceinline__ int choose_exactly(const GateArgs& g, const T* logits, float most, double* key, double* worth, int32_t* list)
{
    const int lane = threadIdx.x & 63, experts = g.experts;
    const double low = -(double)INFINITY;
    const bool by_logit = !g.bias && g.groups == 1;   // the scores are in the logits' order
    const bool sigmoid = g.score == HGB_SIGMOID;
    bool bad = false;
    double sum = 0;
    wave_order();
#pragma unroll 4
    for (int e = lane; e < experts; e += 64) {
        const float z = gate_logit((float)logits[e], &bad);
        double s = z;
        if (!by_logit && z != -INFINITY) sum += s = exp(sigmoid ? -s : s - (double)most);
        key[e] = z == -INFINITY ? low : s;   // exp is never -infinity
    }
    if (!by_logit) {
        if (!sigmoid) {
#pragma unroll 1
            for (int s = 1; s < 64; s *= 2) sum += __shfl_xor(sum, s);
        }
#pragma unroll 1
        for (int e = lane; e < experts; e += 64) {
            const double s = key[e], b = g.bias ? gate_logit(g.bias[e], &bad) : 0.0f;
            key[e] = s == low ? low : (sigmoid ? 1 : s) / (sigmoid ? 1 + s : sum) + b;
        }
    }
    wave_order();
    if (g.groups > 1) {
        const int per = g.per;
#pragma unroll 1
        for (int q = lane; q < g.groups; q += 64) {
            double a = low, b = low;   // the largest two of the group
#pragma unroll 8
            for (int e = q * per; e < (q + 1) * per; ++e) {
                const double x = key[e], under = x < a ? x : a;
                a = x > a ? x : a;
                b = under > b ? under : b;
            }
            worth[q] = g.best == 1 ? a : a + b;
        }
        wave_order();
#pragma unroll 1
        for (int q = lane; q < g.groups; q += 64) {
            int before = 0;
#pragma unroll 1
            for (int o = 0; o < g.groups; ++o) before += worth[o] > worth[q] || (worth[o] == worth[q] && o < q);
            if (before >= g.keep)
#pragma unroll 1
                for (int e = q * per; e < (q + 1) * per; ++e) key[e] = low;
        }
        wave_order();
    }
    int k = 0;
#pragma unroll 1
    for (; k < g.top; ++k) {
        double best = low;
        int at = experts;
#pragma unroll 4
        for (int e = lane; e < experts; e += 64) {
            const bool take = key[e] > best;
            best = take ? key[e] : best;
            at = take ? e : at;
        }
        wave_first(&best, &at);
        if (!(best > low)) break;
        if (lane == 0) {
            key[at] = low;
            list[k] = at;
        }
        wave_order();
    }
    return k;
}

// 2^log_group lanes a row, V experts in each.
//
// The choice is by 32-bit keys, which carry the expert's number in their low
// bits, so that one maximum finds both: where 16-bit logits decide alone, the
// whole number, and the order is exact.  Elsewhere the number within the lane,
// cut from the key's precision, and two keys that follow each other in a row's
// order may be closer than their error:
//   the cut        V 2^-23 |key|, of a key among the smallest numbers V 2^-149
//   a softmax      27 2^-24 of the row's largest, 1 / sum: exp of a difference
//                  d by exp2 is off by (2 |d| + 2) 2^-24 with |d| e^-|d| < 0.4,
//                  the sum by 20 roundings, the quotient by 3
//   a sigmoid      3 2^-24: s (1 - s) (2 |z| + 2) < 1, and two roundings
// and the sum with the bias 2^-24 |key|.  Such a row is chosen again by its
// whole wave in 64 bits: about one in 1,300 of 256 distinct 32-bit logits, but
// one in three of 256 logits of bf16 whose keys are equal where they are (with
// groups, or a bias of zeros).  Bound by vector instructions: a row of 256
// costs a wave about 300, half of them for the 9 maxima.  32,768 rows of 256, 8
// of them out of 4 of 8 groups: 38 to 49 us, as the last wave falls, 27 without
// the rows that are chosen again, with 64-bit keys throughout 103; bf16 without
// a bias 109, logits that are all equal 130.
template <typename T, int V>
__global__ __launch_bounds__(256) void k_gate(const GateArgs g)
{
    extern __shared__ __align__(16) char smem[];
    const int log_group = g.log_group, lanes = 1 << log_group, l = threadIdx.x & (lanes - 1), first = l * V;
    const int in_block = threadIdx.x >> log_group, rows = 256 >> log_group;
    const int64_t row = (int64_t)block_number() * rows + in_block;
    const bool live = row < g.n;
    const T* logits = (const T*)g.logits + (live ? row : 0) * g.stride;
    const bool by_logit = !g.bias && g.groups == 1, whole = by_logit && sizeof(T) < 4;
    const int wave = threadIdx.x >> 6, in_wave = (threadIdx.x & 63) >> log_group, wave_rows = 64 >> log_group;
    // LDS: the rows' choices, then each wave's own
    int32_t* list = (int32_t*)smem + in_block * g.top;
    char* own = smem + gate_list_bytes(rows, g.top) + wave * g.wave_bytes;
    bool bad = false;

    float z[V], most = -INFINITY;
    load_vals<V>(z, logits + first, live ? g.experts - first : 0);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        z[j] = live && first + j < g.experts ? gate_logit(z[j], &bad) : -INFINITY;
        most = fmaxf(most, z[j]);
    }
    most = unordered(lanes_max(ordered(most), log_group));

    uint32_t key[V];
    constexpr uint32_t kNone = 0x007fffffu;   // -infinity's, and what the number in its low bits makes of it
    float sum = 0.0f, slack = 0.0f;           // of softmax; how far two keys are off, besides by parts of theirs
    bool close = false;
    if (whole) {
#pragma unroll
        for (int j = 0; j < V; ++j)   // + 0: one zero.  A 16-bit value's float has the low 13 bits alike: 10 hold an expert
            key[j] = (ordered(z[j] + 0.0f) & ~1023u) | (uint32_t)(1023 - first - j);
    } else {
        float v[V];
        if (by_logit) {
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = z[j] + 0.0f;   // one zero
            slack = FLT_MIN;   // zeros tie, whatever the cut makes of them
        } else {
            float bias[V];
            if (g.bias) load_vals<V>(bias, g.bias + first, g.experts - first);
            if (g.score == HGB_SOFTMAX) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    v[j] = z[j] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((z[j] - most) * 1.44269504f);
                    sum += v[j];
                }
                sum = group_sum(sum, log_group);
                const float over = sum > 0.0f ? 1.0f / sum : 0.0f;
                slack = 54 * 0x1p-24f * over;
#pragma unroll
                for (int j = 0; j < V; ++j) v[j] *= over;
            } else {
                slack = 6 * 0x1p-24f;
#pragma unroll
                for (int j = 0; j < V; ++j) v[j] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z[j] * -1.44269504f));
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (g.bias) v[j] = gate_logit(v[j] + bias[j], &bad);   // a bad bias makes a bad sum
                if (z[j] == -INFINITY) v[j] = -INFINITY;
            }
        }
        if (g.groups > 1) {
            float* sums = (float*)own + in_wave * 2 * g.groups;
            int32_t* kept = (int32_t*)sums + g.groups;
            const int per = g.per;
            uint32_t big = 0;   // the row's largest |key|
#pragma unroll
            for (int j = 0; j < V; ++j) big = max(big, v[j] == -INFINITY ? 0 : __float_as_uint(v[j]) & 0x7fffffffu);
            // how far two groups' sums are off: four keys, and the sums' roundings
            const float off = 2 * slack + 8 * 0x1p-24f * __uint_as_float(lanes_max(big, log_group));
            const bool even = per % V == 0 && (per / V & (per / V - 1)) == 0;   // a group is the whole of 2^k lanes
            const int mine = first / per;
            // -infinity only where a key is: two finite keys may pass the lowest float
            auto worth = [&](float a, float b) { return g.best == 1 ? a : b == -INFINITY ? b : fmaxf(a + b, -FLT_MAX); };
            if (even) {
                float a = -INFINITY, b = -INFINITY;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    b = fmaxf(b, fminf(a, v[j]));
                    a = fmaxf(a, v[j]);
                }
                for (int s = 1; s < per / V; s *= 2) {
                    const float c = __shfl_xor(a, s), d = __shfl_xor(b, s);
                    b = fmaxf(fminf(a, c), fmaxf(b, d));
                    a = fmaxf(a, c);
                }
                if (first < g.experts) sums[mine] = worth(a, b);   // all its lanes the same
            } else {
                // One group after the other, each by all lanes: for few groups.
                // 32,768 rows, 16 experts chosen: 990 in 33 groups 0.49 ms, 1,008
                // in 63 (whole lanes) 0.24, 1,023 in 341 6.6, in 1,023 50.
                for (int q = 0; q < g.groups; ++q) {
                    float a = -INFINITY, b = -INFINITY;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const int e = first + j;
                        const float x = e >= q * per && e < (q + 1) * per ? v[j] : -INFINITY;
                        b = fmaxf(b, fminf(a, x));
                        a = fmaxf(a, x);
                    }
                    for (int s = 1; s < lanes; s *= 2) {
                        const float c = __shfl_xor(a, s), d = __shfl_xor(b, s);
                        b = fmaxf(fminf(a, c), fmaxf(b, d));
                        a = fmaxf(a, c);
                    }
                    if (l == 0) sums[q] = worth(a, b);
                }
            }
            wave_order();
            // kept: fewer than `keep` groups may come before; out: that many surely do
            for (int q = even ? mine : l; q < (even ? mine + 1 : g.groups) && q < g.groups; q += lanes) {
                const float own = sums[q];
                int may = 0, sure = 0;
                for (int o = 0; o < g.groups; ++o) {
                    const float other = sums[o];
                    // both of the lowest worth: a tie, which the order of the groups decides
                    const bool tie = own == -INFINITY && other == own;
                    may += tie ? o < q : o != q && other >= own - off;
                    sure += tie ? o < q : other > own + off;
                }
                close = close || (live && may >= g.keep && sure < g.keep);
                if (even) {
#pragma unroll
                    for (int j = 0; j < V; ++j) v[j] = may < g.keep ? v[j] : -INFINITY;
                } else {
                    kept[q] = may < g.keep;
                }
            }
            if (!even) {
                wave_order();
                int q = mine, in = first - q * per;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (in++ == per) {
                        in = 1;
                        ++q;
                    }
                    if (q < g.groups && !kept[q]) v[j] = -INFINITY;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = (ordered(v[j]) & ~(uint32_t)(V - 1)) | (uint32_t)(V - 1 - j);
    }

    int found = 0;
    float last = INFINITY;
    for (int k = 0; k < g.top + !whole; ++k) {   // one more: is it apart from the last?
        uint32_t mine = key[0];
#pragma unroll
        for (int j = 1; j < V; ++j) mine = max(mine, key[j]);
        const uint32_t best = lanes_max(mine, log_group);
        const bool any = best > kNone;
        const uint64_t rows_left = __ballot(any && l == 0);
        if (!rows_left) break;
        const bool owner = any && mine == best;
        if (!whole) {
            const float now = unordered(best);
            // more owners than rows: the same key in two lanes of one
            const bool twice = __popcll(__ballot(owner)) != __popcll(rows_left);
            close = close || twice || (any && last - now <= (V + 1) * 0x1p-23f * fabsf(now) + slack);
            last = now;
        }
        if (k < g.top) {
            if (owner) list[k] = whole ? 1023 - (int)(best & 1023) : first + V - 1 - (int)(best & (V - 1));
            found += any;
        }
        const uint32_t gone = owner ? best : 0;
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = key[j] == gone ? 0 : key[j];
    }
    if (!whole) {
        double* keys = (double*)own;
        for (uint64_t again = __ballot(close && live); again;) {   // row by row of the wave
            const int at = __ffsll((unsigned long long)again) - 1, r = at >> log_group;
            const T* its = (const T*)g.logits + (row - in_wave + r) * g.stride;
            const int n = choose_exactly<T>(g, its, __shfl(most, at), keys, keys + g.experts, (int32_t*)smem + (wave * wave_rows + r) * g.top);
            if (in_wave == r) found = n;
            again &= lanes == 64 ? 0 : ~(((1ull << lanes) - 1) << (r * lanes));
        }
    }

    // the shares: the lanes take the row's slots side by side
    wave_order();
    auto slot = [&](int k) { return (float)logits[list[k]]; };
    float high = most, by = sum;
    if (g.renormalise) {
        high = -INFINITY;
        for (int k = l; k < found; k += lanes) high = fmaxf(high, slot(k));
        high = unordered(lanes_max(ordered(high), log_group));
    } else if (g.score == HGB_SOFTMAX && by_logit) {
#pragma unroll
        for (int j = 0; j < V; ++j) by += z[j] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((z[j] - most) * 1.44269504f);
        by = group_sum(by, log_group);
    }
    // 1 / (1 + exp(-z)) is exp(z) to 32 bits below -17, and need not underflow in a ratio
    const bool ratio = g.score == HGB_SOFTMAX || (g.renormalise && high < -17.0f);
    auto score = [&](float v) { return ratio ? expf(v - high) : 1.0f / (1.0f + expf(-v)); };
    if (g.renormalise) {
        by = 0.0f;
        for (int k = l; k < found; k += lanes) by += score(slot(k));
        by = group_sum(by, log_group);
    } else if (g.score == HGB_SIGMOID) {
        by = 1.0f;
    }
    if (live)
        for (int k = l; k < g.top; k += lanes) {
            g.chosen[row * g.top + k] = k < found ? list[k] : -1;
            g.share[row * g.top + k] = k < found ? g.scale * (score(slot(k)) / by) : 0.0f;
        }
    if (bad) atomicOr(g.err, kVecErrScore);
}

// The lanes of a row first take its slots side by side, whose gradients meet
// the experts in LDS, then the experts, four or eight at a time next to each
// other (a lane's 16 in a row: 19 us instead of 12.5 for 32,768 x 256 fp32, LDS
// banks met four times).  Bound by its chain of looks at the slots (6 us for
// 32,768 x 64 bf16, 9.4 MB) and, from 256 experts on, by the bytes: 2.7 TB/s.
template <typename T, int V>
__global__ __launch_bounds__(256) void k_gate_grad(const GateGradArgs g)
{
    extern __shared__ __align__(16) char smem[];
    const int lanes = 1 << g.log_group, l = threadIdx.x & (lanes - 1), in_block = threadIdx.x >> g.log_group;
    const int64_t row = (int64_t)block_number() * (256 >> g.log_group) + in_block;
    const bool live = row < g.n;
    constexpr int W = V < kVals<T> ? V : kVals<T>;
    float* ds = (float*)smem + in_block * (V << g.log_group);
    auto expert = [&](int c) { return (c * lanes + l) * W; };   // the first of a lane's chunk c
    const T* logits = (const T*)g.logits + row * g.stride;
    bool bad = false, other = false;

    float z[V], most = -INFINITY, sum = 0.0f;
    const bool dense = g.score == HGB_SOFTMAX && !g.renormalise;   // every logit has a gradient
    if (dense) {
#pragma unroll
        for (int c = 0; c < V / W; ++c) {
            float part[W];
            load_vals<W>(part, live ? logits + expert(c) : (const T*)g.logits, live ? g.experts - expert(c) : 0);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                z[c * W + j] = live && expert(c) + j < g.experts ? gate_logit(part[j], &other) : -INFINITY;
                most = fmaxf(most, z[c * W + j]);
            }
        }
        most = unordered(lanes_max(ordered(most), g.log_group));
#pragma unroll
        for (int j = 0; j < V; ++j) {
            z[j] = z[j] == -INFINITY ? 0.0f : expf(z[j] - most);
            sum += z[j];
        }
        sum = group_sum(sum, g.log_group);
    }
#pragma unroll
    for (int c = 0; c < V / W; ++c)
#pragma unroll
        for (int j = 0; j < W; ++j) ds[expert(c) + j] = 0.0f;
    wave_order();

    // a slot's expert's logit, or -infinity
    auto slot = [&](int k, int32_t* e) {
        *e = live ? g.chosen[row * g.top + k] : -1;
        if (*e < 0 || *e >= g.experts) {
            if (*e != -1) bad = true;
            return -INFINITY;
        }
        return gate_logit((float)logits[*e], &other);
    };
    float high = most, by = sum, dot = 0.0f;
    if (!dense && g.renormalise) {
        for (int k = l; k < g.top; k += lanes) {
            int32_t e;
            high = fmaxf(high, slot(k, &e));
        }
        high = unordered(lanes_max(ordered(high), g.log_group));
    }
    const bool ratio = g.score == HGB_SOFTMAX || (g.renormalise && high < -17.0f);
    auto score = [&](float v) { return v == -INFINITY ? 0.0f : ratio ? expf(v - high) : 1.0f / (1.0f + expf(-v)); };
    if (!dense && g.renormalise) {
        by = 0.0f;
        for (int k = l; k < g.top; k += lanes) {
            int32_t e;
            by += score(slot(k, &e));
        }
        by = group_sum(by, g.log_group);
    }
    if (g.score == HGB_SIGMOID && !g.renormalise) by = 1.0f;
    const float over = by > 0.0f ? 1.0f / by : 0.0f;
    if (g.renormalise || dense) {
        for (int k = l; k < g.top; k += lanes) {
            int32_t e;
            const float s = score(slot(k, &e)) * over;
            if (s > 0.0f) dot = __builtin_fmaf(g.grad[row * g.top + k], s, dot);
        }
        dot = group_sum(dot, g.log_group);
    }
    // Gate names an expert once in a row, a caller may name it in several slots:
    // those are summed in the slots' order, which float atomics do not keep.  A
    // lane that does not find its own mark shares its expert.
    for (int first = 0; first < g.top; first += lanes) {
        const int k = first + l;
        int32_t e = -1;
        const float v = k < g.top ? slot(k, &e) : -INFINITY;
        const bool counts = v != -INFINITY;
        const float before = counts && first > 0 ? ds[e] : 0.0f;
        wave_order();
        if (counts) ds[e] = __int_as_float(l);
        float d = counts ? g.grad[row * g.top + k] : 0.0f;
        if (!dense && counts) {
            d = (d - dot) * (score(v) * over);
            if (g.score == HGB_SIGMOID) d *= 1.0f / (1.0f + expf(v));   // 1 - s
        }
        wave_order();
        float all = before + d;
        if (__ballot(counts && __float_as_int(ds[e]) != l)) {
            all = before;
            for (int j = 0; j < min(lanes, g.top - first); ++j) {
                const int named = __shfl(counts ? e : -1, j, lanes);
                const float add = __shfl(d, j, lanes);
                if (named == e) all += add;
            }
        }
        wave_order();
        if (counts) ds[e] = all;   // the lanes of one expert the same
        wave_order();
    }
#pragma unroll
    for (int c = 0; c < V / W; ++c) {
        float out[W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const float d = ds[expert(c) + j];
            out[j] = g.scale * (dense ? (z[c * W + j] == 0.0f ? 0.0f : (d - dot) * (z[c * W + j] * over)) : d);
        }
        if (live) store_vals<W>(out, (T*)g.out + row * g.out_stride + expert(c), g.experts - expert(c));
    }
    if (bad) atomicOr(g.err, kVecErrExpert);
}

}  // namespace hgb
