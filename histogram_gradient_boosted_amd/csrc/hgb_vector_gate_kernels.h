// Device kernels of the gate (gfx950): each row's experts, their shares, and
// the logits' gradient.  Internal header: included by hgb_vector_gate.hip only.
#pragma once

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
    int groups, keep, best;
    int top;
    int renormalise;
    float scale;
    int log_group;
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

// Reductions over the 2^log_group lanes that share a row.
template <typename K, typename F>
__device__ inline K row_reduce(K x, int log_group, F f)
{
    for (int s = 1; s < (1 << log_group); s *= 2) x = f(x, __shfl_xor(x, s));
    return x;
}
template <typename K>
__device__ inline K row_max(K x, int log_group)
{
    return row_reduce(x, log_group, [](K a, K b) { return a > b ? a : b; });
}
template <typename K>
__device__ inline K row_sum(K x, int log_group)
{
    return row_reduce(x, log_group, [](K a, K b) { return a + b; });
}

// A logit as the gate takes it: NaN and +infinity are masked, and reported.
__device__ inline float gate_logit(float l, bool* bad)
{
    if (l < INFINITY) return l;
    *bad = true;
    return -INFINITY;
}

// 2^log_group lanes a row, V experts in each.
template <typename T, int V>
__global__ __launch_bounds__(256) void k_gate(const GateArgs g)
{
    typedef double K;   // of the keys
    extern __shared__ __align__(16) char smem[];
    const int lanes = 1 << g.log_group, l = threadIdx.x & (lanes - 1), in_block = threadIdx.x >> g.log_group;
    const int64_t row = (int64_t)block_number() * (256 >> g.log_group) + in_block;
    const bool live = row < g.n;
    const K low = -(K)INFINITY;
    const int first = l * V;
    bool bad = false;

    float z[V];
    load_vals<V>(z, (const T*)g.logits + (live ? row : 0) * g.stride + first, live ? g.experts - first : 0);
    float most = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        z[j] = first + j < g.experts && live ? gate_logit(z[j], &bad) : -INFINITY;
        most = fmaxf(most, z[j]);
    }
    most = row_max(most, g.log_group);

    K key[V];
    const bool plain = !g.bias && g.groups == 1;   // the scores are in the logits' order
    if (plain) {
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = z[j];
    } else {
        K sum = 0;
        if (g.score == HGB_SOFTMAX) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                key[j] = z[j] == -INFINITY ? (K)0 : exp((K)z[j] - (K)most);
                sum += key[j];
            }
            sum = row_sum(sum, g.log_group);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (g.score == HGB_SOFTMAX) key[j] /= sum;
            else key[j] = 1 / (1 + exp(-(K)z[j]));
            const float b = g.bias && first + j < g.experts ? gate_logit(g.bias[first + j], &bad) : 0.0f;
            key[j] = z[j] == -INFINITY ? low : key[j] + (K)b;
        }
    }
    if (g.groups > 1) {
        K* worth = (K*)smem + in_block * g.groups;
        const int per = g.experts / g.groups;
        for (int q = 0; q < g.groups; ++q) {
            K a = low, b = low;   // the largest two of the group
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int e = first + j;
                if (e < q * per || e >= (q + 1) * per) continue;
                if (key[j] > a) {
                    b = a;
                    a = key[j];
                } else if (key[j] > b) {
                    b = key[j];
                }
            }
            for (int s = 1; s < lanes; s *= 2) {
                const K c = __shfl_xor(a, s), d = __shfl_xor(b, s);
                b = a > c ? (b > c ? b : c) : (a > d ? a : d);
                a = a > c ? a : c;
            }
            if (l == 0) worth[q] = g.best == 1 ? a : a + b;
        }
        __syncthreads();
        // a value's group is kept if fewer than `keep` come before it
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (first + j >= g.experts) continue;
            const int q = (first + j) / per;
            const K mine = worth[q];
            int before = 0;
            for (int o = 0; o < g.groups; ++o) before += worth[o] > mine || (worth[o] == mine && o < q);
            if (before >= g.keep) key[j] = low;
        }
    }

    int rank[V];
#pragma unroll
    for (int j = 0; j < V; ++j) rank[j] = -1;
    int found = 0;
    const int base = (threadIdx.x & 63) & ~(lanes - 1);   // the row's first lane in the wave
    for (; found < g.top; ++found) {
        K mine = low;
        int at = -1;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (key[j] > mine) {
                mine = key[j];
                at = j;
            }
        const K best = row_max(mine, g.log_group);
        const bool any = best > low;
        const uint64_t owners = __ballot(any && mine == best) >> base;
        if (!__ballot(any)) break;
        const int owner = __ffsll((unsigned long long)(lanes == 64 ? owners : owners & ((1ull << lanes) - 1))) - 1;
        if (any && owner == l) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j == at) {
                    key[j] = low;
                    rank[j] = found;
                }
        }
    }

    // shares, from the chosen logits
    float s[V], sum = 0.0f, high = -INFINITY;
    int count = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (rank[j] >= 0) {
            high = fmaxf(high, z[j]);
            ++count;
        }
    high = row_max(high, g.log_group);
    count = row_sum(count, g.log_group);
    float whole = 0.0f;
    if (!g.renormalise && g.score == HGB_SOFTMAX) {
#pragma unroll
        for (int j = 0; j < V; ++j) whole += z[j] == -INFINITY ? 0.0f : expf(z[j] - most);
        whole = row_sum(whole, g.log_group);
        high = most;
    }
    // 1 / (1 + exp(-z)) is exp(z) to 32 bits below -17, and need not underflow in a ratio
    const bool ratio = g.score == HGB_SOFTMAX || (g.renormalise && high < -17.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        s[j] = rank[j] < 0 ? 0.0f : ratio ? expf(z[j] - high) : 1.0f / (1.0f + expf(-z[j]));
        sum += s[j];
    }
    sum = row_sum(sum, g.log_group);
    const float by = g.renormalise ? sum : g.score == HGB_SOFTMAX ? whole : 1.0f;
    if (live) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (rank[j] >= 0) {
                g.chosen[row * g.top + rank[j]] = first + j;
                g.share[row * g.top + rank[j]] = g.scale * (s[j] / by);
            }
        for (int k = count + l; k < g.top; k += lanes) {
            g.chosen[row * g.top + k] = -1;
            g.share[row * g.top + k] = 0.0f;
        }
    }
    if (bad) atomicOr(g.err, kVecErrScore);
}

// The lanes of a row first take its slots side by side, whose gradients meet
// the experts in LDS, then the experts.
template <typename T, int V>
__global__ __launch_bounds__(256) void k_gate_grad(const GateGradArgs g)
{
    extern __shared__ __align__(16) char smem[];
    const int lanes = 1 << g.log_group, l = threadIdx.x & (lanes - 1), in_block = threadIdx.x >> g.log_group;
    const int64_t row = (int64_t)block_number() * (256 >> g.log_group) + in_block;
    const bool live = row < g.n;
    const int first = l * V, width = V << g.log_group;
    float* ds = (float*)smem + in_block * width;
    const T* logits = (const T*)g.logits + row * g.stride;
    bool bad = false, other = false;

    float z[V], most = -INFINITY, sum = 0.0f;
    const bool dense = g.score == HGB_SOFTMAX && !g.renormalise;   // every logit has a gradient
    if (dense) {
        load_vals<V>(z, live ? logits + first : (const T*)g.logits, live ? g.experts - first : 0);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            z[j] = live && first + j < g.experts ? gate_logit(z[j], &other) : -INFINITY;
            most = fmaxf(most, z[j]);
        }
        most = row_max(most, g.log_group);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            z[j] = z[j] == -INFINITY ? 0.0f : expf(z[j] - most);
            sum += z[j];
        }
        sum = row_sum(sum, g.log_group);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) ds[first + j] = 0.0f;
    __syncthreads();

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
        high = row_max(high, g.log_group);
    }
    const bool ratio = g.score == HGB_SOFTMAX || (g.renormalise && high < -17.0f);
    auto score = [&](float v) { return v == -INFINITY ? 0.0f : ratio ? expf(v - high) : 1.0f / (1.0f + expf(-v)); };
    if (!dense && g.renormalise) {
        by = 0.0f;
        for (int k = l; k < g.top; k += lanes) {
            int32_t e;
            by += score(slot(k, &e));
        }
        by = row_sum(by, g.log_group);
    }
    if (g.score == HGB_SIGMOID && !g.renormalise) by = 1.0f;
    const float over = by > 0.0f ? 1.0f / by : 0.0f;
    if (g.renormalise || dense) {
        for (int k = l; k < g.top; k += lanes) {
            int32_t e;
            const float s = score(slot(k, &e)) * over;
            if (s > 0.0f) dot = __builtin_fmaf(g.grad[row * g.top + k], s, dot);
        }
        dot = row_sum(dot, g.log_group);
    }
    for (int k = l; k < g.top; k += lanes) {
        int32_t e;
        const float v = slot(k, &e);
        if (v == -INFINITY) continue;
        float d = g.grad[row * g.top + k];
        if (!dense) {
            d = (d - dot) * (score(v) * over);
            if (g.score == HGB_SIGMOID) d *= 1.0f / (1.0f + expf(v));   // 1 - s
        }
        atomicAdd(ds + e, d);
    }
    __syncthreads();
    float out[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float d = ds[first + j];
        out[j] = g.scale * (dense ? (z[j] == 0.0f ? 0.0f : (d - dot) * (z[j] * over)) : d);
    }
    if (live) store_vals<V>(out, (T*)g.out + row * g.out_stride + first, g.experts - first);
    if (bad) atomicOr(g.err, kVecErrExpert);
}

}  // namespace hgb
