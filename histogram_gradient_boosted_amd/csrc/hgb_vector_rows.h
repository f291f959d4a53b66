// Rows of vectors in the vector verbs' kernels (gfx950): loads and stores of any
// alignment, and sums over groups of lanes.  Internal header.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

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

// Keeps a wave's accesses to LDS before and after in order.
__device__ inline void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
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

}  // namespace hgb
