// Argument checks that the vector verbs' entry points share.
#pragma once

#include "hgb.h"
#include "hgb_ctx.h"
#include "hgb_vector_plan.h"

#include <initializer_list>
#include <numeric>

namespace hgb {

inline int elem_size(int32_t type) { return type == HGB_F32 ? 4 : 2; }
inline bool is_type(int32_t type) { return type == HGB_F32 || type == HGB_BF16 || type == HGB_F16; }

// A matrix argument's pointer, type and row stride.
inline hgb_status check_rows(hgb_ctx* c, const char* verb, const char* name, const void* p, int32_t type, int64_t rows,
                             int64_t dim, int64_t stride)
{
    if (!is_type(type)) return fail(c, HGB_E_INVALID, "%s: %s has an unknown type %d", verb, name, type);
    if (stride < dim) return fail(c, HGB_E_INVALID, "%s: %s's rows overlap (stride %lld below %lld values)", verb, name,
                                  (long long)stride, (long long)dim);
    if (stride > ((int64_t)1 << 40)) return fail(c, HGB_E_INVALID, "%s: %s's stride is too large", verb, name);
    if (rows > 0 && !p) return fail(c, HGB_E_INVALID, "%s: %s is null", verb, name);
    if ((uintptr_t)p % elem_size(type)) return fail(c, HGB_E_INVALID, "%s: %s is not aligned to its type", verb, name);
    return HGB_OK;
}

// The bytes of an argument: `rows` runs of `width`, `step` apart.
struct Span {
    const char* begin;
    int64_t width;
    int64_t rows = 1, step = 0;
};

inline Span span(const void* p, int32_t type, int64_t rows, int64_t dim, int64_t stride)
{
    const int64_t size = elem_size(type);
    if (!p || rows < 1) return {(const char*)p, 0};
    if (rows == 1 || stride == dim) return {(const char*)p, rows * dim * size};
    return {(const char*)p, dim * size, rows, stride * size};
}

inline Span span(const int32_t* p, int64_t n) { return {(const char*)p, p ? n * 4 : 0}; }
inline Span span(const float* p, int64_t n) { return {(const char*)p, p ? n * 4 : 0}; }

// Whether two arguments share a byte.  Where both extents meet, their rows may
// still lie side by side: with g the greatest divisor of both steps, every row
// of a is at begin(a) modulo g and every row of b at begin(b), so that they are
// apart if one row of each is, on a ring of g bytes.  That finds every overlap,
// and nothing else where the steps are equal or one argument is a single run.
inline bool overlap(const Span& a, const Span& b)
{
    if (a.width < 1 || b.width < 1) return false;
    const auto extent = [](const Span& s) { return (__int128)(s.rows - 1) * s.step + s.width; };
    const __int128 ahead = (__int128)(intptr_t)b.begin - (intptr_t)a.begin;   // of a's first byte
    if (ahead >= extent(a) || -ahead >= extent(b)) return false;
    const int64_t g = a.rows == 1 ? b.step : b.rows == 1 ? a.step : std::gcd(a.step, b.step);
    if (g == 0) return true;
    const int64_t at = (int64_t)((ahead % g + g) % g);
    return at < a.width || at + b.width > g;
}

// No output overlaps an input or another output; a workspace counts as an output.
inline hgb_status check_apart(hgb_ctx* c, const char* verb, std::initializer_list<Span> outs, std::initializer_list<Span> ins)
{
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const Span& in : ins)
            if (overlap(*o, in)) return fail(c, HGB_E_INVALID, "%s: an output overlaps an input", verb);
        for (auto other = outs.begin(); other != o; ++other)
            if (overlap(*o, *other)) return fail(c, HGB_E_INVALID, "%s: an output overlaps another", verb);
    }
    return HGB_OK;
}

// Pointers to 32-bit values are aligned to them.
inline hgb_status check_words(hgb_ctx* c, const char* verb, std::initializer_list<const void*> words)
{
    for (const void* p : words)
        if ((uintptr_t)p % 4) return fail(c, HGB_E_INVALID, "%s: a pointer is not aligned to 4 bytes", verb);
    return HGB_OK;
}

inline hgb_status check_dim(hgb_ctx* c, const char* verb, int64_t rows, int64_t dim)
{
    if (rows < 0 || rows > kVecMaxRows)
        return fail(c, HGB_E_INVALID, "%s: %lld rows are outside [0, 2^31)", verb, (long long)rows);
    if (dim < 1) return fail(c, HGB_E_INVALID, "%s: dim must be positive", verb);
    if (dim > kVecMaxDim) return fail(c, HGB_E_UNSUPPORTED, "%s: dim is above %lld", verb, (long long)kVecMaxDim);
    return HGB_OK;
}

inline hgb_status check_workspace(hgb_ctx* c, const char* verb, const void* p, int64_t have, int64_t need)
{
    if (need > 0 && (!p || have < need))
        return fail(c, HGB_E_INVALID, "%s: the workspace holds %lld bytes, needs %lld", verb, (long long)(p ? have : 0),
                    (long long)need);
    if ((uintptr_t)p % 16) return fail(c, HGB_E_INVALID, "%s: the workspace is not aligned to 16 bytes", verb);
    return HGB_OK;
}

#define HGB_TRY(expr)                      \
    do {                                   \
        hgb_status s_ = (expr);            \
        if (s_ != HGB_OK) return s_;       \
    } while (0)

// Runs an entry point's body: no C++ exception leaves the library.
template <typename F>
hgb_status guarded(hgb_ctx* c, F&& body)
{
    if (!c) return HGB_E_INVALID;
    try {
        c->err.clear();
        return body();
    } catch (...) {
        return HGB_E_DEVICE;
    }
}

// f with a null pointer of the type's element, so that generic code names it.
template <typename F>
hgb_status by_type(int32_t type, F&& f)
{
    if (type == HGB_F32) return f((float*)nullptr);
    if (type == HGB_BF16) return f((__bf16*)nullptr);
    return f((_Float16*)nullptr);
}

}  // namespace hgb
