// hgb: the vector verbs of the C ABI (see include/hgb.h for the contract):
// token embedding, layer norm and rows sorted by expert, with their gradients.
//
// Host side: argument checks and launches.  The kernels live in
// hgb_vector_kernels.h, the launch plans in hgb_vector_plan.h.  Nothing here
// allocates or waits: a verb's scratch is its caller's workspace, so calls may
// be captured into a graph.
#include "hgb.h"
#include "hgb_ctx.h"
#include "hgb_vector_kernels.h"
#include "hgb_vector_plan.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <initializer_list>
#include <numeric>
#include <type_traits>

using namespace hgb;

namespace {

int elem_size(int32_t type) { return type == HGB_F32 ? 4 : 2; }
bool is_type(int32_t type) { return type == HGB_F32 || type == HGB_BF16 || type == HGB_F16; }

// A matrix argument's pointer, type and row stride.
hgb_status check_rows(hgb_ctx* c, const char* verb, const char* name, const void* p, int32_t type, int64_t rows,
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

Span span(const void* p, int32_t type, int64_t rows, int64_t dim, int64_t stride)
{
    const int64_t size = elem_size(type);
    if (!p || rows < 1) return {(const char*)p, 0};
    if (rows == 1 || stride == dim) return {(const char*)p, rows * dim * size};
    return {(const char*)p, dim * size, rows, stride * size};
}

Span span(const int32_t* p, int64_t n) { return {(const char*)p, p ? n * 4 : 0}; }
Span span(const float* p, int64_t n) { return {(const char*)p, p ? n * 4 : 0}; }

// Whether two arguments share a byte.  Where both extents meet, their rows may
// still lie side by side: with g the greatest divisor of both steps, every row
// of a is at begin(a) modulo g and every row of b at begin(b), so that they are
// apart if one row of each is, on a ring of g bytes.  That finds every overlap,
// and nothing else where the steps are equal or one argument is a single run.
bool overlap(const Span& a, const Span& b)
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
hgb_status check_apart(hgb_ctx* c, const char* verb, std::initializer_list<Span> outs, std::initializer_list<Span> ins)
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
hgb_status check_words(hgb_ctx* c, const char* verb, std::initializer_list<const void*> words)
{
    for (const void* p : words)
        if ((uintptr_t)p % 4) return fail(c, HGB_E_INVALID, "%s: a pointer is not aligned to 4 bytes", verb);
    return HGB_OK;
}

hgb_status check_dim(hgb_ctx* c, const char* verb, int64_t rows, int64_t dim)
{
    if (rows < 0 || rows > kVecMaxRows)
        return fail(c, HGB_E_INVALID, "%s: %lld rows are outside [0, 2^31)", verb, (long long)rows);
    if (dim < 1) return fail(c, HGB_E_INVALID, "%s: dim must be positive", verb);
    if (dim > kVecMaxDim) return fail(c, HGB_E_UNSUPPORTED, "%s: dim is above %lld", verb, (long long)kVecMaxDim);
    return HGB_OK;
}

hgb_status check_workspace(hgb_ctx* c, const char* verb, const void* p, int64_t have, int64_t need)
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

// The pairs of a table's type and its vectors' type: the same, or 16 bits
// beside a 32-bit table.
bool is_pair(int32_t table, int32_t vec) { return table == vec || table == HGB_F32; }

template <typename F>
hgb_status by_pair(int32_t table, int32_t vec, F&& f)
{
    if (table == HGB_F32) return by_type(vec, [&](auto* v) { return f((float*)nullptr, v); });
    return by_type(vec, [&](auto* v) { return f(v, v); });
}

// f with the plan's values a lane and waves a row, and how the rows end in
// vectors of V, as types.
template <typename F>
void by_shape(const NormPlan& p, int64_t dim, int V, F&& f)
{
    auto shaped = [&](auto values, auto waves) {
        if (dim % V == 0) f(values, waves, std::integral_constant<int, kEven>());
        else f(values, waves, std::integral_constant<int, kBack>());
    };
    auto with = [&](auto values) {
        if (p.waves == 4) shaped(values, std::integral_constant<int, 4>());
        else shaped(values, std::integral_constant<int, 1>());
    };
    const std::integral_constant<int, 8> eight;
    const std::integral_constant<int, 1> one;
    if (p.waves == 16) shaped(std::integral_constant<int, 16>(), std::integral_constant<int, 16>());
    else if (p.values == 8 && dim < V) f(eight, one, std::integral_constant<int, kPart>());
    else if (p.values == 8) shaped(eight, one);
    else if (p.values == 16) with(std::integral_constant<int, 16>());
    else with(std::integral_constant<int, 32>());
}

// Whether a call that reads and writes `bytes` stores its rows past the caches
// (and loads past them what it reads once: the embedding gradient's rows, the
// sorted rows of the routing).  Above three quarters of the 256 MB of the
// memory-side cache, what is left there of the output must be written out
// beside a later kernel's reads.  In us, past the caches and not, bf16: embed of
// 3,670,016 tokens 81 and 152, then layer_norm of the same values 301 and 334
// together; of 1,835,008 tokens 129 and 173 together; of 917,504 tokens (a call
// of 118 MB) 71 and 64 together, so not below.  route_gather and route_combine
// of 32,768 rows of 1,024, four experts each, 116 and 158.
bool streams(int64_t bytes) { return bytes >= (int64_t)192 << 20; }

dim3 row_grid(const RowMap& m, int64_t rows)
{
    const GridSpan g = span_blocks(row_blocks(m, rows));
    return dim3(g.x, (unsigned)m.slices, g.z);
}

int log2_of(int p) { return 31 - __builtin_clz((unsigned)p); }

// Blocks for a zero fill of `bytes`: a wave's 16-byte stores 16 times over, at most two blocks a CU.
int zero_blocks(const hgb_ctx* c, int64_t bytes, int threads)
{
    return (int)std::min<int64_t>(2 * c->n_cu, vec_ceil(bytes, (int64_t)threads * 16 * 16));
}

template <int ITEMS>
hgb_status launch_sort_small(hgb_ctx* c, const SortIn& in, const SortOut& out, const SortPlan& p, const ZeroFill& z)
{
    const int threads = (int)std::max<int64_t>(std::max<int64_t>(64, p.radix), vec_up(vec_ceil(in.n, ITEMS), 64));
    const size_t lds = 4 * ((size_t)small_pair_words(p, ITEMS, threads) + (size_t)(threads / 64) * p.radix + p.radix + 16);
    if (lds > 65536) HGB_TRY(raise_lds(c, k_sort_small<ITEMS>));
    k_sort_small<ITEMS><<<1 + zero_blocks(c, z.rows * z.cols * z.elem, threads), threads, lds, c->stream>>>(in, out, p, z);
    HGB_LAUNCHED(c, "k_sort_small");
    return HGB_OK;
}

template <bool FIRST, int ITEMS>
hgb_status launch_scatter(hgb_ctx* c, const SortIn& in, const SortOut& out, const SortPlan& p, int shift,
                          const uint32_t* counts, const ZeroFill& z)
{
    const size_t lds = 4 * (scatter_pair_words(ITEMS) + (size_t)(kSortThreads / 64) * p.radix + 2 * (size_t)p.radix + 16);
    if (lds > 65536) HGB_TRY(raise_lds(c, k_sort_scatter<FIRST, ITEMS>));
    k_sort_scatter<FIRST, ITEMS><<<p.blocks + zero_blocks(c, z.rows * z.cols * z.elem, kSortThreads), kSortThreads, lds,
                                   c->stream>>>(in, out, p, shift, counts, z);
    HGB_LAUNCHED(c, "k_sort_scatter");
    return HGB_OK;
}

template <bool FIRST>
hgb_status launch_pass(hgb_ctx* c, const SortIn& in, const SortOut& out, const SortPlan& p, int shift, uint32_t* counts,
                       const ZeroFill& with_count, const ZeroFill& with_scatter)
{
    if (p.count) {
        const ZeroFill& z = with_count;
        k_sort_count<FIRST><<<p.blocks + zero_blocks(c, z.rows * z.cols * z.elem, kSortThreads), kSortThreads, 4 * p.row,
                              c->stream>>>(in, p, shift, counts, z);
        HGB_LAUNCHED(c, "k_sort_count");
    }
    if (p.items == 1) return launch_scatter<FIRST, 1>(c, in, out, p, shift, counts, with_scatter);
    if (p.items == 4) return launch_scatter<FIRST, 4>(c, in, out, p, shift, counts, with_scatter);
    return launch_scatter<FIRST, kSortItems>(c, in, out, p, shift, counts, with_scatter);
}

// The sort of in.tokens into `out` (out.to: into whichever of a and b the
// last pass writes; returned in *sorted), and the zeros beside it: an equal
// part of their rows with each launch, so that the fill hides the sort's waits.
hgb_status launch_sort(hgb_ctx* c, SortIn in, SortOut out, const SortPlan& p, const ZeroFill& z, uint32_t* counts, uint2* a,
                       uint2* b, const uint2** sorted)
{
    if (p.small) {
        if (a) out.to = a;
        if (sorted) *sorted = a;
        return p.items == 1 ? launch_sort_small<1>(c, in, out, p, z) : launch_sort_small<4>(c, in, out, p, z);
    }
    const int launches = p.passes * (p.count ? 2 : 1);
    auto part = [&](int launch) {
        const int64_t first = z.rows * launch / launches, end = z.rows * (launch + 1) / launches;
        ZeroFill r = z;
        r.out = (char*)z.out + first * z.stride * z.elem;
        r.rows = end - first;
        return r;
    };
    for (int pass = 0; pass < p.passes; ++pass) {
        const int shift = pass * p.bits, launch = p.count ? 2 * pass : pass;
        const ZeroFill one = part(launch), two = p.count ? part(launch + 1) : one;
        if (a) out.to = pass & 1 ? b : a;
        if (pass == 0) {
            HGB_TRY(launch_pass<true>(c, in, out, p.pass(pass), shift, counts, one, two));
        } else {
            in.from = pass & 1 ? a : b;
            HGB_TRY(launch_pass<false>(c, in, out, p.pass(pass), shift, counts, one, two));
        }
    }
    if (sorted) *sorted = out.to;
    return HGB_OK;
}

}  // namespace

extern "C" {

hgb_status hgb_embed(hgb_ctx* c, const void* table, int32_t table_type, int64_t table_stride, int64_t vocab, int64_t dim,
                     const int32_t* tokens, int64_t n_tokens, int32_t pad, float scale, void* out, int32_t out_type,
                     int64_t out_stride)
{
    return guarded(c, [&]() -> hgb_status {
        HGB_TRY(check_dim(c, "embed", n_tokens, dim));
        if (vocab < 1 || vocab > kVecMaxVocab) return fail(c, HGB_E_INVALID, "embed: vocab is outside [1, 2^31 - 2]");
        HGB_TRY(check_rows(c, "embed", "table", table, table_type, vocab, dim, table_stride));
        HGB_TRY(check_rows(c, "embed", "out", out, out_type, n_tokens, dim, out_stride));
        if (!is_pair(table_type, out_type))
            return fail(c, HGB_E_UNSUPPORTED, "embed: out has the table's type, or 16 bits beside a 32-bit table");
        if (n_tokens > 0 && !tokens) return fail(c, HGB_E_INVALID, "embed: tokens is null");
        HGB_TRY(check_words(c, "embed", {tokens}));
        HGB_TRY(check_apart(c, "embed", {span(out, out_type, n_tokens, dim, out_stride)},
                            {span(table, table_type, vocab, dim, table_stride), span(tokens, n_tokens)}));
        if (n_tokens == 0) return HGB_OK;
        HGB_HIP(c, hipSetDevice(c->device));
        ProfScope ps(c, HGB_KERNEL_EMBED);
        return by_pair(table_type, out_type, [&](auto* t, auto* u) -> hgb_status {
            using T = std::remove_pointer_t<decltype(t)>;
            using U = std::remove_pointer_t<decltype(u)>;
            const RowMap m = plan_rows(dim, kVals<T, U>);
            const int64_t bytes = dim * (n_tokens * (int64_t)sizeof(U) + std::min(n_tokens, vocab) * (int64_t)sizeof(T));
            k_embed<T, U><<<row_grid(m, n_tokens), 256, 0, c->stream>>>(
                (const T*)table, table_stride, (int)vocab, (int)dim, tokens, (int)n_tokens, pad, scale, (U*)out, out_stride, m,
                streams(bytes), c->dev_words + kWordVectors);
            HGB_LAUNCHED(c, "k_embed");
            return HGB_OK;
        });
    });
}

int64_t hgb_embed_backward_workspace(int64_t n_tokens, int64_t vocab, int64_t dim)
{
    if (n_tokens < 0 || n_tokens > kVecMaxRows || vocab < 1 || vocab > kVecMaxVocab || dim < 1 || dim > kVecMaxDim) return -1;
    return n_tokens == 0 ? 0 : plan_embed(n_tokens, vocab, dim).bytes;
}

hgb_status hgb_embed_backward(hgb_ctx* c, const void* grad, int32_t grad_type, int64_t grad_stride, int64_t n_tokens,
                              int64_t dim, const int32_t* tokens, int32_t pad, float scale, int64_t vocab, void* out,
                              int32_t out_type, int64_t out_stride, void* workspace, int64_t workspace_bytes)
{
    return guarded(c, [&]() -> hgb_status {
        HGB_TRY(check_dim(c, "embed_backward", n_tokens, dim));
        if (vocab < 1 || vocab > kVecMaxVocab)
            return fail(c, HGB_E_INVALID, "embed_backward: vocab is outside [1, 2^31 - 2]");
        HGB_TRY(check_rows(c, "embed_backward", "grad", grad, grad_type, n_tokens, dim, grad_stride));
        HGB_TRY(check_rows(c, "embed_backward", "out", out, out_type, vocab, dim, out_stride));
        if (!is_pair(out_type, grad_type))
            return fail(c, HGB_E_UNSUPPORTED, "embed_backward: grad has out's type, or 16 bits beside a 32-bit out");
        if (n_tokens > 0 && !tokens) return fail(c, HGB_E_INVALID, "embed_backward: tokens is null");
        HGB_TRY(check_words(c, "embed_backward", {tokens}));
        const EmbedPlan p = plan_embed(n_tokens, vocab, dim);
        const Span to = span(out, out_type, vocab, dim, out_stride), from = span(grad, grad_type, n_tokens, dim, grad_stride);
        HGB_TRY(check_apart(c, "embed_backward", {to}, {from, span(tokens, n_tokens)}));
        if (n_tokens > 0) {
            HGB_TRY(check_workspace(c, "embed_backward", workspace, workspace_bytes, p.bytes));
            HGB_TRY(check_apart(c, "embed_backward", {to, Span{(const char*)workspace, p.bytes}}, {from, span(tokens, n_tokens)}));
        }
        HGB_HIP(c, hipSetDevice(c->device));
        ProfScope ps(c, HGB_KERNEL_EMBED);
        ZeroFill z;
        z.out = out;
        z.rows = vocab;
        z.cols = dim;
        z.stride = out_stride;
        z.elem = elem_size(out_type);
        z.stream = streams(dim * (n_tokens * elem_size(grad_type) + vocab * z.elem));
        if (n_tokens == 0) {
            k_zero_rows<<<(unsigned)std::min<int64_t>(vec_ceil(vocab * dim * z.elem, 4096 * 4), 8 * c->n_cu), 256, 0,
                          c->stream>>>(z);
            HGB_LAUNCHED(c, "k_zero_rows");
            return HGB_OK;
        }
        char* ws = (char*)workspace;
        SortIn in{tokens, nullptr, n_tokens, vocab, pad, kVecErrToken, c->dev_words + kWordVectors};
        const uint2* pairs = nullptr;
        HGB_TRY(launch_sort(c, in, SortOut{}, p.sort, z, (uint32_t*)ws, (uint2*)(ws + p.off_a), (uint2*)(ws + p.off_b), &pairs));
        return by_pair(out_type, grad_type, [&](auto* u, auto* t) -> hgb_status {
            using U = std::remove_pointer_t<decltype(u)>;
            using T = std::remove_pointer_t<decltype(t)>;
            float* part = (float*)(ws + p.off_part);
            uint32_t* ends = (uint32_t*)(ws + p.off_ends);
            const RowMap m = plan_rows(dim, kVals<T, U>);
            k_embed_sum<T, U><<<row_grid(m, p.chunks), 256, 0, c->stream>>>(
                pairs, n_tokens, (const T*)grad, grad_stride, dim, vocab, scale, (U*)out, out_stride, part, p.part_stride, ends,
                p.chunk, p.chunks, m, z.stream);
            HGB_LAUNCHED(c, "k_embed_sum");
            if (p.chunks > 1) {
                // two blocks a CU before a block takes more chunks
                const int64_t slices = vec_ceil(dim, 64);
                const int own = vec_pow2(std::min<int64_t>(kJoinChunks, std::max<int64_t>(4, p.chunks * slices / (2 * c->n_cu))));
                k_embed_join<U><<<dim3((unsigned)vec_ceil(p.chunks, own), (unsigned)slices), 256, 0, c->stream>>>(
                    ends, (int)dim, scale, (U*)out, out_stride, part, p.part_stride, (int)p.chunks, own,
                    log2_of(std::min(16, vec_pow2(vec_ceil(dim, 4)))));
                HGB_LAUNCHED(c, "k_embed_join");
            }
            return HGB_OK;
        });
    });
}

hgb_status hgb_layer_norm(hgb_ctx* c, const void* x, int32_t type, int64_t x_stride, int64_t n_rows, int64_t dim,
                          const void* weight, const void* bias, int32_t param_type, float eps, void* y, int64_t y_stride,
                          float* mean, float* rstd)
{
    return guarded(c, [&]() -> hgb_status {
        HGB_TRY(check_dim(c, "layer_norm", n_rows, dim));
        HGB_TRY(check_rows(c, "layer_norm", "x", x, type, n_rows, dim, x_stride));
        HGB_TRY(check_rows(c, "layer_norm", "y", y, type, n_rows, dim, y_stride));
        HGB_TRY(check_rows(c, "layer_norm", "weight", weight, param_type, 0, dim, dim));
        HGB_TRY(check_rows(c, "layer_norm", "bias", bias, param_type, 0, dim, dim));
        if (param_type != type && param_type != HGB_F32)
            return fail(c, HGB_E_UNSUPPORTED, "layer_norm: the parameters have x's type, or 32 bits");
        if (!(eps >= 0.0f) || std::isinf(eps)) return fail(c, HGB_E_INVALID, "layer_norm: eps must be finite and not negative");
        if (n_rows == 0) return HGB_OK;
        if (!mean || !rstd) return fail(c, HGB_E_INVALID, "layer_norm: mean or rstd is null");
        HGB_TRY(check_words(c, "layer_norm", {mean, rstd}));
        HGB_TRY(check_apart(c, "layer_norm", {span(y, type, n_rows, dim, y_stride), span(mean, n_rows), span(rstd, n_rows)},
                            {span(x, type, n_rows, dim, x_stride), span(weight, param_type, 1, dim, dim),
                             span(bias, param_type, 1, dim, dim)}));
        HGB_HIP(c, hipSetDevice(c->device));
        ProfScope ps(c, HGB_KERNEL_NORM);
        return by_type(type, [&](auto* t) -> hgb_status {
            using T = std::remove_pointer_t<decltype(t)>;
            const NormPlan p = plan_norm(dim);
            if (!p.values) {
                k_norm_wide<T><<<(unsigned)std::min<int64_t>(n_rows, 65536), 256, 0, c->stream>>>(
                    (const T*)x, x_stride, n_rows, dim, weight, bias, param_type, eps, (T*)y, y_stride, mean, rstd);
            } else {
                by_shape(p, dim, kVals<T>, [&](auto values, auto waves, auto tail) {
                    constexpr int NV = decltype(values)::value, WPR = decltype(waves)::value, THREADS = norm_threads(WPR);
                    const unsigned blocks =
                        (unsigned)std::min<int64_t>(vec_ceil(n_rows, p.per_block), (int64_t)c->n_cu * 2048 / THREADS);
                    k_norm<T, NV, WPR, decltype(tail)::value><<<blocks, THREADS, 0, c->stream>>>(
                        (const T*)x, x_stride, n_rows, (int)dim, weight, bias, param_type, eps, (T*)y, y_stride, mean, rstd,
                        p.log_group, streams(2 * n_rows * dim * elem_size(type)));
                });
            }
            HGB_LAUNCHED(c, "k_norm");
            return HGB_OK;
        });
    });
}

int64_t hgb_layer_norm_backward_workspace(int64_t n_rows, int64_t dim)
{
    if (n_rows < 0 || n_rows > kVecMaxRows || dim < 1 || dim > kVecMaxDim) return -1;
    return norm_workspace(n_rows, dim);
}

hgb_status hgb_layer_norm_backward(hgb_ctx* c, const void* grad, int64_t grad_stride, const void* x, int64_t x_stride,
                                   int32_t type, int64_t n_rows, int64_t dim, const float* mean, const float* rstd,
                                   const void* weight, int32_t param_type, void* dx, int64_t dx_stride, void* dweight,
                                   void* dbias, void* workspace, int64_t workspace_bytes)
{
    return guarded(c, [&]() -> hgb_status {
        const char* verb = "layer_norm_backward";
        HGB_TRY(check_dim(c, verb, n_rows, dim));
        HGB_TRY(check_rows(c, verb, "grad", grad, type, n_rows, dim, grad_stride));
        HGB_TRY(check_rows(c, verb, "x", x, type, n_rows, dim, x_stride));
        HGB_TRY(check_rows(c, verb, "dx", dx, type, n_rows, dim, dx_stride));
        HGB_TRY(check_rows(c, verb, "weight", weight, param_type, 0, dim, dim));
        HGB_TRY(check_rows(c, verb, "dweight", dweight, param_type, 0, dim, dim));
        HGB_TRY(check_rows(c, verb, "dbias", dbias, param_type, 0, dim, dim));
        if (param_type != type && param_type != HGB_F32)
            return fail(c, HGB_E_UNSUPPORTED, "%s: the parameters have x's type, or 32 bits", verb);
        if (n_rows > 0 && (!mean || !rstd)) return fail(c, HGB_E_INVALID, "%s: mean or rstd is null", verb);
        HGB_TRY(check_words(c, verb, {mean, rstd}));
        const bool params = dweight || dbias;
        const auto apart = [&](int64_t scratch) {
            return check_apart(c, verb,
                               {span(dx, type, n_rows, dim, dx_stride), span(dweight, param_type, 1, dim, dim),
                                span(dbias, param_type, 1, dim, dim), Span{(const char*)workspace, scratch}},
                               {span(x, type, n_rows, dim, x_stride), span(grad, type, n_rows, dim, grad_stride),
                                span(mean, n_rows), span(rstd, n_rows), span(weight, param_type, 1, dim, dim)});
        };
        HGB_TRY(apart(0));
        if (params) {
            HGB_TRY(check_workspace(c, verb, workspace, workspace_bytes, norm_workspace(n_rows, dim)));
            HGB_TRY(apart(norm_workspace(n_rows, dim)));
        }
        HGB_HIP(c, hipSetDevice(c->device));
        ProfScope ps(c, HGB_KERNEL_NORM);
        const NormPlan p = plan_norm(dim);
        const int parts = p.values ? norm_blocks(n_rows, p) : norm_parts(n_rows);
        HGB_TRY(by_type(type, [&](auto* t) -> hgb_status {
            using T = std::remove_pointer_t<decltype(t)>;
            const T* g = (const T*)grad;
            if (!p.values) {
                if (n_rows > 0) {
                    k_norm_wide_dx<T><<<(unsigned)std::min<int64_t>(n_rows, 65536), 256, 0, c->stream>>>(
                        g, grad_stride, (const T*)x, x_stride, n_rows, dim, mean, rstd, weight, param_type, (T*)dx, dx_stride);
                    HGB_LAUNCHED(c, "k_norm_wide_dx");
                }
                if (params) {
                    k_norm_wide_params<T><<<dim3((unsigned)vec_ceil(dim, 256), (unsigned)parts), 256, 0, c->stream>>>(
                        g, grad_stride, (const T*)x, x_stride, n_rows, dim, mean, rstd, (float*)workspace);
                    HGB_LAUNCHED(c, "k_norm_wide_params");
                }
            } else if (n_rows > 0 || params) {
                by_shape(p, dim, kVals<T>, [&](auto values, auto waves, auto tail) {
                    constexpr int NV = decltype(values)::value, WPR = decltype(waves)::value;
                    k_norm_grad<T, NV, WPR, decltype(tail)::value><<<(unsigned)parts, norm_grad_threads(NV, WPR), 0, c->stream>>>(
                        g, grad_stride, (const T*)x, x_stride, n_rows, (int)dim, mean, rstd, weight, param_type, (T*)dx,
                        dx_stride, params ? (float*)workspace : nullptr, dweight, dbias, p.log_group,
                        streams(3 * n_rows * dim * elem_size(type)));
                });
                HGB_LAUNCHED(c, "k_norm_grad");
            }
            return HGB_OK;
        }));
        if (params && (parts > 1 || !p.values)) {
            k_norm_join<<<dim3((unsigned)vec_ceil(dim, 16), 2), 256, 0, c->stream>>>((const float*)workspace, parts, dim, dweight,
                                                                                    dbias, param_type);
            HGB_LAUNCHED(c, "k_norm_join");
        }
        return HGB_OK;
    });
}

// The shape of a routing, as every routing verb takes it.
static hgb_status check_route(hgb_ctx* c, const char* verb, int64_t n_rows, int32_t top, const int32_t* position)
{
    if (n_rows < 0 || n_rows > kVecMaxRows)
        return fail(c, HGB_E_INVALID, "%s: %lld rows are outside [0, 2^31)", verb, (long long)n_rows);
    if (top < 1) return fail(c, HGB_E_INVALID, "%s: top must be positive", verb);
    if (top > kRouteMaxTop) return fail(c, HGB_E_UNSUPPORTED, "%s: top is above %d", verb, kRouteMaxTop);
    if (n_rows * top > kVecMaxRows) return fail(c, HGB_E_INVALID, "%s: the slots do not fit 31 bits", verb);
    if (n_rows > 0 && !position) return fail(c, HGB_E_INVALID, "%s: position is null", verb);
    return HGB_OK;
}

static hgb_status check_experts(hgb_ctx* c, const char* verb, int32_t n_experts)
{
    if (n_experts < 1) return fail(c, HGB_E_INVALID, "%s: n_experts must be positive", verb);
    if (n_experts > kRouteMaxExperts) return fail(c, HGB_E_UNSUPPORTED, "%s: n_experts is above %d", verb, kRouteMaxExperts);
    return HGB_OK;
}

int64_t hgb_route_workspace(int64_t n_rows, int32_t top, int32_t n_experts)
{
    if (n_rows < 0 || n_rows > kVecMaxRows || top < 1 || top > kRouteMaxTop || n_rows * top > kVecMaxRows || n_experts < 1 ||
        n_experts > kRouteMaxExperts)
        return -1;
    return route_workspace(n_rows * top, n_experts);
}

hgb_status hgb_route(hgb_ctx* c, const int32_t* experts, int64_t n_rows, int32_t top, int32_t n_experts, int32_t* order,
                     int32_t* position, int32_t* offsets, void* workspace, int64_t workspace_bytes)
{
    return guarded(c, [&]() -> hgb_status {
        HGB_TRY(check_route(c, "route", n_rows, top, position));
        HGB_TRY(check_experts(c, "route", n_experts));
        if (n_rows > 0 && (!experts || !order)) return fail(c, HGB_E_INVALID, "route: experts or order is null");
        if (!offsets) return fail(c, HGB_E_INVALID, "route: offsets is null");
        const int64_t n = n_rows * top;
        HGB_TRY(check_workspace(c, "route", workspace, workspace_bytes, route_workspace(n, n_experts)));
        HGB_TRY(check_words(c, "route", {experts, order, position, offsets}));
        HGB_TRY(check_apart(c, "route",
                            {span(order, n), span(position, n), span(offsets, (int64_t)n_experts + 1),
                             Span{(const char*)workspace, route_workspace(n, n_experts)}},
                            {span(experts, n)}));
        HGB_HIP(c, hipSetDevice(c->device));
        ProfScope ps(c, HGB_KERNEL_ROUTE);
        SortIn in{experts, nullptr, n, n_experts, -1, kVecErrExpert, c->dev_words + kWordVectors};
        SortOut out{nullptr, order, position, offsets};
        return launch_sort(c, in, out, plan_sort(n, n_experts, true), ZeroFill{}, (uint32_t*)workspace, nullptr, nullptr, nullptr);
    });
}

hgb_status hgb_route_gather(hgb_ctx* c, const void* x, int32_t type, int64_t x_stride, int64_t n_rows, int32_t top, int64_t dim,
                            const int32_t* position, const int32_t* offsets, int32_t n_experts, void* out, int64_t out_stride)
{
    return guarded(c, [&]() -> hgb_status {
        HGB_TRY(check_dim(c, "route_gather", n_rows, dim));
        HGB_TRY(check_route(c, "route_gather", n_rows, top, position));
        HGB_TRY(check_experts(c, "route_gather", n_experts));
        HGB_TRY(check_rows(c, "route_gather", "x", x, type, n_rows, dim, x_stride));
        HGB_TRY(check_rows(c, "route_gather", "out", out, type, n_rows, dim, out_stride));
        if (n_rows == 0) return HGB_OK;
        if (!offsets) return fail(c, HGB_E_INVALID, "route_gather: offsets is null");
        HGB_TRY(check_words(c, "route_gather", {position, offsets}));
        HGB_TRY(check_apart(c, "route_gather", {span(out, type, n_rows * top, dim, out_stride)},
                            {span(x, type, n_rows, dim, x_stride), span(position, n_rows * top),
                             span(offsets, (int64_t)n_experts + 1)}));
        HGB_HIP(c, hipSetDevice(c->device));
        ProfScope ps(c, HGB_KERNEL_ROUTE);
        return by_type(type, [&](auto* t) -> hgb_status {
            using T = std::remove_pointer_t<decltype(t)>;
            const RowMap m = plan_rows(dim, kVals<T>);
            k_route_gather<T><<<row_grid(m, n_rows), 256, 0, c->stream>>>(
                (const T*)x, x_stride, n_rows, top, (int)dim, position, offsets + n_experts, (T*)out, out_stride, m,
                streams(n_rows * (top + 1) * dim * elem_size(type)));
            HGB_LAUNCHED(c, "k_route_gather");
            return HGB_OK;
        });
    });
}

static hgb_status combine(hgb_ctx* c, const char* verb, const void* y, int32_t type, int64_t y_stride, int64_t n_rows,
                          int32_t top, int64_t dim, const int32_t* position, const float* weight, void* out,
                          int64_t out_stride)
{
    HGB_TRY(check_dim(c, verb, n_rows, dim));
    HGB_TRY(check_route(c, verb, n_rows, top, position));
    HGB_TRY(check_rows(c, verb, "the sorted rows", y, type, n_rows, dim, y_stride));
    HGB_TRY(check_rows(c, verb, "out", out, type, n_rows, dim, out_stride));
    if (n_rows == 0) return HGB_OK;
    HGB_TRY(check_words(c, verb, {position, weight}));
    HGB_TRY(check_apart(c, verb, {span(out, type, n_rows, dim, out_stride)},
                        {span(y, type, n_rows * top, dim, y_stride), span(position, n_rows * top), span(weight, n_rows * top)}));
    HGB_HIP(c, hipSetDevice(c->device));
    ProfScope ps(c, HGB_KERNEL_ROUTE);
    return by_type(type, [&](auto* t) -> hgb_status {
        using T = std::remove_pointer_t<decltype(t)>;
        const RowMap m = plan_rows(dim, kVals<T>);
        k_route_combine<T><<<row_grid(m, n_rows), 256, 0, c->stream>>>(
            (const T*)y, y_stride, n_rows, top, (int)dim, position, weight, (T*)out, out_stride, m,
            streams(n_rows * (top + 1) * dim * elem_size(type)));
        HGB_LAUNCHED(c, "k_route_combine");
        return HGB_OK;
    });
}

hgb_status hgb_route_combine(hgb_ctx* c, const void* y, int32_t type, int64_t y_stride, int64_t n_rows, int32_t top,
                             int64_t dim, const int32_t* position, const float* weight, void* out, int64_t out_stride)
{
    return guarded(c, [&]() -> hgb_status {
        return combine(c, "route_combine", y, type, y_stride, n_rows, top, dim, position, weight, out, out_stride);
    });
}

hgb_status hgb_route_gather_backward(hgb_ctx* c, const void* grad, int32_t type, int64_t grad_stride, int64_t n_rows,
                                     int32_t top, int64_t dim, const int32_t* position, void* dx, int64_t dx_stride)
{
    return guarded(c, [&]() -> hgb_status {
        return combine(c, "route_gather_backward", grad, type, grad_stride, n_rows, top, dim, position, nullptr, dx, dx_stride);
    });
}

hgb_status hgb_route_combine_backward(hgb_ctx* c, const void* grad, int32_t type, int64_t grad_stride, const void* y,
                                      int64_t y_stride, int64_t n_rows, int32_t top, int64_t dim, const int32_t* position,
                                      const int32_t* offsets, int32_t n_experts, const float* weight, void* dy,
                                      int64_t dy_stride, float* dweight)
{
    return guarded(c, [&]() -> hgb_status {
        const char* verb = "route_combine_backward";
        HGB_TRY(check_dim(c, verb, n_rows, dim));
        HGB_TRY(check_route(c, verb, n_rows, top, position));
        HGB_TRY(check_experts(c, verb, n_experts));
        HGB_TRY(check_rows(c, verb, "grad", grad, type, n_rows, dim, grad_stride));
        HGB_TRY(check_rows(c, verb, "the sorted rows", y, type, dweight ? n_rows : 0, dim, y_stride));
        HGB_TRY(check_rows(c, verb, "their gradient", dy, type, n_rows, dim, dy_stride));
        if (n_rows == 0) return HGB_OK;
        if (!offsets) return fail(c, HGB_E_INVALID, "%s: offsets is null", verb);
        HGB_TRY(check_words(c, verb, {position, offsets, weight, dweight}));
        HGB_TRY(check_apart(c, verb, {span(dy, type, n_rows * top, dim, dy_stride), span(dweight, n_rows * top)},
                            {span(grad, type, n_rows, dim, grad_stride),
                             span(dweight ? y : nullptr, type, n_rows * top, dim, y_stride), span(position, n_rows * top),
                             span(offsets, (int64_t)n_experts + 1), span(weight, n_rows * top)}));
        HGB_HIP(c, hipSetDevice(c->device));
        ProfScope ps(c, HGB_KERNEL_ROUTE);
        return by_type(type, [&](auto* t) -> hgb_status {
            using T = std::remove_pointer_t<decltype(t)>;
            const int64_t vecs = vec_ceil(dim, kVals<T>), slots = n_rows * top;
            const int lg = log2_of(vec_pow2(std::min<int64_t>(vecs, 64)));
            const bool stream = streams(n_rows * ((dweight ? 2 : 1) * top + 1) * dim * elem_size(type));
            auto* kernel = lg == 6 ? k_route_combine_grad<T, true> : k_route_combine_grad<T, false>;
            const GridSpan blocks = span_blocks(vec_ceil(slots, 256 >> lg));
            kernel<<<dim3(blocks.x, 1, blocks.z), 256, 0, c->stream>>>(
                (const T*)grad, grad_stride, (const T*)y, y_stride, n_rows, top, (int)dim, position, offsets + n_experts, weight,
                (T*)dy, dy_stride, dweight, lg, stream);
            HGB_LAUNCHED(c, "k_route_combine_grad");
            return HGB_OK;
        });
    });
}

}  // extern "C"
