// hgb: the losses of a softmax over the vocabulary (see include/hgb.h for the
// contract): cross entropy and distillation, with their gradients.
//
// Host side: argument checks and launches.  The kernels live in
// hgb_vector_head_kernels.h, the launch plans in hgb_vector_head_plan.h.
#include "hgb.h"
#include "hgb_ctx.h"
#include "hgb_vector_checks.h"
#include "hgb_vector_head_kernels.h"
#include "hgb_vector_head_plan.h"

#include <hip/hip_runtime.h>

#include <cmath>

using namespace hgb;

namespace {

// The arguments that the losses and their gradients share.
struct Head {
    const char* verb;
    const void* x;
    int32_t type;
    int64_t x_stride, n, dim;
    const void* table;
    int64_t table_stride, vocab;
    const int32_t* token;    // [n][top]
    int32_t top;
    int32_t pad;
    float scale;             // of the logits
    const void* teacher;     // null: the cross entropy
    int32_t teacher_type;
    float heat;

    int size() const { return elem_size(type); }
    bool copy_x() const { return !in_place(x, x_stride, dim, size()); }
    bool copy_table() const { return !in_place(table, table_stride, dim, size()); }
    TeacherArgs slots() const { return {token, teacher, teacher_type, top, (int32_t)vocab, heat}; }
};

hgb_status check_head(hgb_ctx* c, const Head& h)
{
    if (h.n < 0 || h.vocab < 1 || h.dim < 1) return fail(c, HGB_E_INVALID, "%s: n_rows is negative, or vocab or dim below one", h.verb);
    if (h.n > kHeadMaxRows || h.vocab > kHeadMaxVocab)
        return fail(c, HGB_E_UNSUPPORTED, "%s: n_rows or vocab is above %lld", h.verb, (long long)kHeadMaxRows);
    if (h.dim > kHeadMaxDim) return fail(c, HGB_E_UNSUPPORTED, "%s: dim is above %lld", h.verb, (long long)kHeadMaxDim);
    HGB_TRY(check_rows(c, h.verb, "x", h.x, h.type, h.n, h.dim, h.x_stride));
    HGB_TRY(check_rows(c, h.verb, "table", h.table, h.type, h.vocab, h.dim, h.table_stride));
    if (!std::isfinite(h.scale * kLog2e)) return fail(c, HGB_E_INVALID, "%s: the logits' scale times log2(e) is not finite", h.verb);
    if (h.top < 1) return fail(c, HGB_E_INVALID, "%s: top must be positive", h.verb);
    if (h.top > kDistillMaxTop) return fail(c, HGB_E_UNSUPPORTED, "%s: top is above %d", h.verb, kDistillMaxTop);
    if (h.n > 0 && !h.token) return fail(c, HGB_E_INVALID, "%s: the tokens are null", h.verb);
    return check_words(c, h.verb, {h.token});
}

// And what a teacher gives.
hgb_status check_teacher(hgb_ctx* c, const Head& h, float temperature)
{
    if (!(temperature > 0.0f) || std::isinf(temperature))
        return fail(c, HGB_E_INVALID, "%s: the temperature must be positive and finite", h.verb);
    if (std::isinf(temperature * temperature)) return fail(c, HGB_E_INVALID, "%s: the temperature's square is not finite", h.verb);
    if (h.n > 0 && !h.teacher) return fail(c, HGB_E_INVALID, "%s: teacher is null", h.verb);
    HGB_TRY(check_rows(c, h.verb, "teacher", h.teacher, h.teacher_type, h.n, 1, 1));
    if (h.teacher_type != h.type && h.teacher_type != HGB_F32)
        return fail(c, HGB_E_UNSUPPORTED, "%s: the teacher's logits have x's type, or 32 bits", h.verb);
    return HGB_OK;
}

template <typename T, int BM, int BN, int WM, int WN, bool A_BY_K, bool B_BY_K, int WHAT>
hgb_status launch_tile(hgb_ctx* c, ProductArgs g, const ProductPlan& p)
{
    auto* kernel = k_product<T, BM, BN, WM, WN, A_BY_K, B_BY_K, WHAT>;
    constexpr int lds = product_lds(BM, BN, WM * WN, WHAT != kStats), blocks = product_blocks(BM, BN, WM * WN, WHAT != kStats);
    if (lds > 65536) HGB_TRY(raise_lds(c, kernel));
    g.splits = p.splits;
    g.tiles_m = (int)p.tiles_m;
    g.tiles_n = (int)p.tiles_n;
    kernel<<<(unsigned)std::min<int64_t>(p.blocks(), (int64_t)blocks * c->n_cu), 64 * WM * WN, lds, c->stream>>>(g);
    HGB_LAUNCHED(c, "k_product");
    return HGB_OK;
}

template <typename T, bool A_BY_K, bool B_BY_K, int WHAT>
hgb_status launch_product(hgb_ctx* c, const ProductArgs& g, const ProductPlan& p)
{
    if (p.tile == kTileLow) return launch_tile<T, 32, 256, 1, 4, A_BY_K, B_BY_K, WHAT>(c, g, p);
    if (p.tile == kTileMiddle) return launch_tile<T, 128, 128, 2, 2, A_BY_K, B_BY_K, WHAT>(c, g, p);
    if constexpr (WHAT == kSum || WHAT == kOut)
        if (p.tile == kTileNarrow) return launch_tile<T, 256, 64, 4, 1, A_BY_K, B_BY_K, WHAT>(c, g, p);
    return launch_tile<T, 256, 256, 2, 2, A_BY_K, B_BY_K, WHAT>(c, g, p);
}

unsigned fill_blocks(const hgb_ctx* c, int64_t threads) { return (unsigned)std::min<int64_t>(vec_ceil(threads, 256), 16 * c->n_cu); }

template <typename T>
hgb_status copy_rows(hgb_ctx* c, const void* x, int64_t stride, int64_t n, int64_t dim, int64_t dp, float* rate, int rate_blocks,
                     void* out)
{
    k_head_copy<T><<<fill_blocks(c, n * dp * (int64_t)sizeof(T) / 16), 256, 0, c->stream>>>((const T*)x, stride, n, (int)dim, (int)dp,
                                                                                            rate, rate_blocks, (T*)out);
    HGB_LAUNCHED(c, "k_head_copy");
    return HGB_OK;
}

// lse, and the target's loss (not a teacher's).
template <typename T>
hgb_status run_forward(hgb_ctx* c, const Head& h, const HeadPlan& p, float* loss, float* lse, char* ws)
{
    const int64_t dp = h.copy_x() ? p.dp : h.dim, wp = h.copy_table() ? p.dp : h.dim;
    Factor fx{h.x, h.x_stride, h.n, dp, 0}, fw{h.table, h.table_stride, h.vocab, wp, 0};
    if (p.copy_x) {
        HGB_TRY(copy_rows<T>(c, h.x, h.x_stride, h.n, h.dim, p.dp, nullptr, 0, ws));
        fx.p = ws;
        fx.stride = p.dp;
    }
    if (p.copy_table) {
        HGB_TRY(copy_rows<T>(c, h.table, h.table_stride, h.vocab, h.dim, p.dp, nullptr, 0, ws + p.off_table));
        fw.p = ws + p.off_table;
        fw.stride = p.dp;
    }
    const char* rows = (const char*)fx.p;
    for (int64_t first = 0; first < h.n; first += p.piece) {
        ProductArgs g{};
        const int64_t n = std::min(p.piece, h.n - first);
        g.a = fx;
        g.a.p = rows + first * fx.stride * (int64_t)sizeof(T);
        g.a.rows = n;
        g.b = fw;
        g.m = (int)n;
        g.n = g.limit = (int)h.vocab;
        g.k_steps = (int)vec_ceil(h.dim * (int64_t)sizeof(T), kStepBytes);
        g.planes = 1;
        g.scale = h.scale * kLog2e;
        const int32_t* target = h.teacher ? nullptr : h.token + first;
        g.target = target;
        g.part = (float2*)(ws + p.off_part);
        g.hit = (float*)(ws + p.off_hit);
        ProductPlan z = p.z;
        z.tiles_m = vec_ceil(n, z.bm);
        HGB_TRY((launch_product<T, false, false, kStats>(c, g, z)));
        // few rows: more threads to each, while that gives no CU a block
        LossArgs l{g.part, p.parts, n, 0, g.hit, target, h.pad, (int32_t)h.vocab, loss ? loss + first : nullptr, lse + first,
                   c->dev_words + kWordVectors};
        while (l.log_rows < 5 && (n >> (l.log_rows + 1)) >= c->n_cu) ++l.log_rows;
        k_head_loss<<<(unsigned)vec_ceil(n, 1 << l.log_rows), 256, 0, c->stream>>>(l);
        HGB_LAUNCHED(c, "k_head_loss");
    }
    return HGB_OK;
}

hgb_status forward(hgb_ctx* c, const Head& h, float* loss, float* lse, float* picked, void* workspace, int64_t workspace_bytes)
{
    if (h.n == 0) return HGB_OK;
    if (!loss || !lse || (h.teacher && !picked)) return fail(c, HGB_E_INVALID, "%s: an output is null", h.verb);
    HGB_TRY(check_words(c, h.verb, {loss, lse, picked}));
    const HeadPlan p = plan_head(h.copy_x(), h.copy_table(), h.size(), h.n, h.vocab, h.dim);
    HGB_TRY(check_workspace(c, h.verb, workspace, workspace_bytes, p.bytes));
    HGB_TRY(check_apart(c, h.verb, {span(loss, h.n), span(lse, h.n), span(picked, h.n * h.top), Span{(const char*)workspace, p.bytes}},
                        {span(h.x, h.type, h.n, h.dim, h.x_stride), span(h.table, h.type, h.vocab, h.dim, h.table_stride),
                         span(h.token, h.n * h.top), span(h.teacher, h.teacher_type, h.n, h.top, h.top)}));
    HGB_HIP(c, hipSetDevice(c->device));
    ProfScope ps(c, HGB_KERNEL_HEAD);
    char* ws = (char*)workspace;
    return by_type(h.type, [&](auto* t) -> hgb_status {
        using T = std::remove_pointer_t<decltype(t)>;
        HGB_TRY(run_forward<T>(c, h, p, h.teacher ? nullptr : loss, lse, ws));
        if (h.teacher) {
            const TeacherArgs slots = h.slots();
            k_distill_pick<T><<<fill_blocks(c, h.n * h.top * 64), 256, 0, c->stream>>>(
                (const T*)h.x, h.x_stride, (const T*)h.table, h.table_stride, h.n, (int)h.dim, slots, picked);
            HGB_LAUNCHED(c, "k_distill_pick");
            k_distill_loss<<<fill_blocks(c, h.n * 64), 256, 0, c->stream>>>(h.n, slots, lse, picked, loss, c->dev_words + kWordVectors);
            HGB_LAUNCHED(c, "k_distill_loss");
        }
        return HGB_OK;
    });
}

struct HeadGrad {
    const float* grad;
    const float* lse;
    const float* picked;
    void* dx;
    int64_t dx_stride;
    void* dtable;
    int32_t dtable_type;
    int64_t dtable_stride;
};

int wide_planes(int32_t type) { return type == HGB_BF16 ? kPlanesBf16 : kPlanesF16; }

template <typename T>
hgb_status run_backward(hgb_ctx* c, const Head& h, const HeadGrad& o, const HeadGradPlan& p, char* ws)
{
    float* rate = (float*)(ws + p.off_rate);
    const float *unit = rate + h.n, *factor = rate + h.n + 1;
    // d (the logits' product): a cross entropy's scale; a distillation's T^2 / T
    RateArgs ra{o.grad, h.teacher ? h.heat : h.scale, h.n, (int32_t)h.vocab, h.token, h.top, h.pad, h.teacher, h.teacher_type,
                rate, c->dev_words + kWordVectors};
    const int rate_blocks = (int)std::min<int64_t>(kRateBlocks, vec_ceil(h.n, 256));
    k_head_rate<<<rate_blocks, 256, 0, c->stream>>>(ra);
    HGB_LAUNCHED(c, "k_head_rate");
    HGB_TRY(copy_rows<T>(c, h.x, h.x_stride, h.n, h.dim, p.dp, rate, rate_blocks, ws));
    const Factor fx{ws, p.dp, h.n, p.dp, 0};
    Factor fw{h.table, h.table_stride, h.vocab, h.dim, 0};
    if (p.copy_table) {
        HGB_TRY(copy_rows<T>(c, h.table, h.table_stride, h.vocab, h.dim, p.dp, nullptr, 0, ws + p.off_table));
        fw = Factor{ws + p.off_table, p.dp, h.vocab, p.dp, 0};
    }
    constexpr int STEP = kStepBytes / (int)sizeof(T);
    // Where dz has more planes, what its rounding left, they come first, the last
    // one in front: the sum over all then adds up the small values before the large.
    T *planes = (T*)(ws + p.off_z), *dz = planes + (p.planes - 1) * p.plane;
    float *sum = (float*)(ws + p.off_dx), *dw = (float*)(ws + p.off_dw);
    for (int64_t first = 0; first < h.vocab; first += p.piece) {
        const int64_t tokens = std::min(p.piece, h.vocab - first);
        Factor piece = fw;
        piece.p = (const char*)fw.p + first * fw.stride * (int64_t)sizeof(T);
        piece.rows = tokens;

        ProductArgs z{};
        z.a = fx;
        z.b = piece;
        z.m = (int)h.n;
        z.n = z.limit = (int)tokens;
        z.k_steps = (int)vec_ceil(h.dim, STEP);
        z.planes = 1;
        z.first = (int)first;
        z.scale = h.scale;
        z.target = h.teacher ? nullptr : h.token;
        z.lse = o.lse;
        z.rate = rate;
        z.unit = unit;
        z.dz = dz;
        z.dz_stride = p.stride;
        z.dz_plane = p.planes > 1 ? -p.plane : 0;
        ProductPlan zp = p.z;
        zp.tiles_n = vec_ceil(tokens, zp.bn);
        HGB_TRY((launch_product<T, false, false, kGrad>(c, z, zp)));
        if (h.teacher) {
            k_distill_dz<T><<<fill_blocks(c, h.n * 64), 256, 0, c->stream>>>(h.n, h.slots(), o.lse, o.picked, rate, unit, (int)first,
                                                                            (int)tokens, dz, p.stride, z.dz_plane);
            HGB_LAUNCHED(c, "k_distill_dz");
        }

        // dx: the sum over the piece's tokens; the pieces' sums in one buffer
        ProductArgs x{};
        x.a = Factor{dz, p.stride, h.n, p.piece, 0};
        x.b = piece;
        x.m = (int)h.n;
        x.n = (int)h.dim;
        x.k_steps = (int)vec_ceil(tokens, STEP);
        x.planes = 1;
        x.sum = sum;
        x.sum_stride = p.width;
        x.add = first > 0;
        ProductPlan xp = p.dx;
        xp.splits = std::min(xp.splits, x.k_steps);   // the last piece may be short: no share of it is empty
        HGB_TRY((launch_product<T, false, true, kSum>(c, x, xp)));

        ProductArgs w{};
        w.a = Factor{planes, p.stride, h.n, p.piece, p.plane};
        w.b = fx;
        w.m = (int)tokens;
        w.n = (int)h.dim;
        w.k_steps = (int)vec_ceil(h.n, STEP);
        w.planes = p.planes;
        char* out = (char*)o.dtable + first * o.dtable_stride * elem_size(o.dtable_type);
        ProductPlan wp = p.dw;
        wp.tiles_m = vec_ceil(tokens, wp.bm);
        if (wp.splits == 1) {
            w.out = out;
            w.out_stride = o.dtable_stride;
            w.out_type = o.dtable_type;
            w.factor = factor;
            HGB_TRY((launch_product<T, true, true, kOut>(c, w, wp)));
        } else {
            w.sum = dw;
            w.sum_stride = p.width;
            HGB_TRY((launch_product<T, true, true, kSum>(c, w, wp)));
            const unsigned blocks = fill_blocks(c, tokens * p.width / 4);
            if (o.dtable_type == HGB_F32)
                k_head_join<float><<<blocks, 256, 0, c->stream>>>(dw, p.width, wp.splits, tokens, (int)h.dim, nullptr, factor,
                                                                  (float*)out, o.dtable_stride);
            else
                k_head_join<T><<<blocks, 256, 0, c->stream>>>(dw, p.width, wp.splits, tokens, (int)h.dim, nullptr, factor, (T*)out,
                                                              o.dtable_stride);
            HGB_LAUNCHED(c, "k_head_join");
        }
    }
    k_head_join<T><<<fill_blocks(c, h.n * p.width / 4), 256, 0, c->stream>>>(sum, p.width, p.dx.splits, h.n, (int)h.dim, rate, factor,
                                                                            (T*)o.dx, o.dx_stride);
    HGB_LAUNCHED(c, "k_head_join");
    return HGB_OK;
}

hgb_status backward(hgb_ctx* c, const Head& h, const HeadGrad& o, void* workspace, int64_t workspace_bytes)
{
    HGB_TRY(check_rows(c, h.verb, "dx", o.dx, h.type, h.n, h.dim, o.dx_stride));
    HGB_TRY(check_rows(c, h.verb, "dtable", o.dtable, o.dtable_type, h.vocab, h.dim, o.dtable_stride));
    if (o.dtable_type != h.type && o.dtable_type != HGB_F32)
        return fail(c, HGB_E_UNSUPPORTED, "%s: dtable has x's type, or 32 bits", h.verb);
    if (h.n > 0 && (!o.grad || !o.lse || (h.teacher && !o.picked))) return fail(c, HGB_E_INVALID, "%s: an input is null", h.verb);
    HGB_TRY(check_words(c, h.verb, {o.grad, o.lse, o.picked}));
    const int64_t n = std::max<int64_t>(h.n, 1);
    const HeadGradPlan p = plan_head_grad(h.copy_table(), h.size(), elem_size(o.dtable_type), n, h.vocab, h.dim,
                                         wide_planes(h.type));
    if (h.n > 0) HGB_TRY(check_workspace(c, h.verb, workspace, workspace_bytes, p.bytes));
    HGB_TRY(check_apart(c, h.verb,
                        {span(o.dx, h.type, h.n, h.dim, o.dx_stride), span(o.dtable, o.dtable_type, h.vocab, h.dim, o.dtable_stride),
                         Span{(const char*)workspace, h.n > 0 ? p.bytes : 0}},
                        {span(h.x, h.type, h.n, h.dim, h.x_stride), span(h.table, h.type, h.vocab, h.dim, h.table_stride),
                         span(h.token, h.n * h.top), span(h.teacher, h.teacher_type, h.n, h.top, h.top), span(o.grad, h.n),
                         span(o.lse, h.n), span(o.picked, h.n * h.top)}));
    HGB_HIP(c, hipSetDevice(c->device));
    ProfScope ps(c, HGB_KERNEL_HEAD);
    if (h.n == 0) {   // no rows: the table's gradient is zero
        k_head_zero<<<fill_blocks(c, vec_ceil(h.vocab * h.dim, 16)), 256, 0, c->stream>>>((char*)o.dtable, o.dtable_stride * elem_size(o.dtable_type),
                                                                               h.vocab, h.dim * elem_size(o.dtable_type));
        HGB_LAUNCHED(c, "k_head_zero");
        return HGB_OK;
    }
    return by_type(h.type, [&](auto* t) -> hgb_status {
        using T = std::remove_pointer_t<decltype(t)>;
        return run_backward<T>(c, h, o, p, (char*)workspace);
    });
}

bool head_sizes(int32_t type, int64_t n, int64_t vocab, int64_t dim)
{
    return is_type(type) && n >= 0 && n <= kHeadMaxRows && vocab >= 1 && vocab <= kHeadMaxVocab && dim >= 1 && dim <= kHeadMaxDim;
}

}  // namespace

extern "C" {

int64_t hgb_head_workspace(const void* x, int64_t x_stride, const void* table, int64_t table_stride, int32_t type, int64_t n_rows,
                           int64_t vocab, int64_t dim)
{
    if (!head_sizes(type, n_rows, vocab, dim)) return -1;
    if (n_rows == 0) return 0;
    const int size = elem_size(type);
    return plan_head(!in_place(x, x_stride, dim, size), !in_place(table, table_stride, dim, size), size, n_rows, vocab, dim).bytes;
}

int64_t hgb_head_backward_workspace(const void*, int64_t, const void* table, int64_t table_stride, int32_t type, int32_t dtable_type,
                                    int64_t n_rows, int64_t vocab, int64_t dim)
{
    if (!head_sizes(type, n_rows, vocab, dim) || !is_type(dtable_type)) return -1;
    if (n_rows == 0) return 0;
    const int size = elem_size(type);
    return plan_head_grad(!in_place(table, table_stride, dim, size), size, elem_size(dtable_type), n_rows, vocab, dim, wide_planes(type))
        .bytes;
}

hgb_status hgb_cross_entropy(hgb_ctx* c, const void* x, int32_t type, int64_t x_stride, int64_t n_rows, int64_t dim, const void* table,
                             int64_t table_stride, int64_t vocab, const int32_t* targets, int32_t pad, float scale, float* loss,
                             float* lse, void* workspace, int64_t workspace_bytes)
{
    return guarded(c, [&]() -> hgb_status {
        const Head h{"cross_entropy", x, type, x_stride, n_rows, dim, table, table_stride, vocab, targets, 1, pad, scale,
                     nullptr, HGB_F32, 1.0f};
        HGB_TRY(check_head(c, h));
        return forward(c, h, loss, lse, nullptr, workspace, workspace_bytes);
    });
}

hgb_status hgb_cross_entropy_backward(hgb_ctx* c, const float* grad, const void* x, int32_t type, int64_t x_stride, int64_t n_rows,
                                      int64_t dim, const void* table, int64_t table_stride, int64_t vocab, const int32_t* targets,
                                      int32_t pad, float scale, const float* lse, void* dx, int64_t dx_stride, void* dtable,
                                      int32_t dtable_type, int64_t dtable_stride, void* workspace, int64_t workspace_bytes)
{
    return guarded(c, [&]() -> hgb_status {
        const Head h{"cross_entropy_backward", x, type, x_stride, n_rows, dim, table, table_stride, vocab, targets, 1, pad, scale,
                     nullptr, HGB_F32, 1.0f};
        HGB_TRY(check_head(c, h));
        return backward(c, h, HeadGrad{grad, lse, nullptr, dx, dx_stride, dtable, dtable_type, dtable_stride}, workspace,
                        workspace_bytes);
    });
}

hgb_status hgb_distill(hgb_ctx* c, const void* x, int32_t type, int64_t x_stride, int64_t n_rows, int64_t dim, const void* table,
                       int64_t table_stride, int64_t vocab, const int32_t* tokens, const void* teacher, int32_t teacher_type,
                       int32_t top, float temperature, float* loss, float* lse, float* picked, void* workspace,
                       int64_t workspace_bytes)
{
    return guarded(c, [&]() -> hgb_status {
        const Head h{"distill", x, type, x_stride, n_rows, dim, table, table_stride, vocab, tokens, top, -1,
                     1.0f / temperature, teacher, teacher_type, temperature};
        HGB_TRY(check_head(c, h));
        HGB_TRY(check_teacher(c, h, temperature));
        return forward(c, h, loss, lse, picked, workspace, workspace_bytes);
    });
}

hgb_status hgb_distill_backward(hgb_ctx* c, const float* grad, const void* x, int32_t type, int64_t x_stride, int64_t n_rows,
                                int64_t dim, const void* table, int64_t table_stride, int64_t vocab, const int32_t* tokens,
                                const void* teacher, int32_t teacher_type, int32_t top, float temperature, const float* lse,
                                const float* picked, void* dx, int64_t dx_stride, void* dtable, int32_t dtable_type,
                                int64_t dtable_stride, void* workspace, int64_t workspace_bytes)
{
    return guarded(c, [&]() -> hgb_status {
        const Head h{"distill_backward", x, type, x_stride, n_rows, dim, table, table_stride, vocab, tokens, top, -1,
                     1.0f / temperature, teacher, teacher_type, temperature};
        HGB_TRY(check_head(c, h));
        HGB_TRY(check_teacher(c, h, temperature));
        return backward(c, h, HeadGrad{grad, lse, picked, dx, dx_stride, dtable, dtable_type, dtable_stride}, workspace,
                        workspace_bytes);
    });
}

}  // extern "C"
