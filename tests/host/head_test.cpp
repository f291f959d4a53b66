// The gate and the head's losses on the host alone: their plans, what their C
// entry points refuse, and what they ask of the runtime, whose launch functions
// are this program's and run nothing.  No buffer is touched: addresses are made
// up.  Usage: head_test plan | planes | refusals | grids | no_rows | factors
#include "hgb_vector_head_plan.h"
#ifdef WITH_LIBRARY
#include "hgb_ctx.h"
#endif

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <map>

using namespace hgb;

static int failures = 0, checks = 0;

#define CHECK(cond)                                                              \
    do {                                                                         \
        ++checks;                                                                \
        if (!(cond) && ++failures <= 20) std::printf("line %d: %s\n", __LINE__, #cond); \
    } while (0)

static const int64_t kRows[] = {1, 31, 32, 33, 255, 256, 257, 5001, 16384, 40000, 1 << 20, 1 << 24};
static const int64_t kVocabs[] = {1, 2, 255, 256, 257, 1023, 7196, 32768, 262144, 1 << 24};
static const int64_t kDims[] = {1, 3, 8, 64, 65, 129, 512, 1024, 5000, 32768};

static void check_product(const ProductPlan& p, int64_t m, int64_t n, int64_t steps)
{
    CHECK(p.bm == kTiles[p.tile].bm && p.bn == kTiles[p.tile].bn);
    CHECK((p.tile == kTileLow) == (m <= kTileFew));
    CHECK(p.tiles_m * p.bm >= m && (p.tiles_m - 1) * p.bm < m && p.tiles_n * p.bn >= n && (p.tiles_n - 1) * p.bn < n);
    CHECK(p.splits >= 1 && (p.splits == 1 || p.splits <= steps));   // no share is empty
    CHECK(p.blocks() * 256 < (int64_t)1 << 32);
}

static void plans()
{
    for (int size : {2, 4})
        for (int64_t n : kRows)
            for (int64_t vocab : kVocabs)
                for (int64_t dim : kDims) {
                    for (int copy = 0; copy < 4; ++copy) {
                        const HeadPlan p = plan_head(copy & 1, copy & 2, size, n, vocab, dim);
                        CHECK(p.dp >= dim && p.dp * size % 16 == 0 && p.dp - dim < 16 / size);
                        CHECK(p.piece >= 1 && p.piece <= n && (p.piece == n || p.piece % kTileRows == 0));
                        check_product(p.z, p.piece, vocab, 1);
                        CHECK(p.parts == p.z.tiles_n * kTiles[p.z.tile].wn && p.z.tile != kTileNarrow);
                        CHECK(p.off_table >= (p.copy_x ? n * p.dp * size : 0) && p.off_table % 256 == 0);
                        CHECK(p.off_part >= p.off_table + (p.copy_table ? vocab * p.dp * size : 0) && p.off_part % 256 == 0);
                        CHECK(p.off_hit >= p.off_part + p.parts * p.piece * 8 && p.bytes >= p.off_hit + n * 4);
                    }
                    for (int out : {2, 4}) {
                        if (out < size) continue;
                        const HeadGradPlan p = plan_head_grad(true, size, out, n, vocab, dim);
                        CHECK(p.planes == (out > size ? 2 : 1) && p.piece % kTileCols == 0 && p.stride > p.piece && p.stride * size % 16 == 0);
                        CHECK(p.plane == n * p.stride);
                        CHECK(p.pieces * p.piece >= vocab && (p.pieces - 1) * p.piece < vocab);
                        CHECK(p.piece == kTileCols || n * p.piece * p.planes * size <= kPieceBytes);
                        const int step = kStepBytes / size;
                        check_product(p.z, n, p.piece, 1);
                        check_product(p.dx, n, dim, std::min(p.piece, vocab) / step);
                        check_product(p.dw, std::min(p.piece, vocab), dim, vec_ceil(n, step) * p.planes);
                        CHECK(p.width >= dim && p.width % 4 == 0);
                        CHECK(p.off_table >= n * p.dp * size && p.off_rate >= p.off_table + vocab * p.dp * size);
                        CHECK(p.off_z >= p.off_rate + (n + kRateWords) * 4 && p.off_dx >= p.off_z + p.plane * p.planes * size);
                        CHECK(p.off_dw >= p.off_dx + p.dx.splits * n * p.width * 4);
                        CHECK(p.bytes >= p.off_dw + (p.dw.splits > 1 ? p.dw.splits * p.piece * p.width * 4 : 0));
                        CHECK(p.off_table % 16 == 0 && p.off_z % 16 == 0 && p.off_dx % 16 == 0 && p.off_dw % 16 == 0);
                    }
                }
    for (int e = 1; e <= kRouteMaxExperts; ++e) {
        const GatePlan p = plan_gate(e);
        CHECK((p.values << p.log_group) >= e && p.log_group <= 6 && p.per_block << p.log_group == 256);
        CHECK(p.log_group == 0 || (p.values << (p.log_group - 1)) < e);
        for (int groups : {1, e})
            for (int top : {1, std::min(e, 64)}) CHECK(gate_lds(p, e, groups, top, true) <= 163840 && gate_lds(p, e, groups, top, false) <= 65536);
    }
    alignas(16) char row[64];
    CHECK(in_place(row, 16, 8, 2) && !in_place(row + 2, 16, 8, 2) && !in_place(row, 15, 8, 2) && !in_place(row, 16, 7, 2));
    CHECK(in_place(row, 4, 4, 4) && !in_place(row, kHeadMaxStride + 8, 8, 2));
}

// Three planes of bf16's logits' gradient beside a 32-bit dtable.
static void planes()
{
    for (int64_t n : kRows)
        for (int64_t vocab : kVocabs)
            for (int64_t dim : kDims) {
                const HeadGradPlan p = plan_head_grad(true, 2, 4, n, vocab, dim, kPlanesBf16);
                CHECK(p.planes == 3 && plan_head_grad(true, 2, 2, n, vocab, dim, kPlanesBf16).planes == 1);
                CHECK(p.piece == kTileCols || n * p.piece * 2 * 2 <= kPieceBytes);   // a third plane takes half as much again
                CHECK(p.piece % kTileCols == 0 && p.pieces * p.piece >= vocab && (p.pieces - 1) * p.piece < vocab);
                CHECK(p.plane == n * p.stride && p.off_dx >= p.off_z + 3 * p.plane * 2 && p.off_dx % 16 == 0);
                check_product(p.dw, std::min(p.piece, vocab), dim, vec_ceil(n, kStepBytes / 2) * 3);
            }
}

#ifdef WITH_LIBRARY
static int launches = 0;

extern "C" {
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipGetLastError(void) { return hipSuccess; }
static std::map<const void*, int> limits;
hipError_t hipFuncSetAttribute(const void* fn, hipFuncAttribute which, int value)
{
    if (which != hipFuncAttributeMaxDynamicSharedMemorySize || value < 0 || value > 163840) return hipErrorInvalidValue;
    limits[fn] = value;
    return hipSuccess;
}
struct Shape {
    dim3 grid, block;
    size_t lds;
    hipStream_t stream;
} shape;
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t stream)
{
    shape = {grid, block, lds, stream};
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* stream)
{
    *grid = shape.grid;
    *block = shape.block;
    *lds = shape.lds;
    *stream = shape.stream;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void* fn, dim3 grid, dim3 block, void**, size_t lds, hipStream_t)
{
    ++launches;
    const auto limit = limits.find(fn);
    CHECK(lds <= (size_t)(limit == limits.end() ? 65536 : limit->second));
    CHECK(grid.x > 0 && grid.y > 0 && grid.z > 0 && block.x * block.y * block.z <= 1024);
    CHECK((uint64_t)grid.x * block.x < (uint64_t)1 << 32 && grid.y < 65536 && grid.z < 65536);
    return hipSuccess;
}
}  // extern "C"

static char* at(int k) { return (char*)((uint64_t)(k + 1) << 57); }
static const int64_t kRoom = (int64_t)1 << 56;

static void grids()
{
    hgb_ctx c;   // no device behind it
    c.dev_words = (uint32_t*)4096;
    void *x = at(1), *w = at(3), *dx = at(5), *dw = at(6), *ws = at(14), *teacher = at(7);
    float *loss = (float*)at(8), *lse = (float*)at(9), *picked = (float*)at(10), *grad = (float*)at(11);
    int32_t* tok = (int32_t*)at(12);
    auto ok = [&](hgb_status s) {
        ++checks;
        if (s != HGB_OK && ++failures <= 20) std::printf("status %d, %s\n", s, c.err.c_str());
    };
    for (int32_t type : {HGB_F32, HGB_BF16, HGB_F16})
        for (int64_t n : kRows)
            for (int64_t vocab : kVocabs)
                for (int64_t dim : kDims) {
                    if (n * vocab > (int64_t)1 << 40 && dim > 8) continue;   // many pieces, all alike
                    ok(hgb_cross_entropy(&c, x, type, dim, n, dim, w, dim, vocab, tok, -1, 1, loss, lse, ws, kRoom));
                    ok(hgb_distill(&c, x, type, dim, n, dim, w, dim, vocab, tok, teacher, type, 64, 2, loss, lse, picked, ws, kRoom));
                    ok(hgb_cross_entropy_backward(&c, grad, x, type, dim, n, dim, w, dim, vocab, tok, -1, 1, lse, dx, dim, dw, HGB_F32,
                                                  dim, ws, kRoom));
                    ok(hgb_distill_backward(&c, grad, x, type, dim, n, dim, w, dim, vocab, tok, teacher, type, 64, 2, lse, picked, dx,
                                            dim, dw, type, dim, ws, kRoom));
                }
    for (int64_t n : {(int64_t)0, (int64_t)1, (int64_t)257, (int64_t)1 << 24, (int64_t)33554431})
        for (int32_t e : {1, 8, 9, 64, 512, 513, 1023}) {
            ok(hgb_gate(&c, x, HGB_BF16, e, n, e, HGB_SOFTMAX, nullptr, e, e, 1, 1, 1, 1, tok, loss));
            ok(hgb_gate(&c, x, HGB_F32, e, n, e, HGB_SIGMOID, lse, 1, 1, 2, std::min(e, 64), 0, 1, tok, loss));
            ok(hgb_gate_backward(&c, grad, x, HGB_F16, e, n, e, HGB_SOFTMAX, tok, std::min(e, 64), 0, 1, dx, e));
        }
    ok(hgb_gate(&c, x, HGB_BF16, 1023, 2147483647, 1023, HGB_SOFTMAX, nullptr, 1, 1, 2, 1, 1, 1, tok, loss));
    ok(hgb_gate_backward(&c, grad, x, HGB_F32, 1023, 2147483647, 1023, HGB_SOFTMAX, tok, 1, 1, 1, dx, 1023));
    CHECK(launches > 0);
}

// Factors that are finite, and not so as the kernels take them: the logits'
// times log2(e), the loss's T^2.
static void factors()
{
    hgb_ctx c;   // no device behind it
    c.dev_words = (uint32_t*)4096;
    void *x = at(1), *w = at(3), *dx = at(5), *dw = at(6), *ws = at(14), *teacher = at(7);
    float *loss = (float*)at(8), *lse = (float*)at(9), *picked = (float*)at(10), *grad = (float*)at(11);
    int32_t* tok = (int32_t*)at(12);
    auto takes = [&](float scale) {
        return hgb_cross_entropy(&c, x, HGB_F32, 4, 2, 4, w, 4, 9, tok, -1, scale, loss, lse, ws, kRoom) == HGB_OK;
    };
    auto heats = [&](float t) {
        const hgb_status s = hgb_distill(&c, x, HGB_F32, 4, 2, 4, w, 4, 9, tok, teacher, HGB_F32, 3, t, loss, lse, picked, ws, kRoom);
        const hgb_status b = hgb_distill_backward(&c, grad, x, HGB_F32, 4, 2, 4, w, 4, 9, tok, teacher, HGB_F32, 3, t, lse, picked, dx, 4,
                                                  dw, HGB_F32, 4, ws, kRoom);
        CHECK(s == b && (s == HGB_OK || s == HGB_E_INVALID));
        return s == HGB_OK;
    };
    CHECK(takes(2.3e38f) && takes(-2.3e38f) && takes(0.0f) && takes(-0.5f) && takes(1e-45f));
    CHECK(!takes(2.4e38f) && !takes(-3.4e38f) && !takes(NAN));
    CHECK(heats(1.8e19f) && heats(1.0f) && heats(1e-18f) && heats(5e-39f));
    CHECK(!heats(1.9e19f) && !heats(3.4e38f) && !heats(4e-39f) && !heats(1e-45f));
}

// Gradients of no rows: one launch each, which clears the table's gradient.
static void no_rows()
{
    hgb_ctx c;   // no device behind it
    c.dev_words = (uint32_t*)4096;
    void *w = at(3), *dw = at(6);
    for (int32_t type : {HGB_F32, HGB_BF16, HGB_F16})
        for (int64_t vocab : {1, 2, 3, 5, 8, 15, 16, 17, 300, 1 << 24})
            for (int64_t dim : {1, 2, 3, 4, 5, 7, 8, 16, 17, 1024})
                for (int32_t out : {type, (int32_t)HGB_F32}) {
                    const int before = launches;
                    CHECK(hgb_cross_entropy_backward(&c, nullptr, nullptr, type, dim, 0, dim, w, dim, vocab, nullptr, -1, 1, nullptr,
                                                     nullptr, dim, dw, out, dim, nullptr, 0) == HGB_OK);
                    CHECK(hgb_distill_backward(&c, nullptr, nullptr, type, dim, 0, dim, w, dim, vocab, nullptr, nullptr, type, 4, 2,
                                               nullptr, nullptr, nullptr, dim, dw, out, dim, nullptr, 0) == HGB_OK);
                    CHECK(launches == before + 2);
                }
}

static void refusals()
{
    hgb_ctx c;   // no device behind it
    alignas(16) static float f[1024];
    static int32_t i[64];
    alignas(16) static char ws[1 << 20];
    auto is = [&](hgb_status got, hgb_status want, const char* word) {
        ++checks;
        if (got != want || !std::strstr(c.err.c_str(), word)) {
            ++failures;
            std::printf("got %d \"%s\", wanted %d \"%s\"\n", got, c.err.c_str(), want, word);
        }
    };
    const int32_t F = HGB_F32, B = HGB_BF16;
    const hgb_status bad = HGB_E_INVALID, no = HGB_E_UNSUPPORTED;
    float *o = f + 512, *o2 = f + 576, *o3 = f + 640;
    int32_t* e = (int32_t*)(f + 700);
    // gate(ctx, logits, type, stride, n, experts, score, bias, groups, keep, best, top, renormalise, scale, chosen, share)
    is(hgb_gate(&c, nullptr, F, 8, 2, 8, 0, nullptr, 1, 1, 2, 2, 1, 1, e, o), bad, "logits is null");
    is(hgb_gate(&c, f, 9, 8, 2, 8, 0, nullptr, 1, 1, 2, 2, 1, 1, e, o), bad, "unknown type");
    is(hgb_gate(&c, f, F, 7, 2, 8, 0, nullptr, 1, 1, 2, 2, 1, 1, e, o), bad, "overlap");
    is(hgb_gate(&c, (char*)f + 2, F, 8, 2, 8, 0, nullptr, 1, 1, 2, 2, 1, 1, e, o), bad, "aligned");
    is(hgb_gate(&c, f, F, 8, -1, 8, 0, nullptr, 1, 1, 2, 2, 1, 1, e, o), bad, "rows");
    is(hgb_gate(&c, f, F, 8, (int64_t)1 << 31, 8, 0, nullptr, 1, 1, 2, 2, 1, 1, e, o), bad, "rows");
    is(hgb_gate(&c, f, F, 8, (int64_t)1 << 30, 8, 0, nullptr, 1, 1, 2, 2, 1, 1, e, o), bad, "slots");
    is(hgb_gate(&c, f, F, 8, 2, 0, 0, nullptr, 1, 1, 2, 2, 1, 1, e, o), bad, "n_experts");
    is(hgb_gate(&c, f, F, 1024, 2, 1024, 0, nullptr, 1, 1, 2, 2, 1, 1, e, o), no, "n_experts");
    is(hgb_gate(&c, f, F, 8, 2, 8, 2, nullptr, 1, 1, 2, 2, 1, 1, e, o), bad, "score");
    is(hgb_gate(&c, f, F, 8, 2, 8, 0, nullptr, 3, 1, 2, 2, 1, 1, e, o), bad, "groups");
    is(hgb_gate(&c, f, F, 8, 2, 8, 0, nullptr, 0, 1, 2, 2, 1, 1, e, o), bad, "groups");
    is(hgb_gate(&c, f, F, 8, 2, 8, 0, nullptr, 2, 3, 2, 2, 1, 1, e, o), bad, "keep");
    is(hgb_gate(&c, f, F, 8, 2, 8, 0, nullptr, 2, 0, 2, 2, 1, 1, e, o), bad, "keep");
    is(hgb_gate(&c, f, F, 8, 2, 8, 0, nullptr, 2, 1, 3, 2, 1, 1, e, o), bad, "best");
    is(hgb_gate(&c, f, F, 8, 2, 8, 0, nullptr, 8, 4, 2, 2, 1, 1, e, o), bad, "best");
    is(hgb_gate(&c, f, F, 8, 2, 8, 0, nullptr, 2, 1, 2, 5, 1, 1, e, o), bad, "eligible");
    is(hgb_gate(&c, f, F, 8, 2, 8, 0, nullptr, 1, 1, 2, 0, 1, 1, e, o), bad, "top");
    is(hgb_gate(&c, f, F, 100, 2, 100, 0, nullptr, 1, 1, 2, 65, 1, 1, e, o), no, "top");
    is(hgb_gate(&c, f, F, 8, 2, 8, 0, nullptr, 1, 1, 2, 2, 1, NAN, e, o), bad, "scale");
    is(hgb_gate(&c, f, F, 8, 2, 8, 0, nullptr, 1, 1, 2, 2, 1, 1, nullptr, o), bad, "null");
    is(hgb_gate(&c, f, F, 8, 2, 8, 0, (float*)((char*)f + 402), 1, 1, 2, 2, 1, 1, e, o), bad, "4 bytes");
    is(hgb_gate(&c, f, F, 8, 2, 8, 0, nullptr, 1, 1, 2, 2, 1, 1, e, f + 15), bad, "overlaps");
    is(hgb_gate(&c, f, F, 8, 2, 8, 0, nullptr, 1, 1, 2, 2, 1, 1, e, (float*)e + 3), bad, "overlaps");
    is(hgb_gate(&c, f, F, 8, 2, 8, 0, o + 3, 1, 1, 2, 2, 1, 1, e, o), bad, "overlaps");
    // gate_backward(ctx, grad, logits, type, stride, n, experts, score, chosen, top, renormalise, scale, dlogits, stride)
    is(hgb_gate_backward(&c, nullptr, f, F, 8, 2, 8, 0, i, 2, 1, 1, o, 8), bad, "null");
    is(hgb_gate_backward(&c, o2, f, F, 8, 2, 8, 0, nullptr, 2, 1, 1, o, 8), bad, "null");
    is(hgb_gate_backward(&c, o2, f, F, 8, 2, 8, 0, i, 2, 1, 1, nullptr, 8), bad, "dlogits is null");
    is(hgb_gate_backward(&c, o2, f, F, 8, 2, 8, 0, i, 2, 1, 1, o, 7), bad, "overlap");
    is(hgb_gate_backward(&c, o2, f, F, 8, 2, 8, 0, i, 2, 1, 1, f + 8, 8), bad, "overlaps");
    is(hgb_gate_backward(&c, o2, f, F, 8, 2, 8, 0, i, 2, 1, INFINITY, o, 8), bad, "scale");
    // cross_entropy(ctx, x, type, stride, n, dim, table, stride, vocab, targets, pad, scale, loss, lse, ws, bytes)
    const int64_t big = (int64_t)1 << 20;
    float* w = f + 128;
    is(hgb_cross_entropy(&c, nullptr, F, 4, 2, 4, w, 4, 9, i, -1, 1, o, o2, ws, big), bad, "x is null");
    is(hgb_cross_entropy(&c, f, F, 4, 2, 4, nullptr, 4, 9, i, -1, 1, o, o2, ws, big), bad, "table is null");
    is(hgb_cross_entropy(&c, f, 5, 4, 2, 4, w, 4, 9, i, -1, 1, o, o2, ws, big), bad, "unknown type");
    is(hgb_cross_entropy(&c, f, F, 3, 2, 4, w, 4, 9, i, -1, 1, o, o2, ws, big), bad, "overlap");
    is(hgb_cross_entropy(&c, f, F, 4, 2, 4, w, 3, 9, i, -1, 1, o, o2, ws, big), bad, "overlap");
    is(hgb_cross_entropy(&c, f, F, 4, -1, 4, w, 4, 9, i, -1, 1, o, o2, ws, big), bad, "n_rows");
    is(hgb_cross_entropy(&c, f, F, 4, 2, 4, w, 4, 0, i, -1, 1, o, o2, ws, big), bad, "vocab");
    is(hgb_cross_entropy(&c, f, F, 4, 2, 0, w, 4, 9, i, -1, 1, o, o2, ws, big), bad, "dim");
    is(hgb_cross_entropy(&c, f, F, 4, kHeadMaxRows + 1, 4, w, 4, 9, i, -1, 1, o, o2, ws, big), no, "n_rows");
    is(hgb_cross_entropy(&c, f, F, 4, 2, 4, w, 4, kHeadMaxVocab + 1, i, -1, 1, o, o2, ws, big), no, "vocab");
    is(hgb_cross_entropy(&c, f, F, 32769, 2, 32769, w, 32769, 9, i, -1, 1, o, o2, ws, big), no, "dim");
    is(hgb_cross_entropy(&c, f, F, 4, 2, 4, w, 4, 9, nullptr, -1, 1, o, o2, ws, big), bad, "tokens");
    is(hgb_cross_entropy(&c, f, F, 4, 2, 4, w, 4, 9, i, -1, INFINITY, o, o2, ws, big), bad, "scale");
    is(hgb_cross_entropy(&c, f, F, 4, 2, 4, w, 4, 9, i, -1, 1, nullptr, o2, ws, big), bad, "output");
    is(hgb_cross_entropy(&c, f, F, 4, 2, 4, w, 4, 9, i, -1, 1, o, o2, ws, 64), bad, "workspace");
    is(hgb_cross_entropy(&c, f, F, 4, 2, 4, w, 4, 9, i, -1, 1, o, o2, nullptr, big), bad, "workspace");
    is(hgb_cross_entropy(&c, f, F, 4, 2, 4, w, 4, 9, i, -1, 1, o, o2, ws + 8, big - 8), bad, "16 bytes");
    is(hgb_cross_entropy(&c, f, F, 4, 2, 4, w, 4, 9, i, -1, 1, o, o + 1, ws, big), bad, "overlaps");
    is(hgb_cross_entropy(&c, f, F, 4, 2, 4, w, 4, 9, i, -1, 1, w + 35, o2, ws, big), bad, "overlaps");
    is(hgb_cross_entropy(&c, f, F, 4, 2, 4, w, 4, 9, i, -1, 1, (float*)ws, o2, ws, big), bad, "overlaps");
    // cross_entropy_backward(ctx, grad, x, type, stride, n, dim, table, stride, vocab, targets, pad, scale, lse, dx, stride, dtable, type, stride, ws, bytes)
    is(hgb_cross_entropy_backward(&c, nullptr, f, F, 4, 2, 4, w, 4, 9, i, -1, 1, o, o2, 4, o3, F, 4, ws, big), bad, "input");
    is(hgb_cross_entropy_backward(&c, f + 64, f, F, 4, 2, 4, w, 4, 9, i, -1, 1, nullptr, o2, 4, o3, F, 4, ws, big), bad, "input");
    is(hgb_cross_entropy_backward(&c, f + 64, f, F, 4, 2, 4, w, 4, 9, i, -1, 1, o, nullptr, 4, o3, F, 4, ws, big), bad, "dx is null");
    is(hgb_cross_entropy_backward(&c, f + 64, f, F, 4, 2, 4, w, 4, 9, i, -1, 1, o, o2, 4, nullptr, F, 4, ws, big), bad, "dtable is null");
    is(hgb_cross_entropy_backward(&c, f + 64, f, F, 4, 2, 4, w, 4, 9, i, -1, 1, o, o2, 3, o3, F, 4, ws, big), bad, "overlap");
    is(hgb_cross_entropy_backward(&c, f + 64, f, F, 4, 2, 4, w, 4, 9, i, -1, 1, o, o2, 4, o3, B, 4, ws, big), no, "dtable");
    is(hgb_cross_entropy_backward(&c, f + 64, f, F, 4, 2, 4, w, 4, 9, i, -1, 1, o, o2, 4, o3, F, 4, ws, 64), bad, "workspace");
    is(hgb_cross_entropy_backward(&c, f + 64, f, F, 4, 2, 4, w, 4, 9, i, -1, 1, o, f + 4, 4, o3, F, 4, ws, big), bad, "overlaps");
    is(hgb_cross_entropy_backward(&c, f + 64, f, F, 4, 2, 4, w, 4, 9, i, -1, 1, o, o2, 4, o2 + 7, F, 4, ws, big), bad, "overlaps");
    // distill(ctx, x, type, stride, n, dim, table, stride, vocab, tokens, teacher, type, top, T, loss, lse, picked, ws, bytes)
    float* t = f + 320;
    is(hgb_distill(&c, f, F, 4, 2, 4, w, 4, 9, i, nullptr, F, 3, 1, o, o2, o3, ws, big), bad, "teacher is null");
    is(hgb_distill(&c, f, F, 4, 2, 4, w, 4, 9, i, t, B, 3, 1, o, o2, o3, ws, big), no, "teacher");
    is(hgb_distill(&c, f, F, 4, 2, 4, w, 4, 9, i, t, F, 0, 1, o, o2, o3, ws, big), bad, "top");
    is(hgb_distill(&c, f, F, 4, 2, 4, w, 4, 9, i, t, F, 257, 1, o, o2, o3, ws, big), no, "top");
    is(hgb_distill(&c, f, F, 4, 2, 4, w, 4, 9, i, t, F, 3, 0, o, o2, o3, ws, big), bad, "scale");
    is(hgb_distill(&c, f, F, 4, 2, 4, w, 4, 9, i, t, F, 3, -1, o, o2, o3, ws, big), bad, "temperature");
    is(hgb_distill(&c, f, F, 4, 2, 4, w, 4, 9, i, t, F, 3, INFINITY, o, o2, o3, ws, big), bad, "temperature");
    is(hgb_distill(&c, f, F, 4, 2, 4, w, 4, 9, i, t, F, 3, 1, o, o2, nullptr, ws, big), bad, "output");
    is(hgb_distill(&c, f, F, 4, 2, 4, w, 4, 9, i, t, F, 3, 1, o, o2, t + 5, ws, big), bad, "overlaps");
    is(hgb_distill_backward(&c, f + 64, f, F, 4, 2, 4, w, 4, 9, i, t, F, 3, 1, o, nullptr, o2, 4, o3, F, 4, ws, big), bad, "input");
    is(hgb_distill_backward(&c, f + 64, f, F, 4, 2, 4, w, 4, 9, i, t, F, 3, 1, o, t + 8, t + 13, 4, o3, F, 4, ws, big), bad, "overlaps");
    CHECK(hgb_head_workspace(f, 4, w, 4, F, -1, 9, 4) == -1 && hgb_head_workspace(f, 4, w, 4, F, 2, 0, 4) == -1);
    CHECK(hgb_head_workspace(f, 4, w, 4, 3, 2, 9, 4) == -1 && hgb_head_workspace(f, 4, w, 4, F, 0, 9, 4) == 0);
    CHECK(hgb_head_workspace(f, 4, w, 4, F, kHeadMaxRows + 1, 9, 4) == -1 && hgb_head_workspace(f, 4, w, 4, F, 2, 9, 32769) == -1);
    CHECK(hgb_head_workspace(f + 1, 4, w, 4, F, 2, 9, 4) > hgb_head_workspace(f, 4, w, 4, F, 2, 9, 4));
    CHECK(hgb_head_backward_workspace(f, 4, w, 4, F, 7, 2, 9, 4) == -1 && hgb_head_backward_workspace(f, 4, w, 4, B, F, 0, 9, 4) == 0);
    CHECK(hgb_gate(nullptr, f, F, 8, 2, 8, 0, nullptr, 1, 1, 2, 2, 1, 1, e, o) == bad);
    CHECK(hgb_cross_entropy(nullptr, f, F, 4, 2, 4, w, 4, 9, i, -1, 1, o, o2, ws, big) == bad);
    CHECK(launches == 0);
}
#endif

int main(int argc, char** argv)
{
    if (argc > 1 && !std::strcmp(argv[1], "plan")) plans();
    if (argc > 1 && !std::strcmp(argv[1], "planes")) planes();
#ifdef WITH_LIBRARY
    if (argc > 1 && !std::strcmp(argv[1], "refusals")) refusals();
    if (argc > 1 && !std::strcmp(argv[1], "grids")) grids();
    if (argc > 1 && !std::strcmp(argv[1], "no_rows")) no_rows();
    if (argc > 1 && !std::strcmp(argv[1], "factors")) factors();
#endif
    CHECK(checks > 0);
    std::printf(failures ? "%d of %d checks failed\n" : "%d of %d failed: all checks passed\n", failures, checks);
    return failures != 0;
}
