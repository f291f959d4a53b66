// The vector verbs' plans (hgb_vector_plan.h) and the refusals of their C
// entry points, on the host alone: every call here is refused before it
// touches a device.  Usage: vector_test plan | vector_test refusals
#include "hgb_vector_plan.h"

#include <cstdio>
#include <cstring>

#ifdef WITH_LIBRARY
#include "hgb_ctx.h"
#endif

using namespace hgb;

static int failures = 0, checks = 0;

#define CHECK(cond)                                                     \
    do {                                                                \
        ++checks;                                                       \
        if (!(cond)) {                                                  \
            ++failures;                                                 \
            std::printf("line %d: %s\n", __LINE__, #cond);              \
        }                                                               \
    } while (0)

static void plans()
{
    const int64_t ns[] = {1, 2, 63, 64, 65, 1024, 1025, 4097, 16383, 16384, 16385, 100000, 3670016, 8388608, 8388609,
                          100000000, 2147483647};
    const int64_t limits[] = {1, 2, 3, 63, 64, 255, 256, 1022, 1023, 1024, 7196, 65535, 262144, 1 << 20, 2147483646};
    for (int64_t n : ns)
        for (int64_t limit : limits)
            for (int one = 0; one < 2; ++one) {
                if (one && limit > kRouteMaxExperts) continue;
                const SortPlan p = plan_sort(n, limit, one);
                CHECK(p.passes >= 1 && (!one || p.passes == 1));
                CHECK((int64_t)p.bits * p.passes >= vec_bits(limit) && p.bits <= kSortBits);
                CHECK(p.radix == 1 << p.bits && p.radix <= kSortThreads);
                CHECK(p.small == (n <= kSortSmall));
                int bits = 0;
                for (int k = 0; k < p.passes; ++k) {
                    const SortPlan q = p.pass(k);
                    CHECK(q.bits >= 1 && q.bits <= p.bits && q.radix == 1 << q.bits && q.row >= q.radix && q.row <= p.row);
                    CHECK(k * p.bits == bits);   // its digits begin where the last one's end
                    bits += q.bits;
                }
                CHECK(bits == vec_bits(limit));
                CHECK(p.items == 1 || p.items == 4 || p.items == kSortItems);
                const int64_t tile = (int64_t)p.items * kSortThreads;
                // the blocks' shares cover every key, and none starts past the last
                CHECK(p.blocks >= 1 && p.blocks <= kSortMaxBlocks);
                CHECK(p.blocks * p.tiles * tile >= n);
                CHECK((p.blocks - 1) * p.tiles * tile < n);
                if (p.small) {
                    CHECK(p.blocks == 1 && p.tiles == 1 && p.items <= 4 && !p.count);
                    const int64_t pairs = p.passes > 1 ? 2 * tile : 0;
                    CHECK(4 * (pairs + 16 * (int64_t)p.radix + p.radix + 16) <= 163840);
                } else {
                    CHECK(4 * (scatter_pair_words(p.items) + 18 * (int64_t)p.radix + 16) <= 163840);
                    CHECK(p.count || p.blocks <= kSortSelf);
                }
            }
    for (int64_t n : ns)
        for (int64_t dim : {(int64_t)1, (int64_t)7, (int64_t)64, (int64_t)129, (int64_t)1792, (int64_t)1 << 20}) {
            const EmbedPlan p = plan_embed(n, 7196, dim);
            CHECK(p.chunk >= 1 && p.chunk <= kEmbedChunk && p.chunks * p.chunk >= n && (p.chunks - 1) * p.chunk < n);
            CHECK(p.part_stride >= dim && p.part_stride % 4 == 0);
            CHECK(p.off_a >= (p.sort.count ? (int64_t)p.sort.blocks * p.sort.radix * 4 : 0) && p.off_a % 16 == 0);
            CHECK(p.off_b >= p.off_a + n * 8 && p.off_b % 16 == 0);
            CHECK(p.off_part >= p.off_b + (p.sort.passes > 1 && !p.sort.small ? n * 8 : 0) && p.off_part % 16 == 0);
            CHECK(p.bytes >= p.off_part + p.chunks * 2 * p.part_stride * 4);
            CHECK(norm_parts(n) >= 1 && norm_parts(n) <= kNormParts);
            CHECK(norm_workspace(n, dim) >= norm_parts(n) * dim * 8);
        }
    CHECK(norm_parts(0) == 1);
    for (int64_t dim = 1; dim <= 20000; ++dim) {
        const NormPlan p = plan_norm(dim);
        CHECK((p.values > 0) == (dim <= kNormMaxDim));
        if (!p.values) continue;
        const int64_t span = p.waves > 1 ? 64 * p.waves : 1 << p.log_group, columns = span * p.values;
        CHECK(columns >= dim && p.log_group <= 6 && (p.waves == 1 || p.log_group == 6));
        // with more than 8 values a lane the kernels take the lower half of the columns to be in the row
        CHECK(p.values == 8 || 2 * dim > columns);
        CHECK(p.values > 8 || p.waves == 1);
        CHECK(p.per_block * span == norm_threads(p.waves));
        for (int64_t n : ns) {
            CHECK(norm_blocks(n, p) >= 1 && norm_blocks(n, p) <= 2 * kNormParts);
            CHECK(norm_workspace(n, dim) >= (int64_t)norm_blocks(n, p) * dim * 8);
        }
    }
    for (int V : {4, 8})
        for (int64_t dim = 1; dim < 6000; ++dim) {
            const RowMap m = plan_rows(dim, V);
            CHECK((int64_t)m.vecs * V >= dim && (int64_t)(m.vecs - 1) * V < dim);
            CHECK(m.slices * 256 >= m.vecs && (m.slices - 1) * 256 < m.vecs);
            CHECK(m.per >= 1 && (m.per == 1 || m.per * m.vecs <= 256) && row_blocks(m, 1000) * m.per >= 1000);
            for (int t = 0; t < 256; ++t) CHECK((t * m.magic) >> 16 == t / m.vecs);
        }
}

#ifdef WITH_LIBRARY
static void refusals()
{
    hgb_ctx c;   // no device behind it
    float f[64] = {};
    int32_t i[64] = {};
    char ws[4096];
    const int64_t big = (int64_t)1 << 31;
    auto is = [&](hgb_status got, hgb_status want, const char* word) {
        ++checks;
        if (got != want || !std::strstr(c.err.c_str(), word)) {
            ++failures;
            std::printf("got %d \"%s\", wanted %d \"%s\"\n", got, c.err.c_str(), want, word);
        }
    };
    const int32_t F = HGB_F32, B = HGB_BF16;
    // embed(ctx, table, type, stride, vocab, dim, tokens, n, pad, scale, out, type, stride)
    is(hgb_embed(&c, nullptr, F, 4, 3, 4, i, 5, -1, 1, f, F, 4), HGB_E_INVALID, "table is null");
    is(hgb_embed(&c, f, 7, 4, 3, 4, i, 5, -1, 1, f, F, 4), HGB_E_INVALID, "unknown type");
    is(hgb_embed(&c, f, F, 3, 3, 4, i, 5, -1, 1, f, F, 4), HGB_E_INVALID, "overlap");
    is(hgb_embed(&c, (char*)f + 2, F, 4, 3, 4, i, 5, -1, 1, f, F, 4), HGB_E_INVALID, "aligned");
    is(hgb_embed(&c, f, F, 4, 0, 4, i, 5, -1, 1, f, F, 4), HGB_E_INVALID, "vocab");
    is(hgb_embed(&c, f, F, 4, 2147483647, 4, i, 5, -1, 1, f, F, 4), HGB_E_INVALID, "vocab");
    is(hgb_embed(&c, f, F, 4, 3, 0, i, 5, -1, 1, f, F, 4), HGB_E_INVALID, "dim");
    is(hgb_embed(&c, f, F, 1 << 21, 3, 1 << 21, i, 5, -1, 1, f, F, 1 << 21), HGB_E_UNSUPPORTED, "dim");
    is(hgb_embed(&c, f, F, 4, 3, 4, i, big, -1, 1, f, F, 4), HGB_E_INVALID, "rows");
    is(hgb_embed(&c, f, F, 4, 3, 4, i, -1, -1, 1, f, F, 4), HGB_E_INVALID, "rows");
    is(hgb_embed(&c, f, F, 4, 3, 4, nullptr, 5, -1, 1, f + 32, F, 4), HGB_E_INVALID, "tokens");
    is(hgb_embed(&c, f, B, 4, 3, 4, i, 5, -1, 1, f + 32, F, 4), HGB_E_UNSUPPORTED, "type");
    is(hgb_embed(&c, f, F, 4, 3, 4, i, 5, -1, 1, f + 11, F, 4), HGB_E_INVALID, "overlaps");
    is(hgb_embed_backward(&c, f, F, 4, 5, 4, i, -1, 1, 3, f + 32, F, 4, ws, 16), HGB_E_INVALID, "workspace");
    is(hgb_embed_backward(&c, f, F, 4, 5, 4, i, -1, 1, 3, f + 32, F, 4, nullptr, 1 << 20), HGB_E_INVALID, "workspace");
    is(hgb_embed_backward(&c, f, F, 4, 5, 4, i, -1, 1, 3, f + 32, B, 4, ws, 4096), HGB_E_UNSUPPORTED, "grad");
    is(hgb_embed_backward(&c, f, F, 4, 5, 4, i, -1, 1, 3, f + 19, F, 4, ws, 4096), HGB_E_INVALID, "overlaps");
    CHECK(hgb_embed_backward_workspace(-1, 3, 4) == -1 && hgb_embed_backward_workspace(5, 0, 4) == -1);
    CHECK(hgb_embed_backward_workspace(5, 3, 0) == -1 && hgb_embed_backward_workspace(0, 3, 4) == 0);
    // layer_norm(ctx, x, type, stride, rows, dim, weight, bias, ptype, eps, y, stride, mean, rstd)
    is(hgb_layer_norm(&c, f, F, 4, 2, 4, f + 40, f + 44, B, 1e-5f, f + 8, 4, f + 50, f + 52), HGB_E_UNSUPPORTED, "parameters");
    is(hgb_layer_norm(&c, f, F, 4, 2, 4, nullptr, nullptr, F, -1e-5f, f + 8, 4, f + 50, f + 52), HGB_E_INVALID, "eps");
    is(hgb_layer_norm(&c, f, F, 4, 2, 4, nullptr, nullptr, F, 1e-5f, f + 8, 4, nullptr, f + 52), HGB_E_INVALID, "mean");
    is(hgb_layer_norm(&c, f, F, 4, 2, 4, nullptr, nullptr, F, 1e-5f, f + 7, 4, f + 50, f + 52), HGB_E_INVALID, "overlaps");
    is(hgb_layer_norm_backward(&c, f, 4, f + 8, 4, F, 2, 4, f + 50, f + 52, nullptr, F, f + 16, 4, nullptr, f + 40, ws, 8),
       HGB_E_INVALID, "workspace");
    is(hgb_layer_norm_backward(&c, f, 4, f + 8, 4, F, 2, 4, f + 50, f + 52, nullptr, F, f, 4, nullptr, nullptr, ws, 8),
       HGB_E_INVALID, "overlaps");
    is(hgb_layer_norm_backward(&c, f, 4, f + 8, 4, F, 2, 4, nullptr, f + 52, nullptr, F, f + 16, 4, nullptr, nullptr, ws, 8),
       HGB_E_INVALID, "mean");
    CHECK(hgb_layer_norm_backward_workspace(-1, 4) == -1 && hgb_layer_norm_backward_workspace(4, 0) == -1);
    // route
    is(hgb_route(&c, i, 4, 0, 3, i + 8, i + 16, i + 24, nullptr, 0), HGB_E_INVALID, "top");
    is(hgb_route(&c, i, 4, 65, 3, i + 8, i + 16, i + 24, nullptr, 0), HGB_E_UNSUPPORTED, "top");
    is(hgb_route(&c, i, big / 2, 2, 3, i + 8, i + 16, i + 24, nullptr, 0), HGB_E_INVALID, "slots");
    is(hgb_route(&c, i, 4, 2, 0, i + 8, i + 16, i + 24, nullptr, 0), HGB_E_INVALID, "n_experts");
    is(hgb_route(&c, i, 4, 2, 1024, i + 8, i + 16, i + 24, nullptr, 0), HGB_E_UNSUPPORTED, "n_experts");
    is(hgb_route(&c, nullptr, 4, 2, 3, i + 8, i + 16, i + 24, nullptr, 0), HGB_E_INVALID, "experts");
    is(hgb_route(&c, i, 4, 2, 3, i + 8, nullptr, i + 24, nullptr, 0), HGB_E_INVALID, "position");
    is(hgb_route(&c, i, 4, 2, 3, i + 8, i + 16, nullptr, nullptr, 0), HGB_E_INVALID, "offsets");
    is(hgb_route(&c, i, 20000, 2, 3, i + 8, i + 16, i + 24, ws, 4), HGB_E_INVALID, "workspace");
    CHECK(hgb_route_workspace(4, 2, 1024) == -1 && hgb_route_workspace(4, 2, 3) == 0 && hgb_route_workspace(20000, 2, 3) > 0);
    is(hgb_route_gather(&c, f, F, 4, 2, 2, 4, i, nullptr, 3, f + 8, 4), HGB_E_INVALID, "offsets");
    is(hgb_route_gather(&c, f, F, 4, 2, 2, 4, i, i, 3, f + 4, 4), HGB_E_INVALID, "overlaps");
    is(hgb_route_combine(&c, nullptr, F, 4, 2, 2, 4, i, f, f + 32, 4), HGB_E_INVALID, "null");
    is(hgb_route_combine(&c, f, F, 4, 2, 2, 4, i, nullptr, f + 12, 4), HGB_E_INVALID, "overlaps");
    is(hgb_route_gather_backward(&c, f, F, 4, 2, 2, 4, nullptr, f + 32, 4), HGB_E_INVALID, "position");
    is(hgb_route_combine_backward(&c, f, F, 4, f + 8, 4, 2, 2, 4, i, nullptr, 3, f, f + 24, 4, f + 60), HGB_E_INVALID, "offsets");
    is(hgb_route_combine_backward(&c, f, F, 4, f + 8, 4, 2, 2, 4, i, i, 3, f, f + 8, 4, f + 60), HGB_E_INVALID, "overlaps");
    // every pointer's alignment, and every output against every input and the other outputs
    int32_t* odd = (int32_t*)((char*)i + 2);
    is(hgb_embed(&c, f, F, 4, 3, 4, odd, 5, -1, 1, f + 32, F, 4), HGB_E_INVALID, "aligned");
    is(hgb_embed(&c, f, F, 4, 3, 4, (int32_t*)(f + 36), 5, -1, 1, f + 32, F, 4), HGB_E_INVALID, "overlaps");
    is(hgb_embed_backward(&c, f, F, 4, 5, 4, i, -1, 1, 3, f + 32, F, 4, f + 40, 1 << 20), HGB_E_INVALID, "overlaps");
    is(hgb_layer_norm(&c, f, F, 4, 2, 4, f + 8, nullptr, F, 1e-5f, f + 9, 4, f + 50, f + 52), HGB_E_INVALID, "overlaps");
    is(hgb_layer_norm(&c, f, F, 4, 2, 4, nullptr, nullptr, F, 1e-5f, f + 16, 4, f + 50, f + 51), HGB_E_INVALID, "another");
    is(hgb_layer_norm(&c, f, F, 4, 2, 4, nullptr, nullptr, F, 1e-5f, f + 16, 4, (float*)odd, f + 51), HGB_E_INVALID, "aligned");
    is(hgb_layer_norm_backward(&c, f, 4, f + 8, 4, F, 2, 4, f + 50, f + 52, nullptr, F, f + 16, 4, f + 40, f + 41, ws, 4096),
       HGB_E_INVALID, "another");
    is(hgb_layer_norm_backward(&c, f, 4, f + 8, 4, F, 2, 4, f + 50, f + 52, nullptr, F, f + 16, 4, f + 40, f + 44, f + 48, 4096),
       HGB_E_INVALID, "overlaps");
    is(hgb_route(&c, i, 4, 2, 3, i + 4, i + 16, i + 24, nullptr, 0), HGB_E_INVALID, "overlaps");
    is(hgb_route(&c, i, 4, 2, 3, i + 8, i + 12, i + 24, nullptr, 0), HGB_E_INVALID, "another");
    is(hgb_route(&c, odd, 4, 2, 3, i + 8, i + 16, i + 24, nullptr, 0), HGB_E_INVALID, "aligned");
    is(hgb_route_gather(&c, f, F, 4, 2, 2, 4, odd, i, 3, f + 8, 4), HGB_E_INVALID, "aligned");
    is(hgb_route_gather(&c, f, F, 4, 2, 2, 4, (int32_t*)(f + 20), i, 3, f + 8, 4), HGB_E_INVALID, "overlaps");
    is(hgb_route_combine(&c, f, F, 4, 2, 2, 4, i, f + 33, f + 32, 4), HGB_E_INVALID, "overlaps");
    is(hgb_route_combine_backward(&c, f, F, 4, f + 8, 4, 2, 2, 4, i, i + 8, 3, f, f + 24, 4, f + 39), HGB_E_INVALID, "another");
    CHECK(hgb_embed(nullptr, f, F, 4, 3, 4, i, 5, -1, 1, f, F, 4) == HGB_E_INVALID);
    CHECK(hgb_route(nullptr, i, 4, 2, 3, i, i, i, nullptr, 0) == HGB_E_INVALID);
}
#endif

int main(int argc, char** argv)
{
    if (argc > 1 && !std::strcmp(argv[1], "plan")) plans();
#ifdef WITH_LIBRARY
    else refusals();
#endif
    std::printf(failures ? "%d of %d checks failed\n" : "%d of %d failed: all checks passed\n", failures, checks);
    return failures != 0;
}
