// What the vector verbs ask of the runtime, on the host alone: the runtime's
// launch functions are this program's, which hold every launch to the limits of
// a launch and run nothing.  No buffer is touched: addresses are made up.
// Usage: vector_launch_test grids | apart | contexts
#include "hgb_ctx.h"
#include "hgb_vector_plan.h"

#include <cstdint>
#include <cstdio>
#include <cstring>
#include <map>

using namespace hgb;

static int failures = 0, checks = 0, launches = 0;
static char what[200];

#define CHECK(cond, ...)                                  \
    do {                                                  \
        ++checks;                                         \
        if (!(cond) && ++failures <= 20) {                \
            std::printf("%s: %s: ", what, #cond);         \
            std::printf(__VA_ARGS__);                     \
            std::printf("\n");                            \
        }                                                 \
    } while (0)

extern "C" {

hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipGetLastError(void) { return hipSuccess; }

// a kernel's limit of dynamic LDS: one for the process, whoever sets it
static std::map<const void*, int> limits;

hipError_t hipFuncSetAttribute(const void* fn, hipFuncAttribute which, int value)
{
    if (which != hipFuncAttributeMaxDynamicSharedMemorySize || value < 0 || value > 163840) return hipErrorInvalidValue;
    limits[fn] = value;
    return hipSuccess;
}

// <<<grid, block, lds, stream>>>
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
    const int most_lds = limit == limits.end() ? 65536 : limit->second;
    CHECK(lds <= (size_t)most_lds, "%zu bytes of LDS, limit %d", lds, most_lds);
    const uint64_t most = (uint64_t)1 << 32;
    CHECK(grid.x > 0 && grid.y > 0 && grid.z > 0, "%u x %u x %u blocks", grid.x, grid.y, grid.z);
    CHECK(block.x * block.y * block.z <= 1024, "%u threads", block.x * block.y * block.z);
    CHECK((uint64_t)grid.x * block.x < most, "%u blocks of %u in x", grid.x, block.x);
    CHECK((uint64_t)grid.y * block.y < 65536, "%u blocks in y", grid.y);
    CHECK((uint64_t)grid.z * block.z < 65536, "%u blocks in z", grid.z);
    return hipSuccess;
}

}  // extern "C"

static char* at(int k) { return (char*)((uint64_t)(k + 1) << 57); }

// every verb at every size that its checks accept
static void grids()
{
    hgb_ctx c;   // no device behind it
    c.dev_words = (uint32_t*)4096;
    float* mean = (float*)at(10);
    int32_t *tok = (int32_t*)at(11), *pos = (int32_t*)at(12), *off = (int32_t*)at(13);
    void *ws = at(14), *a = at(1), *b = at(3), *d = at(5);
    float *w = (float*)at(15), *dw = (float*)at(16);
    const int64_t ns[] = {0, 1, 7, 4097, 1000000, 16777215, 16777216, 33554433, 67108864, 268435456, 1073741824, 2147483647};
    const int64_t dims[] = {1, 3, 8, 33, 64, 129, 257, 513, 1024, 1025, 1040, 2049, 5001, 16385, 1 << 20};
    auto ok = [&](hgb_status s) { CHECK(s == HGB_OK, "status %d, %s", s, c.err.c_str()); };
    for (int32_t type : {HGB_F32, HGB_BF16})
        for (int64_t dim : dims)
            for (int64_t n : ns) {
                std::snprintf(what, sizeof what, "type %d, %lld rows of %lld", type, (long long)n, (long long)dim);
                ok(hgb_embed(&c, a, type, dim, 1000, dim, tok, n, -1, 1, b, type, dim));
                ok(hgb_embed_backward(&c, a, type, dim, n, dim, tok, -1, 1, 1000, b, type, dim, ws, (int64_t)1 << 56));
                if (n > 0)
                    ok(hgb_embed_backward(&c, a, type, dim, 1000, dim, tok, -1, 1, std::min(n, kVecMaxVocab), b, type, dim, ws,
                                          (int64_t)1 << 56));
                ok(hgb_layer_norm(&c, a, type, dim, n, dim, w, dw, HGB_F32, 1e-5f, b, dim, mean, (float*)tok));
                ok(hgb_layer_norm_backward(&c, a, dim, b, dim, type, n, dim, mean, (float*)tok, w, HGB_F32, d, dim, dw, (float*)pos,
                                           ws, (int64_t)1 << 56));
                for (int32_t top : {1, 2, 7, 64}) {
                    const int64_t rows = n / top;
                    ok(hgb_route(&c, tok, rows, top, 700, (int32_t*)b, pos, off, ws, (int64_t)1 << 56));
                    ok(hgb_route_gather(&c, a, type, dim, rows, top, dim, pos, off, 700, b, dim));
                    ok(hgb_route_gather_backward(&c, a, type, dim, rows, top, dim, pos, b, dim));
                    ok(hgb_route_combine(&c, a, type, dim, rows, top, dim, pos, w, b, dim));
                    ok(hgb_route_combine_backward(&c, a, type, dim, b, dim, rows, top, dim, pos, off, 700, w, d, dim, dw));
                }
            }
}

// the blocks' numbers cover the work, and a number times what a block takes stays below 2^32
static void spans()
{
    const int64_t ns[] = {1, 255, 256, 16777216, 16777217, 67108865, 1073741823, 2147483646, 2147483647};
    auto check = [&](int64_t blocks, int64_t each) {
        std::snprintf(what, sizeof what, "%lld blocks of %lld", (long long)blocks, (long long)each);
        const GridSpan g = span_blocks(blocks);
        CHECK((int64_t)g.x * 256 < (int64_t)1 << 32 && g.z < 65536, "%u x %u", g.x, g.z);
        CHECK(g.z == 1 ? g.x == blocks : g.x == kGridBlocks, "%u x %u", g.x, g.z);
        CHECK((int64_t)g.x * g.z >= blocks && (int64_t)g.x * (g.z - 1) < blocks, "%u x %u", g.x, g.z);
        CHECK(((int64_t)g.x * g.z - 1) * each + each - 1 < (int64_t)1 << 32, "%u x %u", g.x, g.z);
    };
    for (int64_t n : ns) {
        for (int V : {4, 8})
            for (int64_t dim = 1; dim < 3000; ++dim) check(row_blocks(plan_rows(dim, V), n), plan_rows(dim, V).per);
        // the embedding gradient's chunk ends have their place in its workspace
        for (int64_t dim : {1, 7, 64, 129, 1040, 1 << 20})
            for (int64_t vocab : {(int64_t)1, (int64_t)7196, kVecMaxVocab}) {
                const EmbedPlan p = plan_embed(n, vocab, dim);
                std::snprintf(what, sizeof what, "%lld tokens of %lld, vocab %lld", (long long)n, (long long)dim, (long long)vocab);
                CHECK(p.off_ends >= p.off_part + p.chunks * 2 * p.part_stride * 4 && p.off_ends % 4 == 0, "ends at %lld", (long long)p.off_ends);
                CHECK(p.bytes >= p.off_ends + p.chunks * 4, "%lld bytes", (long long)p.bytes);
                CHECK(p.chunks * p.chunk >= n && p.chunks <= 2147483647, "%lld chunks", (long long)p.chunks);
            }
        for (int lg = 0; lg <= 6; ++lg) check(vec_ceil(n, 256 >> lg), 256 >> lg);   // slots by groups of lanes
    }
}

// arguments side by side in one buffer share no byte and are taken; those that share one are not
static void apart()
{
    hgb_ctx c;
    c.dev_words = (uint32_t*)4096;
    float* buf = (float*)at(1);
    float *mean = (float*)at(10), *rstd = (float*)at(11), *ws = (float*)at(14);
    int32_t *tok = (int32_t*)at(12), *pos = (int32_t*)at(13), *off = (int32_t*)at(15);
    const int32_t F = HGB_F32, B = HGB_BF16;
    auto is = [&](const char* name, hgb_status got, bool taken) {
        std::snprintf(what, sizeof what, "%s", name);
        CHECK(got == (taken ? HGB_OK : HGB_E_INVALID), "status %d, %s", got, c.err.c_str());
        CHECK(taken || std::strstr(c.err.c_str(), "overlaps"), "%s", c.err.c_str());
    };
    auto norm = [&](float* x, int64_t xs, float* y, int64_t ys, int64_t n, int64_t dim) {
        return hgb_layer_norm(&c, x, F, xs, n, dim, nullptr, nullptr, F, 1e-5f, y, ys, mean, rstd);
    };
    is("halves", norm(buf, 16, buf + 8, 16, 5, 8), true);
    is("halves, the output first", norm(buf + 8, 16, buf, 16, 5, 8), true);
    is("one value shared", norm(buf, 16, buf + 7, 16, 5, 8), false);
    is("one value shared with the next row", norm(buf, 16, buf + 9, 16, 5, 8), false);
    is("rows further on", norm(buf, 16, buf + 16 * 3 + 8, 16, 5, 8), true);
    is("rows further on, shared", norm(buf, 16, buf + 16 * 3, 16, 5, 8), false);
    is("behind the last row", norm(buf, 16, buf + 16 * 4 + 8, 16, 5, 8), true);
    is("the last row shared", norm(buf, 16, buf + 16 * 4 + 7, 16, 5, 8), false);
    is("one row between others", norm(buf, 16, buf + 8, 8, 1, 8), true);
    is("one row behind the other", norm(buf, 16, buf + 8, 99, 1, 8), true);
    is("strides of 32 and 16", norm(buf, 32, buf + 8, 16, 5, 8), true);
    is("strides of 32 and 16, shared", norm(buf, 32, buf + 4, 16, 5, 8), false);
    is("strides without room for both", norm(buf, 16, buf + 8, 17, 5, 8), false);
    is("far apart", norm(buf, 16, buf + 1000, 17, 5, 8), true);
    is("statistics in the rows' gap", hgb_layer_norm(&c, buf, F, 64, 5, 8, nullptr, nullptr, F, 1e-5f, buf + 16, 64, buf + 32, buf + 37), true);
    is("statistics across a row", hgb_layer_norm(&c, buf, F, 64, 5, 8, nullptr, nullptr, F, 1e-5f, buf + 16, 64, buf + 60, buf + 37), false);
    is("a table beside the output", hgb_embed(&c, buf, F, 24, 100, 8, tok, 50, -1, 1, buf + 8, B, 48), true);
    is("a table under the output", hgb_embed(&c, buf, F, 24, 100, 8, tok, 50, -1, 1, buf + 7, B, 48), false);
    is("the table's gradient beside the rows'",
       hgb_embed_backward(&c, buf, F, 20, 50, 8, tok, -1, 1, 30, buf + 12, F, 20, ws, 1 << 20), true);
    is("the table's gradient over the rows'",
       hgb_embed_backward(&c, buf, F, 20, 50, 8, tok, -1, 1, 30, buf + 13, F, 20, ws, 1 << 20), false);
    is("dx beside x and grad", hgb_layer_norm_backward(&c, buf, 24, buf + 8, 24, F, 5, 8, mean, rstd, nullptr, F, buf + 16, 24, nullptr,
                                                       nullptr, nullptr, 0), true);
    is("dx into grad's next row", hgb_layer_norm_backward(&c, buf, 24, buf + 8, 24, F, 5, 8, mean, rstd, nullptr, F, buf + 17, 24, nullptr,
                                                          nullptr, nullptr, 0), false);
    is("sorted rows beside the rows", hgb_route_gather(&c, buf, F, 16, 6, 2, 8, pos, off, 4, buf + 8, 16), true);
    is("sorted rows over the rows", hgb_route_gather(&c, buf, F, 16, 6, 2, 8, pos, off, 4, buf + 4, 16), false);
    is("answers beside the sums", hgb_route_combine(&c, buf, F, 16, 6, 2, 8, pos, nullptr, buf + 8, 16), true);
    is("answers' gradient beside the answers",
       hgb_route_combine_backward(&c, buf, F, 24, buf + 8, 24, 6, 2, 8, pos, off, 4, mean, buf + 16, 24, rstd), true);
    // extents that do not fit 64 bits
    is("a solid output in the gap of the largest extent",
       hgb_embed(&c, at(0), F, (int64_t)1 << 40, kVecMaxVocab, 8, tok, 50, -1, 1, at(0) + 32, F, 8), true);
    is("a solid output over its first row",
       hgb_embed(&c, at(0), F, (int64_t)1 << 40, kVecMaxVocab, 8, tok, 50, -1, 1, at(0) + 28, F, 8), false);
    is("the largest extents, side by side",
       hgb_embed(&c, at(0), F, (int64_t)1 << 40, kVecMaxVocab, 8, tok, 50, -1, 1, at(0) + 32, F, (int64_t)1 << 40), true);
}

// two contexts turn by turn, whose sorts take more and less LDS of one kernel
static void contexts()
{
    hgb_ctx a, b;
    a.dev_words = b.dev_words = (uint32_t*)4096;
    for (int64_t n : {3000, 300000, 1100000, 5000000})
        for (int experts : {1023, 200, 1023}) {
            std::snprintf(what, sizeof what, "%lld slots of %d experts", (long long)n, experts);
            for (hgb_ctx* c : {&a, &b, &a})
                CHECK(hgb_route(c, (int32_t*)at(1), n, 1, c == &a ? experts : 1223 - experts, (int32_t*)at(2), (int32_t*)at(3),
                                (int32_t*)at(4), at(5), (int64_t)1 << 56) == HGB_OK,
                      "%s", c->err.c_str());
        }
}

int main(int argc, char** argv)
{
    if (argc > 1 && !std::strcmp(argv[1], "grids")) {
        spans();
        grids();
    }
    if (argc > 1 && !std::strcmp(argv[1], "apart")) apart();
    if (argc > 1 && !std::strcmp(argv[1], "contexts")) contexts();
    CHECK(launches > 0, "nothing was launched");
    std::printf(failures ? "%d of %d checks failed\n" : "%d of %d failed: all checks passed\n", failures, checks);
    return failures != 0;
}
