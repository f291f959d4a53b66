// The context (hgb_ctx) and what every entry point needs of it: error
// reporting, launch checks and the per-class timing.  Internal header of
// hgb.hip and hgb_vectors.hip.
#pragma once

#include "hgb.h"
#include "hgb_plan.h"

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <string>
#include <utility>
#include <vector>

namespace hgb {

struct FeatureBest;   // hgb_kernels.h
struct LevelBest;

// Default fixed-point precision of begin_tree (bits below the largest value).
constexpr int kDefaultPrecision = 30;
constexpr int kStages = 16;
constexpr int kEpochEvents = 4;
constexpr int kEpochUses = 6;
// The device and pinned host word in which the vector verbs' kernels flag a
// token or an expert out of range (apart from word 2, which partition_level
// reads and clears).
constexpr int kWordVectors = 12;
constexpr uint32_t kVecErrToken = 1u;
constexpr uint32_t kVecErrExpert = 2u;

struct Stage {
    void* host = nullptr;   // pinned
    void* dev = nullptr;
    size_t cap = 0;
    uint64_t release_seq = 0;    // the context's release count when its consumers were enqueued
    bool pending = false;
    const void* use = nullptr;   // what the kernels read: dev, or the pinned host copy
};

}  // namespace hgb

struct hgb_ctx {
    int device = 0;
    int n_cu = 256;
    hipStream_t stream = nullptr;
    std::string err;

    // dataset plane: feature-major bins, plus a row-major copy when rows are
    // narrow enough for a row to sit in a cache line or two
    void* bins = nullptr;
    void* bins_rm = nullptr;
    int64_t rm_stride = 0;   // bytes per row of the row-major copy (multiple of 16)
    int bin_bytes = 0;
    int64_t n = 0;
    int F = 0, B = 0, S = 0, has_missing = 0;
    bool have_data = false;

    // gradient plane
    int2* q = nullptr;
    int64_t q_cap = 0;
    int precision = hgb::kDefaultPrecision;
    int k_g = 0, k_h = 0;
    bool have_tree = false;
    // hgb_set_async_begin: begin_tree returns without waiting for the maxima;
    // the host reads them (and checks them) at the next call that needs them
    bool async_begin = false;
    bool scales_pending = false;          // the current tree's maxima are not read yet
    int tree_precision = 30;              // the precision the current tree was started with
    hgb_status deferred = HGB_OK;         // a started tree's non-finite values, for hgb_sync
    std::string deferred_msg;

    // level scratch
    int2* gh = nullptr;
    int64_t gh_cap = 0;
    long long* partial = nullptr;   // partial histograms of nodes split over several blocks
    int64_t partial_cap = 0;
    int32_t* part = nullptr;        // partition: chunk counts, left bases, per-node records
    int64_t part_cap = 0;
    int32_t* part_host = nullptr;   // pinned copy of the per-node records
    int64_t part_host_cap = 0;
    uint8_t* part_flags = nullptr;  // partition: direction of each position (1 = left)
    int64_t part_flags_cap = 0;
    hgb::FeatureBest* best = nullptr;
    int64_t best_cap = 0;
    long long* totals = nullptr;
    int64_t totals_cap = 0;
    double* level_terms = nullptr;        // find_level_split: [n_nodes][candidates] gains
    int64_t level_terms_cap = 0;
    hgb::LevelBest* level_best = nullptr;      // find_level_split: per-block winners
    int64_t level_best_cap = 0;

    // this device's copy of the no-allocation scratch array (set up by hgb_create)
    unsigned char* noalloc_scratch = nullptr;

    // small device words: [0..1] max patterns, [2] error flags, [3] 1 when the
    // quantize pass must encode the rows again, [4..11] the quantize scales
    // 2^k (also the next tree's guess) and the split scales 2^-k (four doubles)
    uint32_t* dev_words = nullptr;
    uint32_t* host_words = nullptr;   // pinned
    uint32_t* max_part = nullptr;     // begin_tree: per-block maxima, 2 x kMaxBlocks
    int32_t* rot = nullptr;           // per feature: the skipped slot (stored bins are rotated by it)
    bool skip = false;                // the fills skip each feature's slot 0 (a hot slot exists)
    hipEvent_t host_ready = nullptr;  // hgb_sync: the stream has drained

    hgb::Stage stage[hgb::kStages];
    int stage_next = 0;
    // Stage releases record no event of their own (an event on the stream
    // costs the device about 3 us): every kEpochUses releases, one event of a
    // small ring marks the stream, and a stage is reused once an event
    // recorded after its release has passed.
    uint64_t stage_seq = 0;                     // releases so far
    hipEvent_t epoch_ev[hgb::kEpochEvents] = {};
    uint64_t epoch_seq[hgb::kEpochEvents] = {};      // releases covered by each event
    int epoch_next = 0;
    uint64_t last_epoch_seq = 0;
    // sequence numbers of the results kernels post to pinned host memory:
    // the maxima of each tree (host_words[8]) and the node records of each
    // partition (host_words[9])
    uint32_t tree_seq = 0;
    uint32_t part_seq = 0;

    // HGB_DEBUG_PLAN=1 in the environment prints each fill plan to stderr
    bool debug_plan = false;
    // kernels read the launch plans from pinned host memory (HGB_PLAN_HOST=0:
    // from a device copy)
    bool plan_host = true;
    // HGB_FILL_TUNE="key=value,..." overrides the fill planner (developer
    // tuning): root_lc, root_tile, root_ipc, level_lc, level_tile, level_ipc
    // (ipc = items per CU), align (rows an item boundary is a multiple of),
    // piece (fixed cost of a level item, in rows), il (row-major level fill,
    // wide sums) and root_il (root fill, wide or packed sums): 1 slot-major
    // interleaved tile, 0 feature-major; pair (row-major interleaved level
    // fills with 32-byte chunks: 1 two lanes per row, 0 one); -1 keeps the
    // planner's choice.
    int tune[hgb::kTuneKeys] = {-1, -1, -1, -1, -1, -1, -1, -1, -1, -1, -1};

    // optional per-kernel timing
    bool prof = false;
    std::vector<hipEvent_t> ev_pool;
    // kernels whose dynamic-LDS limit has been raised (raise_lds)
    std::vector<const void*> lds_set;
    std::vector<std::pair<hipEvent_t, hipEvent_t>> ev_pending[HGB_KERNEL_COUNT];
    double prof_ms[HGB_KERNEL_COUNT] = {};
    int64_t prof_launches[HGB_KERNEL_COUNT] = {};
};

namespace hgb {

inline hgb_status fail(hgb_ctx* c, hgb_status st, const char* fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    c->err = buf;
    return st;
}

#define HGB_HIP(c, expr)                                                                   \
    do {                                                                                   \
        hipError_t e_ = (expr);                                                            \
        if (e_ != hipSuccess)                                                              \
            return fail((c), HGB_E_DEVICE, "%s failed: %s", #expr, hipGetErrorString(e_)); \
    } while (0)

#define HGB_LAUNCHED(c, what)                                                              \
    do {                                                                                   \
        hipError_t e_ = hipGetLastError();                                                 \
        if (e_ != hipSuccess)                                                              \
            return fail((c), HGB_E_DEVICE, "launch of %s failed: %s", what,                \
                        hipGetErrorString(e_));                                            \
    } while (0)

// Lets a kernel (without LDS arrays of its own) be launched with all the LDS of
// a CU.  The limit is the kernel's in the process, so every context sets it to
// the same: one that set what its own launch needs could lower another's.
constexpr int kLdsBytes = 160 * 1024;

template <typename K>
hgb_status raise_lds(hgb_ctx* c, K kernel)
{
    const void* fn = (const void*)kernel;
    for (const void* f : c->lds_set)
        if (f == fn) return HGB_OK;
    HGB_HIP(c, hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, kLdsBytes));
    c->lds_set.push_back(fn);
    return HGB_OK;
}

inline hipEvent_t pool_event(hgb_ctx* c)
{
    if (!c->ev_pool.empty()) {
        hipEvent_t e = c->ev_pool.back();
        c->ev_pool.pop_back();
        return e;
    }
    hipEvent_t e = nullptr;
    if (hipEventCreate(&e) != hipSuccess) return nullptr;
    return e;
}

// Brackets the launches of one kernel class with events when timing is on.
struct ProfScope {
    hgb_ctx* c;
    int kernel;
    hipEvent_t start = nullptr;
    ProfScope(hgb_ctx* ctx, int k) : c(ctx), kernel(k)
    {
        if (!c->prof) return;
        start = pool_event(c);
        if (start && hipEventRecord(start, c->stream) != hipSuccess) {
            c->ev_pool.push_back(start);
            start = nullptr;
        }
    }
    ~ProfScope()
    {
        if (!start) return;
        hipEvent_t stop = pool_event(c);
        if (stop && hipEventRecord(stop, c->stream) == hipSuccess) {
            c->ev_pending[kernel].emplace_back(start, stop);
        } else {
            c->ev_pool.push_back(start);
            if (stop) c->ev_pool.push_back(stop);
        }
    }
};

}  // namespace hgb
