// verkv_api.cu -- the C ABI of libverkv: argument checks, workspace carve-up, stream and event
// orchestration, and the host side of the fetch ("Verify Before You Fetch": the abstract page's
// GPU-resident pivotal tokens and sketch with the complete cache in CPU memory; summary page,
// KVFETCH steps 1-5).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <condition_variable>
#include <functional>
#include <mutex>
#include <string>
#include <thread>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "paged.cuh"
#include "verkv_internal.h"

using namespace verkv;

namespace {

// An NVTX range for the lifetime of the object: each stage of the hot path shows up by name on a
// profiler's timeline (the calls cost nothing without a tool attached).
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Alignment the kernels rely on: bf16 rows and queries are read in 16-byte vectors or bulk
// copies; every other array is read and written in 4-byte words.  A null pointer passes (the
// null checks are separate).
bool bad16(const void *p) { return ((uintptr_t)p & 15u) != 0; }
bool bad4(const void *p) { return ((uintptr_t)p & 3u) != 0; }

struct Layout {
    size_t err, flc, nacc, rmask, rnext, scores, qstats, F, slb, fids, fcounts, staging, part_piv, part_fet, total;
    int W, units_layer, qh_layer, max_piv, max_fet, dense_chunks;
};

// MEMCPY-mode staging (page-locked on the host and its device copy): a header of the layer
// units' first staged rows (int64, 256-byte aligned), then the fetched rows of every unit,
// contiguous and unit by unit, so that one copy moves a whole fetch.
size_t staging_header(int units_layer) { return align256((size_t)units_layer * 8); }
size_t staging_bytes(int units_layer, size_t n, size_t d) {
    return staging_header(units_layer) + (size_t)units_layer * n * 4 * d;
}

bool valid_shape(const verkv_shape *s) {
    if (!s) return false;
    const int G = s->q_per_kv;
    return s->batch >= 1 && s->layers >= 1 && s->kv_heads >= 1 &&
           (G == 1 || G == 2 || G == 4 || G == 8) && (s->head_dim == 64 || s->head_dim == 128) &&
           s->n >= 1 && s->n <= 131072 && s->cap >= 1 && s->cap <= s->n &&
           (int64_t)s->batch * s->layers * s->kv_heads <= (1 << 24);
}

bool make_layout(const verkv_shape *s, Layout &L) {
    if (!valid_shape(s)) return false;
    const size_t n = (size_t)s->n, d = (size_t)s->head_dim, G = (size_t)s->q_per_kv;
    L.W = (s->n + 31) / 32;
    L.units_layer = s->batch * s->kv_heads;
    L.qh_layer = L.units_layer * s->q_per_kv;
    L.max_piv = (s->cap + PIV_ITEM_ROWS - 1) / PIV_ITEM_ROWS;
    L.max_fet = (s->n + FET_RANGE - 1) / FET_RANGE;
    L.dense_chunks = (s->n + PART_ROWS - 1) / PART_ROWS;  // >= max_fet: sizes the shared buffer
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = align256(off + bytes);
        return o;
    };
    L.err = take(256);
    L.flc = take((size_t)L.units_layer * 4);
    L.nacc = take((size_t)L.qh_layer * 4);
    L.rmask = take((size_t)L.units_layer * RMASK_W * 4);
    L.rnext = take(4);
    L.scores = take((size_t)L.qh_layer * n * 4);
    L.qstats = take((size_t)L.qh_layer * sizeof(verkv_head_stats));
    L.F = take((size_t)L.qh_layer * L.W * 4);
    L.slb = take((size_t)L.units_layer * L.W * 4);
    L.fids = take((size_t)L.units_layer * n * 4);
    L.fcounts = take((size_t)L.units_layer * 4);
    L.staging = take(staging_bytes(L.units_layer, n, d));
    L.part_piv = take((size_t)L.units_layer * L.max_piv * G * (d + 2) * 4);
    L.part_fet = take((size_t)L.units_layer * L.dense_chunks * G * (d + 2) * 4);
    L.total = off;
    return true;
}

// A small fixed pool of host threads for the MEMCPY-mode gather.
class Pool {
  public:
    explicit Pool(int nthreads) {
        for (int i = 0; i < nthreads; ++i) workers_.emplace_back([this, i] { loop(i); });
    }
    ~Pool() {
        {
            std::lock_guard<std::mutex> g(mu_);
            stop_ = true;
        }
        cv_.notify_all();
        for (auto &t : workers_) t.join();
    }
    int size() const { return (int)workers_.size(); }
    // Runs fn(worker_index) on every worker and waits for all of them.
    void run(const std::function<void(int)> &fn) {
        std::unique_lock<std::mutex> lk(mu_);
        job_ = &fn;
        pending_ = (int)workers_.size();
        ++generation_;
        cv_.notify_all();
        done_cv_.wait(lk, [this] { return pending_ == 0; });
        job_ = nullptr;
    }

  private:
    void loop(int idx) {
        uint64_t seen = 0;
        for (;;) {
            const std::function<void(int)> *job;
            {
                std::unique_lock<std::mutex> lk(mu_);
                cv_.wait(lk, [&] { return stop_ || generation_ != seen; });
                if (stop_) return;
                seen = generation_;
                job = job_;
            }
            (*job)(idx);
            {
                std::lock_guard<std::mutex> g(mu_);
                if (--pending_ == 0) done_cv_.notify_all();
            }
        }
    }
    std::vector<std::thread> workers_;
    std::mutex mu_;
    std::condition_variable cv_, done_cv_;
    const std::function<void(int)> *job_ = nullptr;
    int pending_ = 0;
    uint64_t generation_ = 0;
    bool stop_ = false;
};

}  // namespace

namespace verkv {

cudaError_t ensure_smem(const void *func, size_t bytes) {
    struct Entry {
        int device;
        const void *func;
        size_t bytes;
    };
    static std::mutex mu;
    static std::vector<Entry> done;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> g(mu);
    for (Entry &x : done) {
        if (x.device == dev && x.func == func) {
            if (x.bytes >= bytes) return cudaSuccess;
            e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
            if (e == cudaSuccess) x.bytes = bytes;
            return e;
        }
    }
    e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.push_back({dev, func, bytes});
    return e;
}

}  // namespace verkv

struct verkv_ctx {
    int device = 0;
    int sms = 0;
    cudaStream_t main = nullptr, side = nullptr;
    // Of MEMCPY mode.  e_sel: behind the last selection made outside a capture, the last to touch the host buffers on
    // `main`; e_cap: behind one in a capture; selected: which of the two the last selection has.
    cudaEvent_t e_sel = nullptr, e_fetch = nullptr, e_cap = nullptr, selected = nullptr;
    verkv_shape sh{};
    Layout L{};
    unsigned char *ws = nullptr;
    uint32_t *err = nullptr;
    float *scores = nullptr;
    verkv_head_stats *qstats = nullptr;
    uint32_t *F = nullptr;
    int32_t *fids = nullptr, *fcounts = nullptr;
    int32_t *flc = nullptr;  // per-KV-head completion counters of the certify kernel's fetch list
    int32_t *nacc = nullptr; // per-query-head n_fetch accumulators of the zero-copy refine
    uint32_t *rmask = nullptr; // per-KV-head masks of fetched-row ranges holding rows
    int32_t *rnext = nullptr;  // the zero-copy refine's item counter
    uint32_t *slb = nullptr; // per-KV-head shortlist bitmaps
    int shortlist = 0;       // shortlist size per KV head; 0: every token of L may be fetched
    bool shortlisted = false;  // the last attend built shortlists
    uint16_t *staging = nullptr;
    float *part_piv = nullptr, *part_fet = nullptr;
    int fetch_mode = VERKV_FETCH_ZEROCOPY;
    bool fetch_keys = false;  // move K rows too, although the exact sketch holds every key
    // MEMCPY mode
    unsigned char *host_staging = nullptr;
    int32_t *host_ids = nullptr, *host_counts = nullptr;     // mapped page-locked
    int32_t *host_ids_dev = nullptr, *host_counts_dev = nullptr;
    Pool *pool = nullptr;
    // The preceding attend
    bool pending = false;
    bool attended = false;
    int layer = 0;
    verkv_pivotal piv{};
    const int32_t *user_ids = nullptr, *user_counts = nullptr;
    const void *q = nullptr;
    const void *sketch = nullptr;
    bool sketch_exact = true;  // format of the preceding attend's sketch
    std::string last_error;
    // Failure injection (verkv_test_inject)
    int64_t inject_copy_fail = 0;    // fetch copies still to fail on the host
    int beta_maxit = 0;              // 0: the kernel's default cap
    int sel_gather = 1;              // the select's gathered finish (clusters of 1 and 4)
    int seq0 = 0;                    // Philox sequence index of this context's first sequence
    int64_t score_stall_ns = 0;      // > 0: the next attend's scoring kernel stalls one stage
    int64_t paged_wait_ns = 0;       // > 0: limit of the next paged attention's waits
    bool paged_stall = false;        // and its kernels stall one step each
    int64_t weigh_stall_ns = 0;      // > 0: the next paged_weigh's kernel for many rows stalls, and its limit
    // Measurement
    int64_t launches[VERKV_K_COUNT] = {};
    bool prof_on = false;
    std::vector<cudaEvent_t> prof_pool;
    size_t prof_used = 0;
    struct Rec {
        int kernel;
        cudaEvent_t a, b;
    };
    std::vector<Rec> prof_recs;
};

namespace {

verkv_status fail(verkv_ctx *c, verkv_status st, const std::string &msg) {
    if (c) c->last_error = msg;
    return st;
}

verkv_status cuda_fail(verkv_ctx *c, cudaError_t e, const char *where) {
    return fail(c, VERKV_ECUDA, std::string(where) + ": " + cudaGetErrorString(e));
}

#define VERKV_CUDA(call, where)                              \
    do {                                                     \
        cudaError_t e_ = (call);                             \
        if (e_ != cudaSuccess) return cuda_fail(ctx, e_, where); \
    } while (0)

cudaEvent_t prof_event(verkv_ctx *ctx) {
    if (ctx->prof_used == ctx->prof_pool.size()) {
        cudaEvent_t e = nullptr;
        if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
        ctx->prof_pool.push_back(e);
    }
    return ctx->prof_pool[ctx->prof_used++];
}

// Launch with accounting: counts the launch and, when profiling, brackets it with events.
template <typename F>
cudaError_t tracked(verkv_ctx *ctx, int kernel, cudaStream_t s, F &&launch) {
    cudaEvent_t a = nullptr, b = nullptr;
    if (ctx->prof_on && (a = prof_event(ctx)) != nullptr) cudaEventRecord(a, s);
    const cudaError_t e = launch();
    if (e != cudaSuccess) return e;
    ctx->launches[kernel]++;
    if (a && (b = prof_event(ctx)) != nullptr) {
        cudaEventRecord(b, s);
        ctx->prof_recs.push_back({kernel, a, b});
    }
    return cudaSuccess;
}

LayerIdx layer_idx(const verkv_ctx *ctx, int layer) {
    LayerIdx li;
    li.layers = ctx->sh.layers;
    li.layer = layer;
    li.kv_heads = ctx->sh.kv_heads;
    li.G = ctx->sh.q_per_kv;
    return li;
}

// Arguments of the pivotal partial sums of one layer call.
PartialArgs pivotal_args(const verkv_ctx *ctx, const verkv_pivotal &piv, const void *q,
                         const LayerIdx &li, bool sketch_exact) {
    const int d = ctx->sh.head_dim;
    PartialArgs pa{};
    pa.rows = (const uint16_t *)piv.kv;
    pa.ids = piv.ids;
    pa.pr = piv.r;
    pa.count = piv.count;
    pa.q = (const uint16_t *)q;
    pa.F = ctx->F;
    pa.qstats = ctx->qstats;
    pa.scores = ctx->scores;
    pa.part = ctx->part_piv;
    pa.err = ctx->err;
    pa.row_stride = ctx->sh.cap;
    pa.units_total = ctx->sh.batch * ctx->sh.layers * ctx->sh.kv_heads;
    pa.max_chunks = ctx->L.max_piv;
    pa.n = ctx->sh.n;
    pa.W = ctx->L.W;
    pa.d = d;
    pa.mode = ROWS_PIVOTAL;
    pa.keys = nullptr;
    pa.row16 = d / 4;
    pa.voff16 = d / 8;
    pa.scale = (float)(1.0 / sqrt((double)d));
    pa.li = li;
    pa.sketch_logits = sketch_exact ? 0 : 1;
    return pa;
}

// One host-to-device copy of the MEMCPY-mode fetch, on the side stream (or an injected failure).
cudaError_t copy_rows(verkv_ctx *ctx, void *dst, const void *src, size_t bytes) {
    if (ctx->inject_copy_fail > 0) {
        --ctx->inject_copy_fail;
        return cudaErrorInvalidValue;
    }
    return cudaMemcpyAsync(dst, src, bytes, cudaMemcpyHostToDevice, ctx->side);
}

// ---------------------------------------------------------------------------------------------
// Heads and the paged cache.

// Puts the caller's current device back when the call returns, on every path.
class DeviceRestore {
  public:
    DeviceRestore() { ok_ = cudaGetDevice(&saved_) == cudaSuccess; }
    ~DeviceRestore() {
        if (ok_) cudaSetDevice(saved_);
    }
    DeviceRestore(const DeviceRestore &) = delete;
    DeviceRestore &operator=(const DeviceRestore &) = delete;

  private:
    int saved_ = 0;
    bool ok_ = false;
};

// Rows read or written in 16-byte vectors.
bool bad_rows(const verkv_rows *r) {
    return !r->data || bad16(r->data) || r->token_stride < 0 || r->head_stride < 0 || (r->token_stride & 7) ||
           (r->head_stride & 7);
}
// An output of `tokens` x `heads` rows of d elements: no two rows may share an element.
bool overlapping(const verkv_rows *r, int64_t tokens, int64_t heads, int64_t d) {
    if (tokens <= 1 && heads <= 1) return false;
    if (tokens <= 1) return r->head_stride < d;
    if (heads <= 1) return r->token_stride < d;
    const bool token_major = r->token_stride >= r->head_stride;
    const int64_t inner = token_major ? r->head_stride : r->token_stride;
    const int64_t outer = token_major ? r->token_stride : r->head_stride;
    const int64_t count = token_major ? heads : tokens;
    // nested strides, or (a head's rows inside another's stride) interleaved ones such as the key
    // half of [n][2][d]
    return inner < d || outer < (count - 1) * inner + d;
}
bool valid_dtype(int32_t t) { return t == VERKV_BF16 || t == VERKV_F16; }
bool packed(const verkv_pages *p) { return p->dtype == VERKV_BF16_Q4 || p->dtype == VERKV_F16_Q4; }
// The type of the rows that go with pages.
int row_type(const verkv_pages *p) { return packed(p) ? p->dtype - VERKV_BF16_Q4 : p->dtype; }
bool valid_pages(const verkv_pages *p, const verkv_shape &sh) {
    const int t = p->page_tokens;
    return (valid_dtype(p->dtype) || packed(p)) && (t == 16 || t == 32 || t == 64 || t == 128 || t == 256) && p->num_pages >= 1 && p->kv &&
           !bad16(p->kv) && (int64_t)p->num_pages * sh.kv_heads * t < (1LL << 31);
}
// Tables and lengths of cached tokens in these pages.
bool bad_span(const verkv_span *s, const verkv_pages *pages) {
    return !s->table || !s->length || bad4(s->table) || bad4(s->length) || s->rows < 1 || s->stride < 1 || s->max_length < 0 ||
           s->max_length > (1 << 30) || (int64_t)s->max_length > (int64_t)s->stride * pages->page_tokens;
}
// Most holes that an eviction leaves in a sequence of one head: as many as are chosen, or as it loses.
int evict_room(int max_length, int keep) { return std::max(0, std::min(keep, max_length - keep)); }
int log2_of(int power_of_two) {
    int s = 0;
    while ((1 << s) < power_of_two) ++s;
    return s;
}
bool valid_rope(const verkv_rope *r, int d) {
    return r->rotary_dim >= 0 && r->rotary_dim <= d && r->rotary_dim % 16 == 0 &&
           (r->rotary_dim == 0 || (r->turns && !bad16(r->turns)));
}

// What norm_rotate and append have in common; nullptr, or what is wrong.
const char *heads_args(const verkv_ctx *ctx, HeadsArgs &a, int32_t dtype, int32_t tokens, const verkv_rows *q,
                       const verkv_rows *q_out, const verkv_rows *k, const verkv_head_norm *norm,
                       const verkv_rope *rope, const int32_t *positions) {
    const int d = ctx->sh.head_dim, hk = ctx->sh.kv_heads, hq = hk * ctx->sh.q_per_kv;
    if (!valid_dtype(dtype)) return "unknown type";
    if (tokens < 0) return "tokens must be >= 0";
    if ((q == nullptr) != (q_out == nullptr)) return "q and q_out come together";
    if (q) {
        if (bad_rows(q) || bad_rows(q_out)) return "rows need 16-byte alignment and strides >= 0 that are multiples of 8";
        if (overlapping(q_out, tokens, hq, d)) return "rows of q_out overlap";
        a.q = (const uint16_t *)q->data;
        a.q_ts = q->token_stride;
        a.q_hs = q->head_stride;
        a.q_out = (uint16_t *)q_out->data;
        a.qo_ts = q_out->token_stride;
        a.qo_hs = q_out->head_stride;
        a.hq = hq;
    }
    if (k) {
        if (bad_rows(k)) return "rows need 16-byte alignment and strides >= 0 that are multiples of 8";
        a.k = (const uint16_t *)k->data;
        a.k_ts = k->token_stride;
        a.k_hs = k->head_stride;
        a.hk = hk;
    }
    if (norm) {
        if (!(norm->eps >= 0.0f) || !isfinite(norm->eps)) return "eps must be finite and >= 0";
        if (bad16(norm->q_weight) || bad16(norm->k_weight)) return "norm weights need 16-byte alignment";
        a.wq = (const uint16_t *)norm->q_weight;
        a.wk = (const uint16_t *)norm->k_weight;
        a.eps = norm->eps;
    }
    if (rope) {
        if (!valid_rope(rope, d)) return "rotary_dim must be a multiple of 16 up to head_dim, turns 16-byte aligned";
        a.rd = rope->rotary_dim;
        a.interleaved = rope->interleaved != 0;
        a.turns = rope->turns;
        if (a.rd > 0 && !positions) return "a rotation needs positions";
    }
    if (bad4(positions)) return "positions need 4-byte alignment";
    a.positions = positions;
    a.tokens = tokens;
    a.err = ctx->err;
    return nullptr;
}

constexpr int PAGED_MAX_SEGMENTS = 65536;  // sequences or prefixes of a call

// Rows of a segment, on average and rounded up.
int64_t paged_rows(int64_t q_tokens, int64_t segments, int G) { return (q_tokens + segments - 1) / segments * G; }

// Which kernel a level goes through, by the rows of its segments.  Prefixes of up to 16 rows and own
// tokens of up to 32: k_paged; more: k_paged_wide.  (8 sequences behind 32K tokens, 32 rows:
// k_paged 55 us, k_paged_wide beside it 44; own tokens of 32 sequences of 18 rows, up to 4096 each:
// k_paged 65, k_paged_wide, whose 128 rows are then mostly empty, 84.)
bool paged_wide_prefix(int64_t rows) { return rows > PAGED_ROWS / 2; }
bool paged_wide_own(int64_t rows) { return rows > PAGED_ROWS; }

// Upper bound of the partial rows of one level of `segs` segments, for one head and without the slot a CTA:
// its queries' rows q G, and a ragged row tile a segment.  Tiles have up to 32 rows, or 128 where segments
// have more than 16 rows on average (there are fewer than q G / 16 then), or 256 where more than 128.
int64_t paged_level_rows(int64_t G, int64_t segs, int64_t q_tokens) {
    const int64_t rows = q_tokens * G;
    return rows + std::max(PAGED_ROWS * segs, std::max(std::min(128 * segs, 8 * rows), std::min(256 * segs, 2 * rows)));
}
// Of any call for up to these sizes: both levels, or without prefixes only the sequences' own, and the slots
// of its launches' CTAs.
int64_t paged_rows_bound(int64_t hkv, int64_t G, int64_t seqs, int64_t groups, int64_t q_tokens) {
    // (of k_paged, or over 4-bit pages of a launch of each level: tiles of 32 rows there are only with more than 16 rows, where
    // there is room for k_paged_wide's; of fewer rows, paged_q4_share keeps within k_paged's)
    const int64_t rows = q_tokens * G, few = PAGED_MAX_CTAS * PAGED_ROWS;
    static_assert(PAGED_Q4_CTAS_32 * 32 <= PAGED_MAX_CTAS * PAGED_ROWS && PAGED_Q4_CTAS_16 * 16 <= PAGED_MAX_CTAS * PAGED_ROWS &&
                      PAGED_Q4_CTAS * 8 * 2 <= PAGED_MAX_CTAS * PAGED_ROWS && PAGED_Q4_CTAS_32 * 32 <= PAGED_WIDE_CTAS * 128,
                  "slots of k_paged_q4");
    const int64_t wide = (int64_t)PAGED_WIDE_CTAS * (rows > 128 ? 256 : rows > PAGED_ROWS / 2 ? 128 : 0);
    if (groups == 0) return hkv * paged_level_rows(G, seqs, q_tokens) + std::max(few, wide);
    return hkv * (paged_level_rows(G, seqs, q_tokens) + paged_level_rows(G, groups, q_tokens)) + few + wide;
}
bool paged_sizes_ok(int64_t seqs, int64_t groups, int64_t q_tokens, const verkv_shape &sh) {
    return seqs >= 0 && groups >= 0 && q_tokens >= 0 && seqs <= PAGED_MAX_SEGMENTS && groups <= PAGED_MAX_SEGMENTS &&
           q_tokens * sh.kv_heads * sh.q_per_kv < (1LL << 31);
}
size_t paged_workspace(const verkv_shape &sh, int64_t seqs, int64_t groups, int64_t q_tokens) {
    const size_t rec = align256((size_t)(1 + seqs + groups) * 8) * PAGED_LINES;
    const size_t rows = (size_t)paged_rows_bound(sh.kv_heads, sh.q_per_kv, seqs, groups, q_tokens);
    return 256 + rec + rows * (size_t)(sh.head_dim + 2) * 4 + PAGED_LINES * 512;
}

// Fills in a line over the given segments but its buffers; false if its work cannot be counted in 31 bits.
bool paged_count(const PagedArgs &a, PagedLine &l, int rows_tile, int ctas_max) {
    const int64_t hkv = a.hkv;
    l.tt_shift = log2_of(rows_tile) - a.g_shift;
    int64_t units = 0, steps = 0;
    for (int x = 0; x < 2; ++x) {
        if (!l.with[x]) continue;
        const PagedLevel &lv = a.level[x];
        const int64_t tiles = (a.q_tokens >> l.tt_shift) + lv.rows;
        const int64_t each = (lv.max_length + (1 << l.tile_shift) - 1) >> l.tile_shift;
        units += tiles * hkv;
        steps += tiles * hkv * each;
        // What paged_share goes by: prefixes are taken to be of the bound's length, own tokens of half.
        const int64_t each_row = (a.q_tokens + lv.rows - 1) / lv.rows;
        const double likely = (double)hkv * lv.rows * ((each_row + (1 << l.tt_shift) - 1) >> l.tt_shift);
        const double long_each = x == 0 ? (double)each : 0.5 * (each + 1);
        l.units += likely;
        l.steps += likely * long_each;
        l.cost += likely * (l.grouped ? long_each * (l.tall ? 2.0 : 1.5) : (rows_tile > 16 ? 1.8 : 1.0) * (0.4 * long_each + 0.7));
    }
    l.ctas = (int)std::max<int64_t>(1, std::min<int64_t>(steps, ctas_max));
    // (a run's end is its start plus a run's length, which the last run may pass by a step a CTA)
    if (steps >= (1LL << 31) - 2 * std::max(PAGED_MAX_CTAS, ctas_max) || units + l.ctas >= (1LL << 31)) return false;
    l.slots = (int)units;  // (and one a CTA)
    return true;
}
// Takes its buffers from the workspace at `off`.
void paged_take(const verkv_ctx *ctx, const PagedArgs &a, PagedLine &l, unsigned char *ws, size_t &off) {
    const int rows_tile = 1 << (l.tt_shift + a.g_shift);
    const int64_t segs = (l.with[0] ? a.level[0].rows : 0) + (l.with[1] ? a.level[1].rows : 0);
    l.slots += l.ctas;
    auto take = [&](size_t bytes) {
        unsigned char *p = ws + off;
        off = align256(off + bytes);
        return p;
    };
    l.rec = (int2 *)take((size_t)(1 + segs) * 8);
    l.part_ml = (float *)take((size_t)l.slots * rows_tile * 2 * 4);
    l.part_o = (float *)take((size_t)l.slots * rows_tile * ctx->sh.head_dim * 4);
}
bool paged_line(const verkv_ctx *ctx, const PagedArgs &a, PagedLine &l, int rows_tile, int ctas_max, unsigned char *ws,
                size_t &off) {
    if (!paged_count(a, l, rows_tile, ctas_max)) return false;
    paged_take(ctx, a, l, ws, off);
    return true;
}

// The SMs of a call that launches both kernels.  Their CTAs do not fit on one SM together, and one
// after the other each leaves the GPU idle while it starts and ends, and the one bound by bytes the
// tensor cores of the other.  So k_paged gets SMs of its own beside the others, in proportion to the
// work (8 sequences behind 32K tokens: 46 us one after the other, 44 side by side; 256: 159, 148; 128
// with up to 1000 tokens of their own: 120, 98), unless it would take most of them.  Costs are the us
// of a step on an SM: 0.4 of k_paged, two CTAs an SM, and 0.7 a unit, with 32 rows 1.8 times that; 1.5
// or 2 of k_paged_wide with 128 or 256 rows.  (Measured at d 128; of k_paged 0.45 and 0.5 a step, or 2 times
// with 32 rows, change nothing by more than the spread between runs.)
bool paged_share(PagedLine &wide, PagedLine &own, int sms) {
    const double w = wide.cost, o = own.cost;
    int x = (int)(sms * o / (w + o)) + 1;
    if (x > sms * 3 / 4) return false;
    // Whole runs for each unit of k_paged_wide, where that takes little from either.
    const int n = sms - x, units = (int)std::min<double>(wide.units, sms);
    const int less = n / units * units, more = less + units;
    if (more - n <= x / 5) x = sms - more;
    else if (n - less <= n / 8) x = sms - less;
    own.ctas = std::min(own.ctas, 2 * x);
    wide.ctas = std::min(wide.ctas, sms - x);
    return true;
}

// The same of a call over 4-bit pages, both of whose launches are of k_paged_q4: in proportion to the us of an SM.
// (On one line with a prefix's long units, short own ones gave the CTAs that had them twice the others' time:
// 8 sequences of up to 512 tokens behind 32K 87 us.)  A step is 1.7 us of a CTA, three of which fit on an SM of either
// kind, or with 32 rows 1.9 of one of two, and a unit, which begins and ends alone, 8.  (With 3, 5, 8, 12 a unit: 32
// sequences of up to 16 tokens behind 32K 138, 120, 116, 108 us, 8 behind 2048 21.1, 20.3, 20.7, 25.3.)  Where own
// tokens are most of the work, all SMs take both; of a call of 9 to 16 rows the prefix's tiles of 16 are one an SM then, for
// which the workspace has room.
void paged_q4_share(PagedLine &prefix, PagedLine &own, int sms, int64_t rows) {
    for (PagedLine *l : {&prefix, &own}) {
        l->per_sm = std::min(l->per_sm, 3);
        l->cost = (l->steps * (l->per_sm == 2 ? 1.9 : 1.7) + l->units * 8.0) / l->per_sm;
    }
    const int x = (int)(sms * own.cost / (own.cost + prefix.cost)) + 1;
    if (x > sms * 3 / 4) {
        if (rows > 8 && rows <= 16) prefix.ctas = std::min(prefix.ctas, PAGED_MAX_CTAS * PAGED_ROWS / 16 - PAGED_Q4_CTAS_16);
        return;
    }
    own.ctas = std::min(own.ctas, own.per_sm * x);
    prefix.ctas = std::min(prefix.ctas, prefix.per_sm * (sms - x));
}

}  // namespace

extern "C" {

const char *verkv_status_string(int st) {
    switch (st) {
        case VERKV_OK: return "VERKV_OK";
        case VERKV_EINVAL: return "VERKV_EINVAL";
        case VERKV_EBUDGET: return "VERKV_EBUDGET";
        case VERKV_ECAPACITY: return "VERKV_ECAPACITY";
        case VERKV_ENOCONVERGE: return "VERKV_ENOCONVERGE";
        case VERKV_ECUDA: return "VERKV_ECUDA";
        case VERKV_ECOPY: return "VERKV_ECOPY";
        case VERKV_ETIMEOUT: return "VERKV_ETIMEOUT";
        case VERKV_ESTATE: return "VERKV_ESTATE";
        case VERKV_ETOOLARGE: return "VERKV_ETOOLARGE";
        default: return "VERKV_UNKNOWN";
    }
}

size_t verkv_sketch_bytes(const verkv_shape *shape, int32_t format) {
    if (!valid_shape(shape)) return 0;
    const size_t rows = (size_t)shape->batch * shape->layers * shape->kv_heads * shape->n;
    if (format == VERKV_SKETCH_EXACT) return rows * 2 * shape->head_dim;
    if (format == VERKV_SKETCH_Q2) return rows * q2_row_bytes(shape->head_dim);
    return 0;
}

size_t verkv_workspace_size(const verkv_shape *shape) {
    Layout L;
    return make_layout(shape, L) ? L.total : 0;
}

verkv_status verkv_create(verkv_ctx **out, int device, void *stream, const verkv_shape *shape,
                          void *workspace, size_t workspace_bytes) {
    if (!out) return VERKV_EINVAL;
    *out = nullptr;
    Layout L;
    if (!make_layout(shape, L)) return VERKV_EINVAL;
    if (!workspace || workspace_bytes < L.total || ((uintptr_t)workspace & 255u)) return VERKV_EINVAL;
    verkv_ctx *ctx = new verkv_ctx();
    ctx->device = device;
    ctx->sh = *shape;
    ctx->L = L;
    ctx->main = (cudaStream_t)stream;
    ctx->ws = (unsigned char *)workspace;
    cudaError_t e = cudaSetDevice(device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&ctx->sms, cudaDevAttrMultiProcessorCount, device);
    if (e == cudaSuccess) e = cudaStreamCreateWithFlags(&ctx->side, cudaStreamNonBlocking);
    if (e == cudaSuccess) e = cudaEventCreateWithFlags(&ctx->e_sel, cudaEventDisableTiming);
    if (e == cudaSuccess) e = cudaEventCreateWithFlags(&ctx->e_fetch, cudaEventDisableTiming);
    if (e != cudaSuccess) {
        verkv_destroy(ctx);
        return VERKV_ECUDA;
    }
    unsigned char *w = ctx->ws;
    ctx->err = (uint32_t *)(w + L.err);
    ctx->scores = (float *)(w + L.scores);
    ctx->qstats = (verkv_head_stats *)(w + L.qstats);
    ctx->F = (uint32_t *)(w + L.F);
    ctx->fids = (int32_t *)(w + L.fids);
    ctx->fcounts = (int32_t *)(w + L.fcounts);
    ctx->flc = (int32_t *)(w + L.flc);
    ctx->nacc = (int32_t *)(w + L.nacc);
    ctx->rmask = (uint32_t *)(w + L.rmask);
    ctx->rnext = (int32_t *)(w + L.rnext);
    ctx->slb = (uint32_t *)(w + L.slb);
    ctx->staging = (uint16_t *)(w + L.staging);
    ctx->part_piv = (float *)(w + L.part_piv);
    ctx->part_fet = (float *)(w + L.part_fet);
    e = cudaMemsetAsync(ctx->err, 0, 256, ctx->main);
    if (e == cudaSuccess) e = cudaMemsetAsync(ctx->fcounts, 0, (size_t)L.units_layer * 4, ctx->main);
    if (e == cudaSuccess) e = cudaMemsetAsync(ctx->flc, 0, (size_t)L.units_layer * 4, ctx->main);
    if (e == cudaSuccess) e = cudaMemsetAsync(ctx->nacc, 0, (size_t)L.qh_layer * 4, ctx->main);
    if (e == cudaSuccess) e = cudaMemsetAsync(ctx->rmask, 0, (size_t)L.units_layer * RMASK_W * 4, ctx->main);
    if (e == cudaSuccess) e = cudaMemsetAsync(ctx->rnext, 0, 4, ctx->main);
    if (e != cudaSuccess) {
        verkv_destroy(ctx);
        return VERKV_ECUDA;
    }
    *out = ctx;
    return VERKV_OK;
}

void verkv_destroy(verkv_ctx *ctx) {
    if (!ctx) return;
    // An object may go at any time, also while a graph is being captured (a collector decides): this thread's calls
    // here do not count against a capture then.  A stream that is capturing itself cannot be waited for, nor one that may
    // not be asked (the default stream beside a capture), though what was launched before may still run: of that,
    // only selections touch memory that goes here, and the last one's event can be waited for.
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaThreadExchangeStreamCaptureMode(&mode);
    cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
    const cudaError_t asked = cudaStreamIsCapturing(ctx->main, &capturing);
    if (asked != cudaSuccess) cudaGetLastError();
    if (asked == cudaSuccess && capturing == cudaStreamCaptureStatusNone) cudaStreamSynchronize(ctx->main);
    else if (ctx->e_sel) cudaEventSynchronize(ctx->e_sel);
    if (ctx->side) cudaStreamSynchronize(ctx->side);
    delete ctx->pool;
    if (ctx->host_staging) cudaFreeHost(ctx->host_staging);
    if (ctx->host_ids) cudaFreeHost(ctx->host_ids);
    if (ctx->host_counts) cudaFreeHost(ctx->host_counts);
    for (cudaEvent_t e : ctx->prof_pool) cudaEventDestroy(e);
    if (ctx->e_sel) cudaEventDestroy(ctx->e_sel);
    if (ctx->e_fetch) cudaEventDestroy(ctx->e_fetch);
    if (ctx->e_cap) cudaEventDestroy(ctx->e_cap);
    if (ctx->side) cudaStreamDestroy(ctx->side);
    cudaThreadExchangeStreamCaptureMode(&mode);
    delete ctx;
}

verkv_status verkv_set_sequence_offset(verkv_ctx *ctx, int32_t seq0) {
    if (!ctx) return VERKV_EINVAL;
    if (seq0 < 0) return fail(ctx, VERKV_EINVAL, "sequence offset: must be >= 0");
    ctx->seq0 = seq0;
    return VERKV_OK;
}

verkv_status verkv_set_fetch_mode(verkv_ctx *ctx, int mode_flags) {
    if (!ctx) return VERKV_EINVAL;
    const int mode = mode_flags & ~VERKV_FETCH_KEYS;
    if (mode != VERKV_FETCH_ZEROCOPY && mode != VERKV_FETCH_MEMCPY)
        return fail(ctx, VERKV_EINVAL, "unknown fetch mode");
    ctx->fetch_keys = (mode_flags & VERKV_FETCH_KEYS) != 0;
    if (mode == VERKV_FETCH_MEMCPY && !ctx->host_staging) {
        const size_t rows = (size_t)ctx->L.units_layer * ctx->sh.n;
        VERKV_CUDA(cudaSetDevice(ctx->device), "cudaSetDevice");
        if (!ctx->e_cap) VERKV_CUDA(cudaEventCreateWithFlags(&ctx->e_cap, cudaEventDisableTiming), "cudaEventCreate");
        VERKV_CUDA(cudaHostAlloc((void **)&ctx->host_staging,
                                 staging_bytes(ctx->L.units_layer, ctx->sh.n, ctx->sh.head_dim),
                                 cudaHostAllocDefault), "cudaHostAlloc(staging)");
        VERKV_CUDA(cudaHostAlloc((void **)&ctx->host_ids, rows * 4, cudaHostAllocMapped),
                   "cudaHostAlloc(ids)");
        VERKV_CUDA(cudaHostAlloc((void **)&ctx->host_counts, (size_t)ctx->L.units_layer * 4,
                                 cudaHostAllocMapped), "cudaHostAlloc(counts)");
        VERKV_CUDA(cudaHostGetDevicePointer((void **)&ctx->host_ids_dev, ctx->host_ids, 0),
                   "cudaHostGetDevicePointer(ids)");
        VERKV_CUDA(cudaHostGetDevicePointer((void **)&ctx->host_counts_dev, ctx->host_counts, 0),
                   "cudaHostGetDevicePointer(counts)");
        unsigned hw = std::thread::hardware_concurrency();
        ctx->pool = new Pool((int)std::max(1u, std::min(hw, 16u)));
    }
    ctx->fetch_mode = mode;
    return VERKV_OK;
}

verkv_status verkv_poissoncomp(verkv_ctx *ctx, const float *tau, double eta, verkv_hset H,
                               uint64_t seed, const void *kv_full, float *r_full,
                               const verkv_pivotal *out) {
    if (!ctx) return VERKV_EINVAL;
    if (!tau || !kv_full || !r_full || !out || !out->ids || !out->r || !out->kv || !out->count ||
        !out->resident || !out->c)
        return fail(ctx, VERKV_EINVAL, "poissoncomp: null pointer");
    if (!(eta > 0.0) || eta > 1.0 || H.n_sink < 0 || H.n_local < 0)
        return fail(ctx, VERKV_EINVAL, "poissoncomp: eta must be in (0, 1], H sizes >= 0");
    const int n = ctx->sh.n;
    const int64_t forced = std::min<int64_t>(n, (int64_t)H.n_sink + H.n_local);
    const int n_rest = (int)(n - forced);
    const double eta_n = eta * (double)n;
    const double b_rest = eta_n - (double)forced;
    if (n_rest > 0 && !(b_rest > 0.0))
        return fail(ctx, VERKV_EBUDGET, "poissoncomp: eta * n must exceed the forced H set");
    const NvtxRange nvtx("verkv_poissoncomp");
    if (bad16(kv_full) || bad16(out->kv) || bad4(tau) || bad4(r_full) || bad4(out->ids) ||
        bad4(out->r) || bad4(out->count) || bad4(out->resident) || bad4(out->c))
        return fail(ctx, VERKV_EINVAL, "poissoncomp: kv rows need 16-byte, other arrays 4-byte alignment");
    VERKV_CUDA(cudaSetDevice(ctx->device), "cudaSetDevice");
    const int units = ctx->sh.batch * ctx->sh.layers * ctx->sh.kv_heads;
    PcArgs a{};
    a.tau = tau;
    a.r_full = r_full;
    a.ids = out->ids;
    a.pr = out->r;
    a.count = out->count;
    a.resident = out->resident;
    a.c_out = out->c;
    a.err = ctx->err;
    a.b_rest = b_rest;
    a.eta_n = eta_n;
    a.n = n;
    a.W = ctx->L.W;
    a.cap = ctx->sh.cap;
    a.n_sink = H.n_sink;
    a.n_local = H.n_local;
    a.layers = ctx->sh.layers;
    a.kv_heads = ctx->sh.kv_heads;
    a.n_rest = n_rest;
    int cl = (n + 32767) / 32768;
    cl = std::max(1, std::min(cl, 8));
    int chunk = (n + cl - 1) / cl;
    chunk = (chunk + 1023) / 1024 * 1024;
    a.cl = cl;
    a.chunk = chunk;
    a.seed_lo = (uint32_t)seed;
    a.seed_hi = (uint32_t)(seed >> 32);
    a.seq0 = ctx->seq0;
    VERKV_CUDA(tracked(ctx, VERKV_K_PC_SOLVE, ctx->main, [&] { return launch_pc_solve(a, units, ctx->main); }), "k_pc_solve");
    VERKV_CUDA(tracked(ctx, VERKV_K_PC_GATHER, ctx->main, [&] {
                   return launch_pc_gather((const uint16_t *)kv_full, out->ids, out->count,
                                           (uint16_t *)out->kv, units, ctx->sh.cap, n,
                                           ctx->sh.head_dim, ctx->main);
               }), "k_pc_gather");
    return VERKV_OK;
}

verkv_status verkv_sketch_build(verkv_ctx *ctx, const void *kv_full, int32_t format,
                                void *sketch_out) {
    if (!ctx) return VERKV_EINVAL;
    if (!kv_full || !sketch_out) return fail(ctx, VERKV_EINVAL, "sketch_build: null pointer");
    if (format != VERKV_SKETCH_EXACT && format != VERKV_SKETCH_Q2)
        return fail(ctx, VERKV_EINVAL, "sketch_build: unknown format");
    if (bad16(kv_full) || bad16(sketch_out))
        return fail(ctx, VERKV_EINVAL, "sketch_build: kv_full and the sketch need 16-byte alignment");
    VERKV_CUDA(cudaSetDevice(ctx->device), "cudaSetDevice");
    const int64_t rows = (int64_t)ctx->sh.batch * ctx->sh.layers * ctx->sh.kv_heads * ctx->sh.n;
    if (format == VERKV_SKETCH_Q2) {
        VERKV_CUDA(tracked(ctx, VERKV_K_SKETCH, ctx->main, [&] {
                       return launch_sketch_q2((const uint16_t *)kv_full, (uint8_t *)sketch_out,
                                               rows, ctx->sh.head_dim, ctx->main);
                   }), "k_sketch_q2");
        return VERKV_OK;
    }
    VERKV_CUDA(tracked(ctx, VERKV_K_SKETCH, ctx->main, [&] {
                   return launch_sketch_exact((const uint16_t *)kv_full, (uint16_t *)sketch_out,
                                              rows, ctx->sh.head_dim, ctx->main);
               }), "k_sketch_exact");
    return VERKV_OK;
}

verkv_status verkv_attend_verified(verkv_ctx *ctx, int32_t layer, const void *q,
                                   const verkv_pivotal *pivotal, const float *r_full,
                                   const verkv_sketch *sketch, float eps, float delta,
                                   int32_t *fetch_ids_out, int32_t *fetch_counts_out) {
    if (!ctx) return VERKV_EINVAL;
    if (layer < 0 || layer >= ctx->sh.layers) return fail(ctx, VERKV_EINVAL, "attend: bad layer");
    if (!q || !pivotal || !r_full || !sketch || !sketch->data || !pivotal->ids || !pivotal->r ||
        !pivotal->kv || !pivotal->count || !pivotal->resident)
        return fail(ctx, VERKV_EINVAL, "attend: null pointer");
    if (sketch->format != VERKV_SKETCH_EXACT && sketch->format != VERKV_SKETCH_Q2)
        return fail(ctx, VERKV_EINVAL, "attend: unknown sketch format");
    if (!(eps > 0.0f) || !(delta > 0.0f) || !(delta < 1.0f) || !isfinite(eps))
        return fail(ctx, VERKV_EINVAL, "attend: need eps > 0 and 0 < delta < 1");
    if (bad16(q) || bad16(sketch->data) || bad16(pivotal->kv))
        return fail(ctx, VERKV_EINVAL, "attend: q, the sketch and the pivotal rows need 16-byte alignment");
    if (bad4(r_full) || bad4(pivotal->ids) || bad4(pivotal->r) || bad4(pivotal->count) ||
        bad4(pivotal->resident) || bad4(fetch_ids_out) || bad4(fetch_counts_out))
        return fail(ctx, VERKV_EINVAL, "attend: int32 / float arrays need 4-byte alignment");
    VERKV_CUDA(cudaSetDevice(ctx->device), "cudaSetDevice");
    const NvtxRange nvtx("verkv_attend_verified: score, certificate, selection");
    const LayerIdx li = layer_idx(ctx, layer);
    const int n = ctx->sh.n, d = ctx->sh.head_dim;

    ScoreArgs sa{};
    sa.sketch = (const uint16_t *)sketch->data;
    sa.q = (const uint16_t *)q;
    sa.scores = ctx->scores;
    sa.err = ctx->err;
    sa.n = n;
    sa.d = d;
    sa.scale = (float)(1.0 / sqrt((double)d));
    sa.li = li;
    if (ctx->score_stall_ns > 0) {  // injected: one stalled stage, a short wait limit
        sa.wait_ns = (unsigned long long)ctx->score_stall_ns;
        sa.stall_first = 1;
        ctx->score_stall_ns = 0;
    }
    if (sketch->format == VERKV_SKETCH_Q2) {
        VERKV_CUDA(tracked(ctx, VERKV_K_SCORE, ctx->main, [&] { return launch_score_q2(sa, ctx->L.units_layer, ctx->main, true); }), "k_score_q2");
    } else {
        VERKV_CUDA(tracked(ctx, VERKV_K_SCORE, ctx->main, [&] { return launch_score(sa, ctx->L.units_layer, ctx->main, true); }), "k_score");
    }

    if (ctx->shortlist > 0) {
        ShortlistArgs sla{};
        sla.scores = ctx->scores;
        sla.r_full = r_full;
        sla.out = ctx->slb;
        sla.n = n;
        sla.W = ctx->L.W;
        sla.size = ctx->shortlist;
        sla.li = li;
        VERKV_CUDA(tracked(ctx, VERKV_K_SHORTLIST, ctx->main, [&] { return launch_shortlist(sla, ctx->L.units_layer, ctx->main); }), "k_shortlist");
    }

    CertifyArgs ca{};
    ca.scores = ctx->scores;
    ca.shortlist = ctx->shortlist > 0 ? ctx->slb : nullptr;
    ctx->shortlisted = ctx->shortlist > 0;
    ca.r_full = r_full;
    ca.resident = pivotal->resident;
    ca.F = ctx->F;
    ca.qstats = ctx->qstats;
    ca.err = ctx->err;
    ca.n = n;
    ca.W = ctx->L.W;
    ca.cl = certify_cluster_size(n, ctx->L.qh_layer, ctx->sms);
    ca.chunk = certify_chunk(n, ca.cl);
    ca.eps = eps;
    ca.ldelta = (float)log(2.0 / (double)delta);
    ca.li = li;
    ca.beta_maxit = ctx->beta_maxit;
    ca.sel_gather = ctx->sel_gather;
    // The per-KV-head fetch list is built only for those who read it: the MEMCPY gather, or a
    // caller asking for ids or counts.  The zero-copy refine reads the selection bitmaps.
    const bool need_list = ctx->fetch_mode != VERKV_FETCH_ZEROCOPY || fetch_ids_out || fetch_counts_out;
    ca.fl_counter = need_list ? ctx->flc : nullptr;
    ca.rmask = ctx->rmask;
    ca.refine_next = ctx->rnext;
    ca.ids = ctx->fids;
    ca.counts = ctx->fcounts;
    ca.ids_user = fetch_ids_out;
    ca.counts_user = fetch_counts_out;
    if (ctx->fetch_mode == VERKV_FETCH_MEMCPY) {
        ca.ids_host = ctx->host_ids_dev;
        ca.counts_host = ctx->host_counts_dev;
    }
    VERKV_CUDA(tracked(ctx, VERKV_K_CERTIFY, ctx->main, [&] {
                   return launch_certify(ca, ctx->L.qh_layer, certify_smem_bytes(ca.chunk), ctx->main);
               }), "k_certify");
    // MEMCPY mode: verkv_fetch_refine waits on the host for the selection
    if (ctx->fetch_mode != VERKV_FETCH_ZEROCOPY) {
        cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
        VERKV_CUDA(cudaStreamIsCapturing(ctx->main, &capturing), "cudaStreamIsCapturing");
        ctx->selected = capturing == cudaStreamCaptureStatusNone ? ctx->e_sel : ctx->e_cap;
        VERKV_CUDA(cudaEventRecord(ctx->selected, ctx->main), "cudaEventRecord");
    }

    // The pivotal partial sums need only the selection: in MEMCPY mode they run here, during the
    // host gather; the zero-copy refine kernel of verkv_fetch_refine does them itself.
    if (ctx->fetch_mode != VERKV_FETCH_ZEROCOPY) {
        const PartialArgs pa = pivotal_args(ctx, *pivotal, q, li, sketch->format == VERKV_SKETCH_EXACT);
        int grid = std::min(ctx->L.units_layer * ctx->L.max_piv, ctx->sms * 8);
        VERKV_CUDA(tracked(ctx, VERKV_K_PARTIAL_PIVOTAL, ctx->main, [&] { return launch_partial(pa, ctx->L.units_layer, std::max(grid, 1), ctx->main); }), "k_partial");
    }

    ctx->pending = true;
    ctx->attended = true;
    ctx->layer = layer;
    ctx->piv = *pivotal;
    ctx->user_ids = fetch_ids_out;
    ctx->user_counts = fetch_counts_out;
    ctx->q = q;
    ctx->sketch = sketch->data;
    ctx->sketch_exact = sketch->format == VERKV_SKETCH_EXACT;
    return VERKV_OK;
}

verkv_status verkv_fetch_refine(verkv_ctx *ctx, const int32_t *ids, const int32_t *counts,
                                const void *host_kv, float *o_out, float *lse_out,
                                verkv_head_stats *stats_out) {
    if (!ctx) return VERKV_EINVAL;
    if (!ctx->pending) return fail(ctx, VERKV_ESTATE, "fetch_refine: no preceding attend_verified");
    if ((ids && ids != ctx->user_ids) || (counts && counts != ctx->user_counts))
        return fail(ctx, VERKV_EINVAL, "fetch_refine: ids/counts must be the attend outputs or NULL");
    if (!host_kv || !o_out) return fail(ctx, VERKV_EINVAL, "fetch_refine: null pointer");
    if (bad16(host_kv) || bad4(o_out) || bad4(lse_out) || bad4(stats_out))
        return fail(ctx, VERKV_EINVAL, "fetch_refine: host_kv needs 16-byte, outputs 4-byte alignment");
    VERKV_CUDA(cudaSetDevice(ctx->device), "cudaSetDevice");
    const NvtxRange nvtx("verkv_fetch_refine: fetch, refine, merge");
    const LayerIdx li = layer_idx(ctx, ctx->layer);
    const int n = ctx->sh.n, d = ctx->sh.head_dim;
    // With the exact sketch every key is already on the GPU: only V rows move, unless asked.
    // A 2-bit sketch holds no exact key, so fetched rows bring their K row too.
    const bool v_only = !ctx->fetch_keys && ctx->sketch_exact;
    const size_t row_bytes = (size_t)4 * d;                 // a K|V row of the host cache
    const size_t move_bytes = v_only ? (size_t)2 * d : row_bytes;
    const size_t move_off = v_only ? (size_t)2 * d : 0;     // V follows K inside a row

    PartialArgs pa{};
    pa.q = (const uint16_t *)ctx->q;
    pa.F = ctx->F;
    pa.qstats = ctx->qstats;
    pa.part = ctx->part_fet;
    pa.err = ctx->err;
    pa.rmask = ctx->rmask;
    pa.ids = ctx->fids;
    pa.pr = nullptr;
    pa.count = ctx->fcounts;
    pa.row_stride = n;
    pa.max_chunks = ctx->L.max_fet;
    pa.n = n;
    pa.W = ctx->L.W;
    pa.d = d;
    pa.scale = (float)(1.0 / sqrt((double)d));
    pa.li = li;
    pa.keys = v_only ? (const uint16_t *)ctx->sketch : nullptr;
    int grid = std::max(1, std::min(ctx->L.units_layer * ctx->L.max_fet, ctx->sms * 8));

    MergeArgs ma{};
    ma.part_piv = ctx->part_piv;
    ma.part_fet = ctx->part_fet;
    ma.rmask = ctx->rmask;
    ma.pcount = ctx->piv.count;
    ma.fcount = ctx->fcounts;
    ma.qstats = ctx->qstats;
    ma.o = o_out;
    ma.lse = lse_out;
    ma.stats = stats_out;
    ma.max_piv = ctx->L.max_piv;
    ma.max_fet = ctx->L.max_fet;
    ma.cap = ctx->sh.cap;
    ma.d = d;
    ma.li = li;

    if (ctx->fetch_mode == VERKV_FETCH_ZEROCOPY) {
        // One kernel on the context's stream for the pivotal partial sums and the fetched rows,
        // read straight from page-locked host memory; the merge follows.
        cudaPointerAttributes attr;
        cudaError_t e = cudaPointerGetAttributes(&attr, host_kv);
        if (e != cudaSuccess || attr.type != cudaMemoryTypeHost || !attr.devicePointer) {
            cudaGetLastError();
            return fail(ctx, VERKV_EINVAL, "fetch_refine: host_kv is not page-locked host memory");
        }
        pa.rows = (const uint16_t *)attr.devicePointer;
        pa.mode = ROWS_HOST;
        pa.row16 = d / 4;
        pa.voff16 = d / 8;
        pa.resident = ctx->piv.resident;
        pa.nacc = ctx->nacc;
        pa.refine_next = ctx->rnext;
        ma.nacc = ctx->nacc;
        const PartialArgs piv = pivotal_args(ctx, ctx->piv, ctx->q, li, ctx->sketch_exact);
        const int items = ctx->L.units_layer * (ctx->L.max_fet + ctx->L.max_piv);
        grid = std::max(1, std::min(items, ctx->sms * 8));
        VERKV_CUDA(tracked(ctx, VERKV_K_FETCH_HOST, ctx->main, [&] {
                       return launch_refine(piv, pa, ctx->L.units_layer, grid, ctx->main);
                   }), "k_refine");
    } else {
        VERKV_CUDA(cudaEventSynchronize(ctx->selected), "cudaEventSynchronize");
        // When profiling, two events on the (idle) side stream bracket the host gather.
        cudaEvent_t g0 = ctx->prof_on ? prof_event(ctx) : nullptr;
        if (g0) VERKV_CUDA(cudaEventRecord(g0, ctx->side), "cudaEventRecord");
        const int U = ctx->L.units_layer;
        const unsigned char *src_base = (const unsigned char *)host_kv;
        // Flatten (unit, row) into one index space and split it evenly over the pool.
        std::vector<int64_t> start(U + 1, 0);
        for (int ul = 0; ul < U; ++ul) start[ul + 1] = start[ul] + ctx->host_counts[ul];
        const int64_t total = start[U];
        const int P = ctx->pool->size();
        const size_t head = staging_header(U);
        int64_t *offs = reinterpret_cast<int64_t *>(ctx->host_staging);
        for (int ul = 0; ul < U; ++ul) offs[ul] = start[ul];
        unsigned char *rows_h = ctx->host_staging + head;
        nvtxRangePushA("fetch: host gather");
        ctx->pool->run([&](int w) {
            const int64_t lo = total * w / P, hi = total * (w + 1) / P;
            int ul = (int)(std::upper_bound(start.begin(), start.end(), lo) - start.begin()) - 1;
            for (int64_t x = lo; x < hi; ++x) {
                while (x >= start[ul + 1]) ++ul;
                const int64_t j = x - start[ul];
                const int ug = li.unit_global(ul);
                const int id = ctx->host_ids[(size_t)ul * n + j];
                memcpy(rows_h + (size_t)x * move_bytes,
                       src_base + ((size_t)ug * n + id) * row_bytes + move_off, move_bytes);
            }
        });
        nvtxRangePop();
        if (g0) {
            cudaEvent_t g1 = prof_event(ctx);
            if (g1) {
                VERKV_CUDA(cudaEventRecord(g1, ctx->side), "cudaEventRecord");
                ctx->prof_recs.push_back({VERKV_K_FETCH_GATHER, g0, g1});
            }
        }
        // One copy: the header and every unit's rows.
        const cudaError_t ce = tracked(ctx, VERKV_K_FETCH_COPY, ctx->side, [&]() -> cudaError_t {
            return copy_rows(ctx, ctx->staging, ctx->host_staging, head + (size_t)total * move_bytes);
        });
        if (ce != cudaSuccess)
            return fail(ctx, VERKV_ECOPY, std::string("fetch copy: ") + cudaGetErrorString(ce));
        VERKV_CUDA(cudaEventRecord(ctx->e_fetch, ctx->side), "cudaEventRecord");
        VERKV_CUDA(cudaStreamWaitEvent(ctx->main, ctx->e_fetch, 0), "cudaStreamWaitEvent");
        pa.staged_off = reinterpret_cast<const int64_t *>(ctx->staging);
        pa.rows = reinterpret_cast<const uint16_t *>(reinterpret_cast<const unsigned char *>(ctx->staging) + head);
        pa.mode = ROWS_STAGED;
        pa.row16 = (int)(move_bytes / 16);
        pa.voff16 = v_only ? 0 : d / 8;
        VERKV_CUDA(tracked(ctx, VERKV_K_PARTIAL_STAGED, ctx->main, [&] { return launch_partial(pa, ctx->L.units_layer, grid, ctx->main); }), "k_partial(staged)");
    }

    VERKV_CUDA(tracked(ctx, VERKV_K_MERGE, ctx->main, [&] { return launch_merge(ma, ctx->L.qh_layer, ctx->main); }), "k_merge");
    ctx->pending = false;
    return VERKV_OK;
}

verkv_status verkv_measure_sketch_stream(verkv_ctx *ctx, int32_t layer, const verkv_sketch *sketch) {
    if (!ctx) return VERKV_EINVAL;
    if (layer < 0 || layer >= ctx->sh.layers) return fail(ctx, VERKV_EINVAL, "sketch stream: bad layer");
    if (!sketch || !sketch->data || sketch->format != VERKV_SKETCH_EXACT)
        return fail(ctx, VERKV_EINVAL, "sketch stream: an exact sketch is required");
    if (bad16(sketch->data)) return fail(ctx, VERKV_EINVAL, "sketch stream: 16-byte alignment required");
    VERKV_CUDA(cudaSetDevice(ctx->device), "cudaSetDevice");
    ScoreArgs sa{};
    sa.sketch = (const uint16_t *)sketch->data;
    sa.err = ctx->err;
    sa.n = ctx->sh.n;
    sa.d = ctx->sh.head_dim;
    sa.li = layer_idx(ctx, layer);
    VERKV_CUDA(launch_sketch_stream(sa, ctx->L.units_layer, ctx->main), "k_sketch_stream");
    return VERKV_OK;
}

verkv_status verkv_sync(verkv_ctx *ctx) {
    if (!ctx) return VERKV_EINVAL;
    VERKV_CUDA(cudaSetDevice(ctx->device), "cudaSetDevice");
    VERKV_CUDA(cudaStreamSynchronize(ctx->side), "cudaStreamSynchronize(side)");
    VERKV_CUDA(cudaStreamSynchronize(ctx->main), "cudaStreamSynchronize(main)");
    uint32_t word = 0;
    VERKV_CUDA(cudaMemcpy(&word, ctx->err, sizeof(word), cudaMemcpyDeviceToHost), "read error word");
    if (word == 0) return VERKV_OK;
    VERKV_CUDA(cudaMemset(ctx->err, 0, sizeof(word)), "clear error word");
    if (word & ERR_TAU) return fail(ctx, VERKV_EINVAL, "tau outside (0, 1] or not finite");
    if (word & ERR_CAPACITY) return fail(ctx, VERKV_ECAPACITY, "pivotal set exceeded cap (truncated)");
    if (word & ERR_TIMEOUT) return fail(ctx, VERKV_ETIMEOUT, "a bounded wait on a copy barrier expired");
    if (word & ERR_BADID) return fail(ctx, VERKV_EINVAL, "a pivotal or fetch row id outside [0, n) (skipped)");
    if (word & ERR_PAGE)
        return fail(ctx, VERKV_EINVAL, "a page id, place, length or start outside its range (paged cache)");
    if (word & ERR_BUDGET_SUM) return fail(ctx, VERKV_ENOCONVERGE, "|sum r - eta n| >= 1e-6 n");
    return fail(ctx, VERKV_ENOCONVERGE, "a solve hit its iteration cap");
}

verkv_status verkv_set_shortlist(verkv_ctx *ctx, int32_t size) {
    if (!ctx) return VERKV_EINVAL;
    if (size < 0 || size > SHORTLIST_MAX)
        return fail(ctx, VERKV_EINVAL, "set_shortlist: size must be 0 (off) or 1 .. 256");
    ctx->shortlist = size;
    return VERKV_OK;
}

verkv_status verkv_shortlist_bitmap(verkv_ctx *ctx, uint32_t *out) {
    if (!ctx) return VERKV_EINVAL;
    if (!ctx->shortlisted) return fail(ctx, VERKV_ESTATE, "shortlist_bitmap: no attend with a shortlist");
    if (!out) return fail(ctx, VERKV_EINVAL, "shortlist_bitmap: null pointer");
    VERKV_CUDA(cudaSetDevice(ctx->device), "cudaSetDevice");
    VERKV_CUDA(cudaMemcpyAsync(out, ctx->slb, (size_t)ctx->L.units_layer * ctx->L.W * 4,
                               cudaMemcpyDefault, ctx->main), "copy shortlist");
    return VERKV_OK;
}

verkv_status verkv_attend_dense_host(verkv_ctx *ctx, int32_t layer, const void *q,
                                    const void *host_kv, float *o_out, float *lse_out) {
    if (!ctx) return VERKV_EINVAL;
    if (layer < 0 || layer >= ctx->sh.layers) return fail(ctx, VERKV_EINVAL, "dense: bad layer");
    if (!q || !host_kv || !o_out) return fail(ctx, VERKV_EINVAL, "dense: null pointer");
    if (bad16(q) || bad16(host_kv) || bad4(o_out) || bad4(lse_out))
        return fail(ctx, VERKV_EINVAL, "dense: q and host_kv need 16-byte, outputs 4-byte alignment");
    VERKV_CUDA(cudaSetDevice(ctx->device), "cudaSetDevice");
    cudaPointerAttributes attr;
    cudaError_t e = cudaPointerGetAttributes(&attr, host_kv);
    if (e != cudaSuccess || attr.type != cudaMemoryTypeHost || !attr.devicePointer) {
        cudaGetLastError();
        return fail(ctx, VERKV_EINVAL, "dense: host_kv is not page-locked host memory");
    }
    DenseArgs da{};
    da.rows = (const uint16_t *)attr.devicePointer;
    da.q = (const uint16_t *)q;
    da.part = ctx->part_fet;  // [units_layer][dense_chunks][G][d + 2]
    da.n = ctx->sh.n;
    da.chunks = ctx->L.dense_chunks;
    da.d = ctx->sh.head_dim;
    da.scale = (float)(1.0 / sqrt((double)da.d));
    da.li = layer_idx(ctx, layer);
    const int grid = std::max(1, std::min(ctx->L.units_layer * da.chunks, ctx->sms * 4));
    VERKV_CUDA(tracked(ctx, VERKV_K_DENSE_HOST, ctx->main, [&] {
                   return launch_dense_host(da, ctx->L.units_layer, grid, ctx->main);
               }), "k_dense_host");
    VERKV_CUDA(tracked(ctx, VERKV_K_DENSE_MERGE, ctx->main, [&] {
                   return launch_dense_merge(da, ctx->L.qh_layer, o_out, lse_out, ctx->main);
               }), "k_dense_merge");
    return VERKV_OK;
}

verkv_status verkv_selection_bitmap(verkv_ctx *ctx, uint32_t *out) {
    if (!ctx) return VERKV_EINVAL;
    if (!ctx->attended) return fail(ctx, VERKV_ESTATE, "selection_bitmap: no attend has run");
    if (!out) return fail(ctx, VERKV_EINVAL, "selection_bitmap: null pointer");
    VERKV_CUDA(cudaSetDevice(ctx->device), "cudaSetDevice");
    VERKV_CUDA(cudaMemcpyAsync(out, ctx->F, (size_t)ctx->L.qh_layer * ctx->L.W * 4,
                               cudaMemcpyDefault, ctx->main), "copy F");
    return VERKV_OK;
}

verkv_status verkv_rope_turns(const double *inv_freq, int32_t count, uint64_t *turns) {
    if (!inv_freq || !turns || count < 0) return VERKV_EINVAL;
    for (int32_t i = 0; i < count; ++i)
        if (!isfinite(inv_freq[i]) || fabs(inv_freq[i]) >= 4294967296.0) return VERKV_EINVAL;
    for (int32_t i = 0; i < count; ++i) {
        const double t = fabs(inv_freq[i]) / 6.283185307179586476925286766559;
        const uint64_t x = (uint64_t)ldexp(t - floor(t), 64);  // (the difference is exact)
        turns[i] = inv_freq[i] < 0.0 ? 0u - x : x;             // (of a small negative t it would not be)
    }
    return VERKV_OK;
}

verkv_status verkv_norm_rotate(verkv_ctx *ctx, int32_t dtype, int32_t tokens, const verkv_rows *q,
                               const verkv_rows *q_out, const verkv_rows *k,
                               const verkv_rows *k_out, const verkv_head_norm *norm,
                               const verkv_rope *rope, const int32_t *positions) try {
    if (!ctx) return VERKV_EINVAL;
    if (tokens == 0) return VERKV_OK;
    HeadsArgs a{};
    if (const char *why = heads_args(ctx, a, dtype, tokens, q, q_out, k, norm, rope, positions))
        return fail(ctx, VERKV_EINVAL, std::string("norm_rotate: ") + why);
    if ((k == nullptr) != (k_out == nullptr)) return fail(ctx, VERKV_EINVAL, "norm_rotate: k and k_out come together");
    if (!q && !k) return fail(ctx, VERKV_EINVAL, "norm_rotate: neither queries nor keys");
    if (k) {
        if (bad_rows(k_out)) return fail(ctx, VERKV_EINVAL, "norm_rotate: rows need 16-byte alignment and strides >= 0 that are multiples of 8");
        if (overlapping(k_out, tokens, ctx->sh.kv_heads, ctx->sh.head_dim)) return fail(ctx, VERKV_EINVAL, "norm_rotate: rows of k_out overlap");
        a.k_out = (uint16_t *)k_out->data;
        a.ko_ts = k_out->token_stride;
        a.ko_hs = k_out->head_stride;
    }
    const DeviceRestore restore;
    VERKV_CUDA(cudaSetDevice(ctx->device), "cudaSetDevice");
    const NvtxRange nvtx("verkv_norm_rotate");
    VERKV_CUDA(tracked(ctx, VERKV_K_HEADS, ctx->main, [&] { return launch_heads(a, dtype, ctx->sh.head_dim, ctx->main); }), "k_heads");
    return VERKV_OK;
} catch (...) {
    return VERKV_ECUDA;
}

verkv_status verkv_paged_append(verkv_ctx *ctx, const verkv_pages *pages, int32_t tokens,
                                const verkv_rows *k, const verkv_rows *v, const verkv_rows *q,
                                const verkv_rows *q_out, const verkv_head_norm *norm,
                                const verkv_rope *rope, const int32_t *positions,
                                const int32_t *seq, const int32_t *index, const verkv_span *span) try {
    if (!ctx) return VERKV_EINVAL;
    if (tokens == 0) return VERKV_OK;
    if (!pages || !k || !v || !seq || !index || !span || !span->table) return fail(ctx, VERKV_EINVAL, "paged_append: null pointer");
    if (!valid_pages(pages, ctx->sh)) return fail(ctx, VERKV_EINVAL, "paged_append: bad pool of pages");
    if (span->rows < 1 || span->stride < 1) return fail(ctx, VERKV_EINVAL, "paged_append: an empty table");
    HeadsArgs a{};
    if (const char *why = heads_args(ctx, a, row_type(pages), tokens, q, q_out, k, norm, rope, positions))
        return fail(ctx, VERKV_EINVAL, std::string("paged_append: ") + why);
    if (bad_rows(v)) return fail(ctx, VERKV_EINVAL, "paged_append: rows need 16-byte alignment and strides >= 0 that are multiples of 8");
    if (bad4(seq) || bad4(index) || bad4(span->table)) return fail(ctx, VERKV_EINVAL, "paged_append: int32 arrays need 4-byte alignment");
    a.v = (const uint16_t *)v->data;
    a.v_ts = v->token_stride;
    a.v_hs = v->head_stride;
    a.hv = ctx->sh.kv_heads;
    a.pages = (uint16_t *)pages->kv;
    a.packed = packed(pages);
    a.num_pages = pages->num_pages;
    a.page_shift = log2_of(pages->page_tokens);
    a.seq = seq;
    a.index = index;
    a.table = span->table;
    a.table_rows = span->rows;
    a.table_stride = span->stride;
    const DeviceRestore restore;
    VERKV_CUDA(cudaSetDevice(ctx->device), "cudaSetDevice");
    const NvtxRange nvtx("verkv_paged_append");
    VERKV_CUDA(tracked(ctx, VERKV_K_HEADS, ctx->main, [&] { return launch_heads(a, row_type(pages), ctx->sh.head_dim, ctx->main); }), "k_heads");
    return VERKV_OK;
} catch (...) {
    return VERKV_ECUDA;
}

verkv_status verkv_paged_weigh(verkv_ctx *ctx, const verkv_pages *pages, int32_t seqs, int32_t q_tokens,
                               const verkv_rows *q, const int32_t *q_start, const verkv_span *own, float scale,
                               const float *lse, const float *weights_in, float *weights_out, int32_t places) try {
    if (!ctx) return VERKV_EINVAL;
    const verkv_shape &sh = ctx->sh;
    if (seqs == 0 && q_tokens == 0) return VERKV_OK;
    if (!pages || !own || !weights_out || (q_tokens > 0 && (!q || !lse))) return fail(ctx, VERKV_EINVAL, "paged_weigh: null pointer");
    if (!valid_pages(pages, sh)) return fail(ctx, VERKV_EINVAL, "paged_weigh: bad pool of pages");
    if (!paged_sizes_ok(seqs, 0, q_tokens, sh)) return fail(ctx, VERKV_EINVAL, "paged_weigh: too many sequences or queries, or a negative count");
    if (seqs == 0) return fail(ctx, VERKV_EINVAL, "paged_weigh: queries of no sequence");
    if (!q_start && seqs != q_tokens) return fail(ctx, VERKV_EINVAL, "paged_weigh: without q_start there is one query a sequence");
    if (bad_span(own, pages) || own->rows != seqs) return fail(ctx, VERKV_EINVAL, "paged_weigh: bad table of the sequences' tokens");
    if (places < own->max_length || places > (1 << 30)) return fail(ctx, VERKV_EINVAL, "paged_weigh: places must be at least max_length, and at most 2^30");
    const float scale_log2 = (float)((scale == 0.0f ? 1.0 / sqrt((double)sh.head_dim) : (double)scale) * 1.4426950408889634);
    if (!isfinite(scale_log2)) return fail(ctx, VERKV_EINVAL, "paged_weigh: scale must be finite, also in units of log 2");
    if (q_tokens > 0 && bad_rows(q)) return fail(ctx, VERKV_EINVAL, "paged_weigh: rows need 16-byte alignment and strides >= 0 that are multiples of 8");
    if (bad4(lse) || bad4(weights_in) || bad4(weights_out) || bad4(q_start)) return fail(ctx, VERKV_EINVAL, "paged_weigh: arrays need 4-byte alignment");
    const DeviceRestore restore;
    VERKV_CUDA(cudaSetDevice(ctx->device), "cudaSetDevice");
    const NvtxRange nvtx("verkv_paged_weigh");
    WeighArgs a{};
    a.pages = pages->kv;
    a.table = own->table;
    a.length = own->length;
    a.q_start = q_start;
    a.stride = own->stride;
    a.max_length = own->max_length;
    a.seqs = seqs;
    a.q_tokens = q_tokens;
    a.hkv = sh.kv_heads;
    a.g_shift = log2_of(sh.q_per_kv);
    a.page_shift = log2_of(pages->page_tokens);
    a.num_pages = pages->num_pages;
    a.places = places;
    if (q) {
        a.q = (const uint16_t *)q->data;
        a.q_ts = q->token_stride;
        a.q_hs = q->head_stride;
    }
    a.scale_log2 = scale_log2;
    a.lse = lse;
    a.in = weights_in;
    a.out = weights_out;
    a.err = ctx->err;
    a.wait_ns = PAGED_WAIT_NS;
    if (ctx->weigh_stall_ns > 0) {  // injected: a short wait limit, stalled copies
        a.wait_ns = (unsigned long long)ctx->weigh_stall_ns;
        a.stall = 1;
        ctx->weigh_stall_ns = 0;
    }
    VERKV_CUDA(tracked(ctx, VERKV_K_WEIGH, ctx->main, [&] { return launch_weigh(a, row_type(pages), packed(pages), sh.head_dim, ctx->main); }), "k_weigh");
    return VERKV_OK;
} catch (...) {
    return VERKV_ECUDA;
}

size_t verkv_paged_evict_workspace_size(const verkv_shape *shape, int32_t seqs, int32_t max_length, int32_t keep) {
    if (!valid_shape(shape) || seqs < 0 || seqs > PAGED_MAX_SEGMENTS || max_length < 0 || max_length > (1 << 30) || keep < 1) return 0;
    return 256 + (size_t)seqs * shape->kv_heads * 2 * 4 * (size_t)evict_room(max_length, keep);
}

verkv_status verkv_paged_evict(verkv_ctx *ctx, const verkv_pages *pages, int32_t seqs, const verkv_span *own, int32_t keep,
                               int32_t first, int32_t last, const float *weights_in, float *weights_out, int32_t places,
                               int32_t *kept, void *workspace, size_t workspace_bytes) try {
    if (!ctx) return VERKV_EINVAL;
    const verkv_shape &sh = ctx->sh;
    if (seqs == 0) return VERKV_OK;
    if (!pages || !own || !weights_in || !weights_out || !workspace) return fail(ctx, VERKV_EINVAL, "paged_evict: null pointer");
    if (!valid_pages(pages, sh)) return fail(ctx, VERKV_EINVAL, "paged_evict: bad pool of pages");
    if (seqs < 0 || seqs > PAGED_MAX_SEGMENTS) return fail(ctx, VERKV_EINVAL, "paged_evict: too many sequences, or a negative count");
    if (bad_span(own, pages) || own->rows != seqs) return fail(ctx, VERKV_EINVAL, "paged_evict: bad table of the sequences' tokens");
    if (keep < 1 || first < 0 || last < 0 || (int64_t)first + last > keep) return fail(ctx, VERKV_EINVAL, "paged_evict: keep must be positive and hold the first and the last");
    if (places < own->max_length || places > (1 << 30)) return fail(ctx, VERKV_EINVAL, "paged_evict: places must be at least max_length, and at most 2^30");
    if (bad4(weights_in) || bad4(weights_out) || bad4(kept)) return fail(ctx, VERKV_EINVAL, "paged_evict: arrays need 4-byte alignment");
    if (((uintptr_t)workspace & 255u) || workspace_bytes < verkv_paged_evict_workspace_size(&sh, seqs, own->max_length, keep))
        return fail(ctx, VERKV_EINVAL, "paged_evict: workspace too small or not 256-byte aligned");
    const DeviceRestore restore;
    VERKV_CUDA(cudaSetDevice(ctx->device), "cudaSetDevice");
    const NvtxRange nvtx("verkv_paged_evict");
    EvictArgs a{};
    a.pages = pages->kv;
    a.table = own->table;
    a.length = own->length;
    a.stride = own->stride;
    a.max_length = own->max_length;
    a.seqs = seqs;
    a.hkv = sh.kv_heads;
    a.page_shift = log2_of(pages->page_tokens);
    a.num_pages = pages->num_pages;
    a.keep = keep;
    a.first = first;
    a.last = last;
    a.places = places;
    a.in = weights_in;
    a.out = weights_out;
    a.kept = kept;
    a.lists = (int32_t *)workspace;
    a.room = evict_room(own->max_length, keep);
    a.err = ctx->err;
    VERKV_CUDA(tracked(ctx, VERKV_K_EVICT, ctx->main, [&] { return launch_evict(a, packed(pages), sh.head_dim, ctx->main); }), "k_evict");
    return VERKV_OK;
} catch (...) {
    return VERKV_ECUDA;
}

verkv_status verkv_paged_values(verkv_ctx *ctx, const verkv_pages *pages, void *out) try {
    if (!ctx) return VERKV_EINVAL;
    if (!pages || !out) return fail(ctx, VERKV_EINVAL, "paged_values: null pointer");
    if (!valid_pages(pages, ctx->sh) || !packed(pages)) return fail(ctx, VERKV_EINVAL, "paged_values: a pool of 4-bit pages is required");
    if (bad16(out)) return fail(ctx, VERKV_EINVAL, "paged_values: out needs 16-byte alignment");
    const DeviceRestore restore;
    VERKV_CUDA(cudaSetDevice(ctx->device), "cudaSetDevice");
    const NvtxRange nvtx("verkv_paged_values");
    const long long rows = (long long)pages->num_pages * ctx->sh.kv_heads * pages->page_tokens;
    VERKV_CUDA(tracked(ctx, VERKV_K_PACKED_VALUES, ctx->main, [&] { return launch_q4_values(pages->kv, out, row_type(pages), rows, ctx->sh.head_dim, ctx->main); }), "k_q4_values");
    return VERKV_OK;
} catch (...) {
    return VERKV_ECUDA;
}

size_t verkv_paged_workspace_size(const verkv_shape *shape, int32_t seqs, int32_t groups, int32_t q_tokens) {
    if (!valid_shape(shape) || !paged_sizes_ok(seqs, groups, q_tokens, *shape)) return 0;
    return paged_workspace(*shape, seqs, groups, q_tokens);
}

verkv_status verkv_paged_attend(verkv_ctx *ctx, const verkv_pages *pages, int32_t seqs,
                                int32_t q_tokens, const verkv_rows *q, const int32_t *q_start,
                                const verkv_span *own, const verkv_span *prefix,
                                const int32_t *group_start, float scale, const float *prior_o,
                                const float *prior_lse, void *o_out, float *lse_out,
                                void *workspace, size_t workspace_bytes) try {
    if (!ctx) return VERKV_EINVAL;
    const verkv_shape &sh = ctx->sh;
    if (q_tokens == 0 && seqs >= 0) return VERKV_OK;
    if (!pages || !q || !o_out || !workspace) return fail(ctx, VERKV_EINVAL, "paged_attend: null pointer");
    if (!valid_pages(pages, sh)) return fail(ctx, VERKV_EINVAL, "paged_attend: bad pool of pages");
    const int groups = prefix ? prefix->rows : 0;
    if (!paged_sizes_ok(seqs, groups, q_tokens, sh)) return fail(ctx, VERKV_EINVAL, "paged_attend: too many sequences or queries, or a negative count");
    if (!q_start && seqs != q_tokens) return fail(ctx, VERKV_EINVAL, "paged_attend: without q_start there is one query a sequence");
    if (seqs == 0 && q_tokens != 0) return fail(ctx, VERKV_EINVAL, "paged_attend: queries of no sequence");
    if (seqs > 0 && own && (bad_span(own, pages) || own->rows != seqs)) return fail(ctx, VERKV_EINVAL, "paged_attend: bad table of the sequences' own tokens");
    if (prefix && bad_span(prefix, pages)) return fail(ctx, VERKV_EINVAL, "paged_attend: bad table of the shared prefixes");
    if (prefix && !group_start && groups != 1) return fail(ctx, VERKV_EINVAL, "paged_attend: several prefixes need group_start");
    if (group_start && !prefix) return fail(ctx, VERKV_EINVAL, "paged_attend: group_start without prefixes");
    const float scale_log2 = (float)((scale == 0.0f ? 1.0 / sqrt((double)sh.head_dim) : (double)scale) * 1.4426950408889634);
    if (!isfinite(scale_log2)) return fail(ctx, VERKV_EINVAL, "paged_attend: scale must be finite, also in units of log 2");
    if ((prior_o == nullptr) != (prior_lse == nullptr)) return fail(ctx, VERKV_EINVAL, "paged_attend: prior_o and prior_lse come together");
    if (bad_rows(q)) return fail(ctx, VERKV_EINVAL, "paged_attend: rows need 16-byte alignment and strides >= 0 that are multiples of 8");
    if (bad16(prior_o) || bad16(o_out) || bad4(prior_lse) || bad4(lse_out) || bad4(q_start) || bad4(group_start))
        return fail(ctx, VERKV_EINVAL, "paged_attend: prior_o and o_out need 16-byte, other arrays 4-byte alignment");
    if (((uintptr_t)workspace & 255u) || workspace_bytes < paged_workspace(sh, seqs, groups, q_tokens))
        return fail(ctx, VERKV_EINVAL, "paged_attend: workspace too small or not 256-byte aligned");
    const DeviceRestore restore;
    VERKV_CUDA(cudaSetDevice(ctx->device), "cudaSetDevice");
    const NvtxRange nvtx("verkv_paged_attend");

    PagedArgs a{};
    const int type = row_type(pages);
    a.pages = pages->kv;
    a.q = (const uint16_t *)q->data;
    a.q_ts = q->token_stride;
    a.q_hs = q->head_stride;
    a.q_start = q_start;
    a.group_start = group_start;
    auto level = [](const verkv_span *s) {
        PagedLevel l{};
        if (s) l = {s->table, s->length, s->rows, s->stride, s->max_length};
        return l;
    };
    a.level[0] = level(prefix && prefix->max_length > 0 ? prefix : nullptr);
    a.level[1] = level(own && own->max_length > 0 ? own : nullptr);
    // What the segments of the levels do not look at, the merge does.
    const verkv_span *const spans[2] = {prefix, own};
    for (int x = 0; x < 2; ++x) {
        if (!spans[x] || spans[x]->max_length > 0) continue;
        a.zero_length[x] = spans[x]->length;
        a.zero_rows[x] = spans[x]->rows;
    }
    a.check_q_start = q_start && !a.level[1].rows;
    a.check_group_start = group_start && !a.level[0].rows;
    a.unseen = a.check_q_start || a.check_group_start || a.zero_rows[0] || a.zero_rows[1];
    a.seqs = seqs;
    a.q_tokens = q_tokens;
    a.hkv = sh.kv_heads;
    a.g_shift = log2_of(sh.q_per_kv);
    a.page_shift = log2_of(pages->page_tokens);
    a.num_pages = pages->num_pages;
    a.scale_log2 = scale_log2;
    a.err = ctx->err;
    a.prior_o = prior_o;
    a.prior_lse = prior_lse;
    a.o = (uint16_t *)o_out;
    a.lse = lse_out;
    a.wait_ns = PAGED_WAIT_NS;
    if (ctx->paged_wait_ns > 0) {  // injected: a short wait limit, stalled copies
        a.wait_ns = (unsigned long long)ctx->paged_wait_ns;
        a.stall = ctx->paged_stall;
        ctx->paged_wait_ns = 0;
        ctx->paged_stall = false;
    }

    PagedLines both{};
    PagedLine *lines = both.l;
    size_t off = 256;  // (the first word: PagedArgs::ready)
    if (packed(pages) && (a.level[0].rows || a.level[1].rows)) {
        // A launch of each level, side by side.  Units of 8 rows, or of 16 or 32 where segments have more: K and V's codes are
        // then spread out less often, which long work gains by: 4 sequences of 8192 tokens by their last 64 queries
        // take 164 us with units of 32 for 184 with 16, by 512 1176 for 1360, 8 sequences behind 131072 tokens 116 for 123.  Short
        // work loses by longer units: 8 sequences behind 2048 tokens 21 for 18, 32 with 512 tokens of their own behind 32K
        // 165 for 145, 8 there 47 for 49.  At d = 64 there is half as much to spread out: two prefixes of 8191 with
        // 17 sequences each take 60 us with 32 for 54, 32 sequences behind 32K 61 for 69.
        for (int x = 0; x < 2; ++x) {
            PagedLine &l = lines[x];
            if (!a.level[x].rows) continue;
            l.with[x] = 1;
            l.tile_shift = log2_of(PAGED_TILE);
            const int64_t rows = paged_rows(q_tokens, a.level[x].rows, sh.q_per_kv);
            const int tile = rows <= 8 ? 8 : rows <= 16 || sh.head_dim == 64 ? 16 : 32;
            l.per_sm = tile == 8 ? 4 : tile == 16 ? 3 : 2;
            const int most = tile == 8 ? PAGED_Q4_CTAS : tile == 16 ? PAGED_Q4_CTAS_16 : PAGED_Q4_CTAS_32;
            if (!paged_count(a, l, tile, std::min(ctx->sms * l.per_sm, most)))
                return fail(ctx, VERKV_EINVAL, "paged_attend: more than 2^31 steps of work in one call");
        }
        const bool both_levels = lines[0].ctas && lines[1].ctas;
        if (both_levels) paged_q4_share(lines[0], lines[1], ctx->sms, (int64_t)q_tokens * sh.q_per_kv);
        for (int x = 0; x < 2; ++x)
            if (lines[x].ctas) paged_take(ctx, a, lines[x], (unsigned char *)workspace, off);
        if (off > workspace_bytes) return fail(ctx, VERKV_EINVAL, "paged_attend: workspace too small");
        // (launches that are timed one by one wait for one another)
        if (both_levels && !ctx->prof_on) a.ready = (unsigned long long *)workspace;
        const int first = both_levels && lines[1].cost > lines[0].cost ? 1 : 0;  // the longer one
        for (int turn = 0; turn < 2; ++turn) {
            const PagedLine &l = lines[first ^ turn];
            if (!l.ctas) continue;
            VERKV_CUDA(tracked(ctx, VERKV_K_PAGED_PACKED, ctx->main, [&] { return launch_paged_q4(a, l, turn == 1 && a.ready, type, sh.head_dim, ctx->main); }), "k_paged_q4");
        }
    } else if (a.level[0].rows || a.level[1].rows) {
        // Each level by the rows of its segments; the two lines' launches need not wait for one another.
        const int64_t rows_prefix = a.level[0].rows ? paged_rows(q_tokens, a.level[0].rows, sh.q_per_kv) : 0;
        const int64_t rows_own = a.level[1].rows ? paged_rows(q_tokens, a.level[1].rows, sh.q_per_kv) : 0;
        lines[1].with[0] = paged_wide_prefix(rows_prefix);
        lines[1].with[1] = paged_wide_own(rows_own);
        lines[0].with[0] = rows_prefix > 0 && !lines[1].with[0];
        lines[0].with[1] = rows_own > 0 && !lines[1].with[1];
        const bool few = lines[0].with[0] || lines[0].with[1], many = lines[1].with[0] || lines[1].with[1];
        // Tiles of 256 rows where every level has that many: K and V are read half as often.
        const bool tall = (!lines[1].with[0] || rows_prefix > 128) && (!lines[1].with[1] || rows_own > 128);
        lines[0].tile_shift = log2_of(PAGED_TILE);
        lines[1].tile_shift = log2_of(PAGED_WIDE_TILE);
        lines[1].grouped = 1;
        lines[1].tall = tall;
        // Known here: one query a sequence where q_start is not given, and all of them behind a single prefix.
        lines[0].spare = (!lines[0].with[0] || (groups == 1 && (int64_t)q_tokens * sh.q_per_kv <= 8)) &&
                         (!lines[0].with[1] || !q_start);
        bool ok = true;
        if (many) ok &= paged_line(ctx, a, lines[1], tall ? 256 : 128, std::min(ctx->sms, PAGED_WIDE_CTAS), (unsigned char *)workspace, off);
        const int64_t rows_few = std::max(lines[0].with[0] ? rows_prefix : 0, lines[0].with[1] ? rows_own : 0);
        if (few) ok &= paged_line(ctx, a, lines[0], rows_few <= 16 ? 16 : PAGED_ROWS, std::min(ctx->sms * 2, PAGED_MAX_CTAS), (unsigned char *)workspace, off);
        if (!ok) return fail(ctx, VERKV_EINVAL, "paged_attend: more than 2^31 steps of work in one call");
        if (off > workspace_bytes) return fail(ctx, VERKV_EINVAL, "paged_attend: workspace too small");
        CUtensorMap map;
        auto make_map = [&](int tile) {
            return paged_tensor_map(&map, pages->kv, pages->dtype, (long long)pages->num_pages * a.hkv * pages->page_tokens,
                                    sh.head_dim, std::min(pages->page_tokens, tile));
        };
        // Side by side, the longer one begins first; one after the other, k_paged, whose start is the longer
        // one with many sequences, begins while the kernel ahead of the call still runs.
        const bool beside = few && many && paged_share(lines[1], lines[0], ctx->sms);
        // (launches that are timed one by one wait for one another)
        if (few && many && !ctx->prof_on) a.ready = (unsigned long long *)workspace;
        for (int turn = 0; turn < 2; ++turn) {
            const bool wide = (turn == 0) == (beside || !few);
            if (!(wide ? many : few)) continue;
            const bool second = turn == 1 && a.ready;
            VERKV_CUDA(make_map(wide ? PAGED_WIDE_TILE : PAGED_TILE), "tensor map of the pages");
            VERKV_CUDA(tracked(ctx, wide ? VERKV_K_PAGED_WIDE : VERKV_K_PAGED, ctx->main, [&] {
                           return wide ? launch_paged_wide(a, lines[1], map, second, pages->dtype, sh.head_dim, ctx->main)
                                       : launch_paged(a, lines[0], map, second, pages->dtype, sh.head_dim, ctx->main);
                       }), wide ? "k_paged_wide" : "k_paged");
        }
    }
    VERKV_CUDA(tracked(ctx, VERKV_K_PAGED_MERGE, ctx->main, [&] { return launch_paged_merge(a, both, type, sh.head_dim, ctx->main); }), "k_paged_merge");
    return VERKV_OK;
} catch (...) {
    return VERKV_ECUDA;
}

verkv_status verkv_test_inject(verkv_ctx *ctx, int what, int64_t value) {
    if (!ctx) return VERKV_EINVAL;
    switch (what) {
        case VERKV_INJECT_COPY_FAIL:
            if (value < 0) break;
            ctx->inject_copy_fail = value;
            return VERKV_OK;
        case VERKV_INJECT_BETA_MAXIT:
            if (value < 0 || value > 64) break;
            ctx->beta_maxit = (int)value;
            return VERKV_OK;
        case VERKV_INJECT_SCORE_STALL:
            if (value < 1000 || value > 1000000000LL) break;
            ctx->score_stall_ns = value;
            return VERKV_OK;
        case VERKV_INJECT_WEIGH_STALL:
            if (value < 1000 || value > 1000000000LL) break;
            ctx->weigh_stall_ns = value;
            return VERKV_OK;
        case VERKV_INJECT_PAGED_STALL:
        case VERKV_INJECT_PAGED_LIMIT:
            if (value < 1000 || value > 1000000000LL) break;
            ctx->paged_wait_ns = value;
            ctx->paged_stall = what == VERKV_INJECT_PAGED_STALL;
            return VERKV_OK;
        case VERKV_INJECT_SELECT_GATHER:
            if (value < 0 || value > 1) break;
            ctx->sel_gather = (int)value;
            return VERKV_OK;
        default:
            break;
    }
    return fail(ctx, VERKV_EINVAL, "test_inject: unknown injection or value out of range");
}

verkv_status verkv_profile_enable(verkv_ctx *ctx, int on) {
    if (!ctx) return VERKV_EINVAL;
    ctx->prof_on = on != 0;
    return VERKV_OK;
}

verkv_status verkv_profile_read(verkv_ctx *ctx, int64_t *launches, double *total_ms) {
    if (!ctx || !launches || !total_ms) return VERKV_EINVAL;
    VERKV_CUDA(cudaSetDevice(ctx->device), "cudaSetDevice");
    VERKV_CUDA(cudaStreamSynchronize(ctx->side), "cudaStreamSynchronize(side)");
    VERKV_CUDA(cudaStreamSynchronize(ctx->main), "cudaStreamSynchronize(main)");
    for (const auto &r : ctx->prof_recs) {
        float ms = 0.0f;
        VERKV_CUDA(cudaEventElapsedTime(&ms, r.a, r.b), "cudaEventElapsedTime");
        launches[r.kernel] += 1;
        total_ms[r.kernel] += ms;
    }
    ctx->prof_recs.clear();
    ctx->prof_used = 0;
    return VERKV_OK;
}

verkv_status verkv_profile_timeline(verkv_ctx *ctx, int64_t max_records, int32_t *kernel,
                                    double *start_ms, double *end_ms, int64_t *n_out) {
    if (!ctx || !kernel || !start_ms || !end_ms || !n_out || max_records < 0) return VERKV_EINVAL;
    VERKV_CUDA(cudaSetDevice(ctx->device), "cudaSetDevice");
    VERKV_CUDA(cudaStreamSynchronize(ctx->side), "cudaStreamSynchronize(side)");
    VERKV_CUDA(cudaStreamSynchronize(ctx->main), "cudaStreamSynchronize(main)");
    int64_t k = 0;
    for (const auto &r : ctx->prof_recs) {
        if (k >= max_records) break;
        float a = 0.0f, b = 0.0f;
        VERKV_CUDA(cudaEventElapsedTime(&a, ctx->prof_recs[0].a, r.a), "cudaEventElapsedTime");
        VERKV_CUDA(cudaEventElapsedTime(&b, ctx->prof_recs[0].a, r.b), "cudaEventElapsedTime");
        kernel[k] = r.kernel;
        start_ms[k] = a;
        end_ms[k] = b;
        ++k;
    }
    *n_out = k;
    return VERKV_OK;
}

verkv_status verkv_launch_counts(verkv_ctx *ctx, int64_t *out) {
    if (!ctx || !out) return VERKV_EINVAL;
    for (int k = 0; k < VERKV_K_COUNT; ++k) out[k] = ctx->launches[k];
    return VERKV_OK;
}

const char *verkv_kernel_name(int k) {
    static const char *names[VERKV_K_COUNT] = {
        "k_pc_solve", "k_pc_gather", "k_sketch", "k_score", "k_certify",
        "k_partial(pivotal)", "k_refine", "k_partial(staged)", "k_merge",
        "k_dense_host", "k_dense_merge", "k_shortlist", "fetch_copy", "fetch_gather",
        "k_heads", "k_paged", "k_paged_wide", "k_paged_merge", "k_paged_q4", "k_q4_values", "k_weigh", "k_evict"};
    return (k >= 0 && k < VERKV_K_COUNT) ? names[k] : "";
}

const char *verkv_last_error(verkv_ctx *ctx) { return ctx ? ctx->last_error.c_str() : ""; }

}  // extern "C"
