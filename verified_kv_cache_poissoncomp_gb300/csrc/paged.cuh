// paged.cuh -- argument blocks of the head and paged-attention kernels, and the line of work that
// the attention kernels share.
//
// The line.  Segments are what a set of query rows attends: a shared prefix (rows: every query of
// its group) or a sequence's own pages (rows: its queries).  A segment splits into units: one KV
// head and one tile of up to `tt` query tokens, all q_per_kv heads of each.  A unit's work is the
// number of `tile`-token steps over what its last query sees.  All units' work, laid end to end
// (segment, row tile, head, step), is cut into equal runs of `per` steps, one for each CTA, wherever
// the cuts fall: however uneven the lengths are, no CTA has more than `per` steps, a long unit is
// shared by many CTAs and a CTA takes many short ones.  A run that holds the end of one unit and the
// start of the next costs a CTA about PAGED_SLACK steps more than one piece of the same length: where
// units are few, each gets the same whole number of runs (`room` steps of the line, its own or not),
// if they need not be longer by more than that (8 sequences behind 40000 tokens 56.3 -> 48.2 us, 64
// behind 32768 72.5 -> 62.5).  Lengths are read on the device, so a captured graph follows them.
//
// The piece of unit u in run c goes to the partial slot c + u: walking the line, each step to the next
// piece raises exactly one of the two.  Row tiles come before heads so that the CTAs which read the same
// K and V for other rows do so at about the same time, from the L2 cache (heads first, 1024 rows read a
// 134 MB prefix four times from memory).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#ifdef __CUDACC__
#include <cuda_fp16.h>

#include "verkv_common.cuh"
#endif
#include "verkv_internal.h"

namespace verkv {

// Norm, rotation and append (k_heads.cu).  Strides in elements; a null weight: that part is not
// normalised; rd 0: no rotation; pages null: keys go to k_out and there are no values.
struct HeadsArgs {
    const uint16_t *q, *k, *v;
    uint16_t *q_out, *k_out, *pages;
    long long q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, qo_ts, qo_hs, ko_ts, ko_hs;
    const uint16_t *wq, *wk;
    const uint64_t *turns;
    const int32_t *positions, *seq, *index, *table;
    uint32_t *err;
    int tokens, hq, hk, hv;  // heads of each token to do: queries, keys, values
    int chunks, chunks_q, chunks_k;  // warps a token takes, of them for queries and keys (set by the launcher)
    int rd, interleaved;
    int table_rows, table_stride, num_pages, page_shift;
    float eps;
};
cudaError_t launch_heads(const HeadsArgs &a, int dtype, int d, cudaStream_t s);

// ---------------------------------------------------------------------------------------------
struct PagedLevel {
    const int32_t *table;
    const int32_t *length;
    int rows, stride, max_length;  // rows 0: the level is absent
};

// One launch's share of the work.
struct PagedLine {
    int with[2];                // the levels in it: prefixes first
    int tile_shift;             // log2 of the tokens of a step
    int tt_shift;               // log2 of the query tokens of a row tile, tt
    int ctas;                   // CTAs launched
    int slots;                  // partial slots there is room for
    int tall;                   // (host: tiles of 256 rows)
    int spare;                  // (host: no unit has more than 8 rows)
    double cost, units;         // (host: us of one SM; about how many units)
    int2 *rec;                  // {per, room}, then {work before, units before} of each segment with work; per 0: a bad segment, no work
    int grouped;                // 0: part_o [slots][tt * G][d]; 1: [slots][tt * G / 4][d / 4][4 rows][4]
    float *part_o;
    float *part_ml;             // [slots][tt * G][2]: running maximum (log2 units) and sum
};

struct PagedArgs {
    const uint16_t *q;
    long long q_ts, q_hs;
    const int32_t *q_start, *group_start;
    PagedLevel level[2];  // of the prefixes, and of the sequences' own tokens
    // What no segment looks at: lengths of levels whose bound is 0, and starts of a level that is absent.
    const int32_t *zero_length[2];
    int zero_rows[2];
    bool check_q_start, check_group_start, unseen;  // unseen: any of these
    int seqs, q_tokens, hkv, g_shift, page_shift, num_pages;  // q_per_kv = 2^g_shift
    float scale_log2;  // logits are taken in units of log 2
    uint32_t *err;
    const float *prior_o, *prior_lse;
    uint16_t *o;
    float *lse;
    unsigned long long wait_ns;  // limit of the kernels' waits
    int stall;                   // injected: the first copies of the first CTA are not issued
    unsigned long long *ready;   // where the call's first kernel says that it may read (in the workspace), or null
};

constexpr int PAGED_MAX_CTAS = 304;   // of k_paged: two an SM
constexpr int PAGED_WIDE_CTAS = 152;  // of k_paged_wide
constexpr int PAGED_TILE = 64;        // tokens of a step of k_paged
constexpr int PAGED_ROWS = 32;        // most rows of its units (16 or 32)
constexpr int PAGED_WIDE_TILE = 128;  // and of k_paged_wide
constexpr unsigned long long PAGED_WAIT_NS = 1000000000ull;  // 1 s: limit of a wait
constexpr int PAGED_LINES = 2;        // launches of a call: one of each kernel at most
constexpr int PAGED_SLACK = 2;        // steps a run may be longer for units of whole runs
constexpr int PAGED_ROOMS_MOST = 1 << 21;  // steps of a line whose units may get whole runs

cudaError_t paged_tensor_map(CUtensorMap *map, const void *kv, int dtype, long long rows, int d, int box_rows);
// second: the launch before it on the stream is this call's other kernel, which it need not wait for to
// begin (see paged_begin).
cudaError_t launch_paged(const PagedArgs &a, const PagedLine &l, const CUtensorMap &map, bool second, int dtype, int d,
                         cudaStream_t s);
cudaError_t launch_paged_wide(const PagedArgs &a, const PagedLine &l, const CUtensorMap &map, bool second, int dtype,
                              int d, cudaStream_t s);
struct PagedLines {
    PagedLine l[PAGED_LINES];
};
cudaError_t launch_paged_merge(const PagedArgs &a, const PagedLines &lines, int dtype, int d, cudaStream_t s);

#ifdef __CUDACC__
// ---------------------------------------------------------------------------------------------
// The start of a call's kernel, by the one warp that reads for its CTA, before the CTA's first barrier: on
// return the kernels ahead on the stream have completed and their writes are visible, to copies too.
//
// The call's first kernel waits for them.  The second one, whose launch it allows right then, would wait
// for the first one's end with the same instruction, and that an early launch hands on what the first one
// waited for is nowhere promised.  So the first kernel, having waited, stores a word with release and the
// second loads it with acquire, which orders all that was visible to the one before the other's reads.
// A second kernel that does not find the word (it is not yet there) waits for the first one's end: nothing
// spins.  The merge clears the word for the next call; what an unused workspace holds by chance is some
// other word.  (34 sequences behind two prefixes 34.1 -> 34.9 us, 256 behind one 147.5 -> 149, 8 no more.)
constexpr unsigned long long PAGED_READY = 0x9D5C3A71E64B28F1ull;
__device__ __forceinline__ void paged_begin(const PagedArgs &a, bool second) {
    if (!second) {
        pdl_wait();
        if (a.ready && blockIdx.x == 0) {
            if ((threadIdx.x & 31) == 0) asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(a.ready), "l"(PAGED_READY) : "memory");
            __syncwarp();
        }
    } else {
        unsigned long long word;
        asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(word) : "l"(a.ready) : "memory");
        if (__any_sync(0xFFFFFFFFu, word != PAGED_READY)) pdl_wait();
        asm volatile("fence.proxy.async;" ::: "memory");  // the copies' reads behind these
    }
    pdl_trigger();
}

struct PagedSeg {
    int q0, qn, len, row;
    bool own;
};

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

__device__ __forceinline__ int paged_segments(const PagedArgs &a, const PagedLine &l) {
    return (l.with[0] ? a.level[0].rows : 0) + (l.with[1] ? a.level[1].rows : 0);
}

// Segment i.  Everything read from the device is clamped to its range, so that no later index
// leaves the tensors; `bad` is set where that changed something.
__device__ __forceinline__ PagedSeg paged_segment(const PagedArgs &a, const PagedLine &l, int i, bool &bad) {
    PagedSeg s;
    const int np = l.with[0] ? a.level[0].rows : 0;
    s.own = i >= np;
    s.row = s.own ? i - np : i;
    int s0 = s.row, s1 = s.row + 1;
    if (!s.own) {
        const int r0 = a.group_start ? a.group_start[s.row] : 0;
        const int r1 = a.group_start ? a.group_start[s.row + 1] : a.seqs;
        s0 = clampi(r0, 0, a.seqs);
        s1 = clampi(r1, s0, a.seqs);
        bad |= s0 != r0 || s1 != r1 || (s.row == 0 && r0 != 0) || (s.row == np - 1 && r1 != a.seqs);
    }
    const int r0 = a.q_start ? a.q_start[s0] : s0;
    const int r1 = a.q_start ? a.q_start[s1] : s1;
    s.q0 = clampi(r0, 0, a.q_tokens);
    const int q1 = clampi(r1, s.q0, a.q_tokens);
    bad |= s.q0 != r0 || q1 != r1 || (s0 == 0 && s.q0 != 0) || (s1 == a.seqs && q1 != a.q_tokens);
    s.qn = q1 - s.q0;
    const PagedLevel &lv = a.level[s.own ? 1 : 0];
    const int len = lv.length[s.row];
    s.len = clampi(len, 0, lv.max_length);
    bad |= s.len != len;
    return s;
}

__device__ __forceinline__ int paged_row_tiles(const PagedSeg &s, const PagedLine &l) {
    return (s.qn + (1 << l.tt_shift) - 1) >> l.tt_shift;
}

// Tokens the last query of row tile m sees.
__device__ __forceinline__ int paged_visible(const PagedSeg &s, const PagedLine &l, int m) {
    if (!s.own) return s.len;
    const int last = min(s.qn, (m + 1) << l.tt_shift) - 1;
    return clampi(s.len - (s.qn - 1 - last), 0, s.len);
}
__device__ __forceinline__ int paged_steps(const PagedSeg &s, const PagedLine &l, int m) {
    return (paged_visible(s, l, m) + (1 << l.tile_shift) - 1) >> l.tile_shift;
}
// The sum over k < n of ceil(max(0, b + (k + 1) tt) / T), tt = 2^tt_shift and T = 2^tile_shift.  Without the
// terms that are 0 it is the sum of floor((y + k tt) / T), y >= T.  Where tt is a multiple of T, each term is
// tt / T more than the one before; else, with r = T / tt and c = floor((y mod T) / tt), they are floor(y / T) +
// floor((c + k) / r), and the sum of floor(j / r) over j < c + n has r of each value.
// (A call, as is the search below: a decode step's launches pass this code by.  In line, 8 sequences behind
// 32K tokens took 45.2 us, so 44.0; 43.6 with a loop over the tiles.)
static __device__ __noinline__ int paged_ramp(int b, int n, int tt_shift, int tile_shift) {
    const int none = b >= 0 ? 0 : min(n, -b >> tt_shift);
    n -= none;
    const int y = b + ((none + 1) << tt_shift) + (1 << tile_shift) - 1;
    const int w = n * (y >> tile_shift);
    if (tt_shift >= tile_shift) return w + (int)(((unsigned)n * (unsigned)(n - 1) >> 1) << (tt_shift - tile_shift));
    const int shift = tile_shift - tt_shift;
    const unsigned j = n + ((y & ((1 << tile_shift) - 1)) >> tt_shift), q = j >> shift;
    return w + (int)((q * (q - 1) >> 1 << shift) + (j & ((1u << shift) - 1)) * q);
}
// What all row tiles before m take of the line, for one head.  (A room is given to every unit or none.)
// Of own tokens, the last query of row tile k sees len - qn + (k + 1) tt, that of the last tile all.
__device__ __forceinline__ int paged_steps_before(const PagedSeg &s, const PagedLine &l, int m, int room) {
    if (!s.own || room) return m * (room ? room : paged_steps(s, l, 0));
    const int nt = paged_row_tiles(s, l);
    int w = m == nt && m > 0 ? (s.len + (1 << l.tile_shift) - 1) >> l.tile_shift : 0;
    if (nt > 1) w += paged_ramp(s.len - s.qn, min(m, nt - 1), l.tt_shift, l.tile_shift);
    return w;
}

// The last of `nt` row tiles of own tokens whose steps begin at r or before it, counted over all `heads`.
static __device__ __noinline__ int paged_tile_at(int b, int nt, int r, int heads, int tt_shift, int tile_shift) {
    int m = 0;
#pragma unroll 1
    for (int end = nt; end - m > 1;) {
        const int mid = (m + end) >> 1;
        if (paged_ramp(b, mid, tt_shift, tile_shift) * heads <= r) m = mid;
        else end = mid;
    }
    return m;
}

// One warp's walk over the run of this CTA.  A kernel calls start() and next() at one place each: a
// launch begins with cold instruction caches and fetches its code line by line, so its size is time.
// All lanes hold the same values.  The host has checked that a whole line's steps and units fit 31
// bits; a segment outside its range empties the line.
// ROOMS: units may be given rooms.  (k_paged's runs change units at less cost, and its start at more:
// with rooms 8 sequences of up to 512 tokens took 11.1 us for 10.7.)
template <bool ROOMS>
struct PagedWalk {
    int w, w1;   // next step, end of the run
    int room;    // of every unit on the line, or 0: its steps
    int Wx, Ux;  // work and units before the segment
    int per_head;
    int seg, n, nt;
    PagedSeg s;
    // the current piece
    int head, m, t0, t1, slot;

    __device__ __forceinline__ void load(const PagedArgs &a, const PagedLine &l) {
        bool bad = false;
        s = paged_segment(a, l, seg, bad);
        nt = paged_row_tiles(s, l);
        per_head = paged_steps_before(s, l, nt, ROOMS ? room : 0);
    }

    // Places the walk at the start of run `c`.  Called by a whole warp; the warp of run 0 also writes
    // how long a run is and reports bad segments.  First the whole line's steps, keeping each segment's
    // in shared memory (`cap` of them, at least 32) as it goes, then the place.
    __device__ __forceinline__ void start(const PagedArgs &a, const PagedLine &l, int c, int2 *cache, int cap) {
        const int lane = threadIdx.x & 31;
        n = paged_segments(a, l);
        seg = n;
        w = w1 = room = 0;
        bool bad = false;
        int total = 0;
#pragma unroll 4
        for (int i = lane; i < n; i += 32) {
            const PagedSeg g = paged_segment(a, l, i, bad);
            const int t = paged_row_tiles(g, l), h = paged_steps_before(g, l, t, 0);
            total += h;
            if (i < cap) cache[i] = make_int2(h, t);
        }
        total = __reduce_add_sync(0xFFFFFFFFu, total) * a.hkv;
        bad = __any_sync(0xFFFFFFFFu, bad);
        int per = bad ? 0 : (int)max(1u, ((unsigned)total + l.ctas - 1) / (unsigned)l.ctas);
        if (ROOMS && n <= 32 && per > 0 && total < PAGED_ROOMS_MOST) {
            // A lane a segment.  (Quotients by the fast reciprocal, whose error of two units of the last place
            // is less than the halves added here, up to PAGED_ROOMS_MOST steps; p is put right if not.)
            const int2 g = lane < n ? cache[lane] : make_int2(0, 0);
            const int units = __reduce_add_sync(0xFFFFFFFFu, g.y) * a.hkv;
            if (units <= l.ctas && total > 0) {
                const int runs = (int)__fdividef(l.ctas + 0.5f, (float)units);
                // row tiles of a sequence's own tokens differ: their sum is more than any
                const int each = lane >= (l.with[0] ? a.level[0].rows : 0) ? g.x : (int)(__fdividef((float)g.x, (float)max(g.y, 1)) + 0.5f);
                const int longest = __reduce_max_sync(0xFFFFFFFFu, each);
                int p = (int)__fdividef(longest + runs - 0.5f, (float)runs);
                p += p * runs < longest ? 1 : 0;
                if (p <= per + PAGED_SLACK) {
                    per = p;
                    room = runs * p;
                    total = units * room;
                    if (lane < n) cache[lane].x = g.y * room;
                }
            }
        }
        if (c == 0 && lane == 0) {
            l.rec[0] = make_int2(per, room);
            if (bad) raise_error(a.err, ERR_PAGE);
        }
        if (bad) return;
        w = (int)min((long long)total, (long long)c * per);
        w1 = min(total, w + per);
        if (w >= w1) return;
        int wx = 0, ux = 0;
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + lane;
            int gh = 0, gt = 0;  // steps of one head, row tiles
            if (i < cap && i < n) {
                gh = cache[i].x;
                gt = cache[i].y;
            } else if (i < n) {
                const PagedSeg g = paged_segment(a, l, i, bad);
                gt = paged_row_tiles(g, l);
                gh = paged_steps_before(g, l, gt, 0);  // (no rooms with as many)
            }
            const int mw = gh * a.hkv, mu = gt * a.hkv;
            int sw = mw, su = mu;  // inclusive sums over the lanes
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int pw = __shfl_up_sync(0xFFFFFFFFu, sw, o), pu = __shfl_up_sync(0xFFFFFFFFu, su, o);
                if (lane >= o) {
                    sw += pw;
                    su += pu;
                }
            }
            const int ew = wx + sw - mw, eu = ux + su - mu;
            const unsigned hit = __ballot_sync(0xFFFFFFFFu, w < w1 && w >= ew && w < ew + mw);
            if (hit) {  // the run begins in this lane's segment
                const int at = __ffs(hit) - 1;
                seg = i0 + at - 1;  // (next() goes on to it)
                Wx = __shfl_sync(0xFFFFFFFFu, ew, at);
                Ux = __shfl_sync(0xFFFFFFFFu, eu, at);
                per_head = nt = 0;
                return;
            }
            wx += __shfl_sync(0xFFFFFFFFu, sw, 31);
            ux += __shfl_sync(0xFFFFFFFFu, su, 31);
        }
    }

    // The next piece; false at the end of the run.
    __device__ __forceinline__ bool next(const PagedArgs &a, const PagedLine &l, int c) {
        if (w >= w1) return false;
        while (w >= Wx + per_head * a.hkv) {
            if (++seg >= n) return false;  // lengths changed under the kernel
            Wx += per_head * a.hkv;
            Ux += nt * a.hkv;
            load(a, l);
        }
        // The run in which a segment begins writes its record for the merge.
        if (w == Wx && (threadIdx.x & 31) == 0) l.rec[1 + seg] = make_int2(Wx, Ux);
        int r = w - Wx;
        m = 0;
        int steps = paged_steps(s, l, 0), span = ROOMS && room ? room : steps;
        if (!s.own || (ROOMS && room)) {
            m = (unsigned)r / (unsigned)(span * a.hkv);
            r -= m * span * a.hkv;
            if (ROOMS && s.own) steps = paged_steps(s, l, m);
        } else if (nt > 1) {
            // (not an empty tile: r is inside the segment)
            m = paged_tile_at(s.len - s.qn, nt, r, a.hkv, l.tt_shift, l.tile_shift);
            r -= paged_ramp(s.len - s.qn, m, l.tt_shift, l.tile_shift) * a.hkv;
            span = steps = paged_steps(s, l, m);
        }
        head = (unsigned)r / (unsigned)span;
        r -= head * span;
        t0 = r;
        t1 = min(steps, r + (w1 - w));
        slot = c + Ux + m * a.hkv + head;
        w += min(span - r, w1 - w);
        return t0 < t1;  // (a run behind the end of a unit with room has nothing to do)
    }
};

// 16-bit types of the pages.
// SHIFT: weights are 2^(l - m + SHIFT), up to 2^8 in fp16, away from its subnormals.
struct PgBf16 {
    static constexpr float SHIFT = 0.0f;
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t y;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
        return y;
    }
    static __device__ __forceinline__ float2 unpack(uint32_t x) { return make_float2(bf16lo(x), bf16hi(x)); }
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
struct PgF16 {
    static constexpr float SHIFT = 8.0f;
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t y;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
        return y;
    }
    static __device__ __forceinline__ float2 unpack(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2 *>(&x)); }
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
// What rounding a pair of weights to 16 bits has left out of it, in 16 bits of its own: together they hold
// a weight to within 2^-16 (bf16) or 2^-22 (fp16) of itself.
template <typename T>
__device__ __forceinline__ uint32_t pack_rest(uint32_t packed, float lo, float hi) {
    const float2 f = T::unpack(packed);
    unsigned long long v, w;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    asm("mov.b64 %0, {%1, %2};" : "=l"(w) : "f"(-f.x), "f"(-f.y));
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(w));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
    return T::pack(lo, hi);
}
// 2^x to within 2 units of the last place, 0 for -infinity.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ bool mbar_poll(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity & 1u)
        : "memory");
    return done != 0;
}

// Wait for phase `parity` of the barrier at shared address `bar`; false when *abort is set or the time
// is up.  The first poll is in line and the rest is a call: a warp that issues products or copies runs
// between others that fill the instruction cache, and pays for each line of code it passes.
static __device__ __noinline__ bool paged_wait_long(uint32_t bar, uint32_t parity, volatile int *abort, unsigned long long limit_ns) {
    unsigned long long t0 = 0;
    for (;;) {
        for (int i = 0; i < 16; ++i)
            if (mbar_poll(bar, parity)) return true;
        const unsigned long long t = globaltimer_ns();
        if (t0 == 0) t0 = t;
        if (*abort || t - t0 > limit_ns) return false;
    }
}
__device__ __forceinline__ bool paged_wait(uint32_t bar, uint32_t parity, volatile int *abort, unsigned long long limit_ns) {
    return mbar_poll(bar, parity) || paged_wait_long(bar, parity, abort, limit_ns);
}

__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}
#endif

}  // namespace verkv
