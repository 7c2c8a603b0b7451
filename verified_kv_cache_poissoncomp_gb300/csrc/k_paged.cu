// k_paged.cu -- attention over the paged cache for few query rows, and the merge of partial sums.
//
//   o = sum_i 2^(l_i - m) v_i / sum_i 2^(l_i - m),   l_i = q . k_i scale log2(e), m the running maximum
//
// k_paged: up to 32 query rows (query tokens x heads of one KV head) against a run of cached tokens.
// Bound by the bytes of K and V: a decode step has q_per_kv rows a sequence, a few flops per byte.
// One warp walks the CTA's run of the line (paged.cuh) and copies 64-token steps of K and V into
// a shared-memory ring by TMA (boxes of one page's tokens x 64 channels, 128-byte swizzle); what a
// step is (which rows, which tokens, whether a unit begins or ends with it) travels beside it, so
// one thread's walk drives the CTA.  Four warps take 16 tokens of a step each: S = Q K^T with the
// rows as the m16 of mma.m16n8k16 (K by ldmatrix), the softmax in registers -- each warp keeps its
// own running maximum and sum and rescales only when some row's maximum rises -- and P, already
// in the A operand's layout, times V (ldmatrix, transposed).  At a unit's end the four warps' states
// are joined in shared memory and written as one partial.
//
// k_paged_merge: a warp per query token and head joins the partials of its prefix and its own
// pages, and the caller's prior state, in a fixed order.
#include <math.h>

#include <algorithm>

#include "paged.cuh"
#include "pivotal_mma.cuh"
#include "verkv_common.cuh"

namespace verkv {

namespace {

constexpr int PG_CONS = 4;                     // consumer warps: 16 tokens of a step each
constexpr int PG_NT = 32 * (PG_CONS + 1);      // and one warp that walks and copies

struct StepDesc {
    int flags;       // PG_FIRST | PG_LAST | PG_END
    int valid;       // tokens of the step that some row of the unit sees
    int tok0;        // the step's first token
    int q0, nq;      // query tokens of the row tile
    int head;        // KV head
    int lim0, limd;  // tokens the tile's first query sees, and how many more each next one does
    int slot;        // partial slot, or -1
};
enum { PG_FIRST = 1, PG_LAST = 2, PG_END = 4 };

template <int D, int MT>
struct PagedLayout {
    static constexpr int HALVES = D / 64;
    static constexpr int BOX = PAGED_TILE * 128;
    static constexpr int STAGE = 2 * HALVES * BOX;
    // Two CTAs an SM where 16 rows' sums leave room for them, else one.
    static constexpr int NS = MT == 1 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 10);
    static constexpr int CTAS = MT == 1 ? 2 : 1;
    static constexpr int R = MT * 16;
    static constexpr int RED = NS * STAGE;                  // float [2][R][D]
    static constexpr int ML = RED + 2 * R * D * 4;          // float [4][R][2]
    static constexpr int DESC = ML + PG_CONS * R * 2 * 4;   // StepDesc [NS]
    static constexpr int BARS = (DESC + NS * (int)sizeof(StepDesc) + 7) / 8 * 8;  // full, empty [NS], join
    static constexpr int BYTES = BARS + (2 * NS + 1) * 8 + 8;
};

template <typename T, int D, int MT>
__global__ void __launch_bounds__(PG_NT, PagedLayout<D, MT>::CTAS)
    k_paged(const PagedArgs a, const PagedLine l, const __grid_constant__ CUtensorMap map) {
    using LY = PagedLayout<D, MT>;
    constexpr int KS = D / 16, NS = LY::NS, R = LY::R;
    extern __shared__ __align__(1024) unsigned char pg_smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(pg_smem + LY::BARS), *empty = full + NS, *join = empty + NS;
    volatile int *abort = reinterpret_cast<volatile int *>(join + 1);
    StepDesc *desc = reinterpret_cast<StepDesc *>(pg_smem + LY::DESC);
    float *red = reinterpret_cast<float *>(pg_smem + LY::RED);
    float *ml = reinterpret_cast<float *>(pg_smem + LY::ML);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int k = 0; k < NS; ++k) {
            mbar_init(&full[k], 1);
            mbar_init(&empty[k], PG_CONS);
        }
        mbar_init(join, PG_CONS);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *abort = 0;
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();

    if (warp == PG_CONS) {
        if (lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map)) : "memory");
        const int box = min(1 << a.page_shift, PAGED_TILE);  // tokens of a page in one step
        PagedWalk wk;
        wk.start(a, l, blockIdx.x);
        int j = 0;
        bool go = true;
        while (go && wk.next(a, l, blockIdx.x)) {
            const PagedLevel &lv = wk.s.own ? a.own : a.prefix;
            const int32_t *row = lv.table + (long long)wk.s.row * lv.stride;
            const int vis = paged_visible(wk.s, l.tt, wk.m);
            int ids = 0, ids0 = 1, ids1 = 0;  // lane i: id of page ids0 + i of the sequence
            for (int t = wk.t0; t < wk.t1; ++t, ++j) {
                const int k = j % NS;
                go = *abort == 0;
                if (go && j >= NS) go = mbar_wait_or_abort(&empty[k], (uint32_t)((j / NS - 1) & 1), abort);
                go = __all_sync(0xFFFFFFFFu, go);
                if (!go) break;
                const int tok0 = t * PAGED_TILE, valid = min(PAGED_TILE, vis - tok0);
                const int pages = (valid + box - 1) / box;
                const int p0 = tok0 >> a.page_shift;
                if (p0 < ids0 || p0 + pages > ids1) {
                    ids0 = p0;
                    ids1 = p0 + 32;
                    const int p = p0 + lane;
                    int id = 0;
                    if (p <= (vis - 1) >> a.page_shift) {
                        id = row[p];
                        if (id < 0 || id >= a.num_pages) {
                            raise_error(a.err, ERR_PAGE);
                            id = 0;
                        }
                    }
                    ids = id;
                }
                if (lane == 0) {
                    StepDesc s;
                    s.flags = (t == wk.t0 ? PG_FIRST : 0) | (t + 1 == wk.t1 ? PG_LAST : 0);
                    s.valid = valid;
                    s.tok0 = tok0;
                    s.q0 = wk.s.q0 + wk.m * l.tt;
                    s.nq = min(l.tt, wk.s.qn - wk.m * l.tt);
                    s.head = wk.head;
                    s.lim0 = wk.s.own ? wk.s.len - (wk.s.qn - 1 - wk.m * l.tt) : wk.s.len;
                    s.limd = wk.s.own ? 1 : 0;
                    s.slot = wk.slot < l.slots ? wk.slot : -1;
                    if (s.slot < 0) raise_error(a.err, ERR_PAGE);
                    desc[k] = s;
                    mbar_expect_tx(&full[k], (uint32_t)(pages * box * 4 * D));
                }
                __syncwarp();
                const int id = __shfl_sync(0xFFFFFFFFu, ids, (p0 + lane - ids0) & 31);
                if (lane < pages) {
                    // page ids0 + i holds tokens tok0 + lane * box ..: a page of more than one step is
                    // read at the step's offset in it
                    const int y = (((id * a.hkv + wk.head) << a.page_shift) + ((tok0 + lane * box) & ((1 << a.page_shift) - 1)));
                    unsigned char *st = pg_smem + (size_t)k * LY::STAGE + lane * box * 128;
#pragma unroll
                    for (int b = 0; b < 2 * LY::HALVES; ++b) tma_load_2d(st + b * LY::BOX, &map, b * 64, y, &full[k]);
                }
                __syncwarp();
            }
        }
        if (go) {  // tell the consumers that the run is over
            const int k = j % NS;
            if (j >= NS) go = mbar_wait_or_abort(&empty[k], (uint32_t)((j / NS - 1) & 1), abort);
            if (go && lane == 0) {
                desc[k].flags = PG_END;
                mbar_arrive(&full[k]);
            }
        }
        if (!go) {
            // A wait ran out.  Let the copies of this CTA land before it exits: the steps j - NS ..
            // j - 1 are the ones that may be in flight.
            if (lane == 0) {
                *abort = 1;
                raise_error(a.err, ERR_TIMEOUT);
                for (int i = max(0, j - NS); i < j; ++i) mbar_wait_bounded(&full[i % NS], (uint32_t)((i / NS) & 1));
            }
        }
        __syncwarp();
    } else {
        const int g = lane >> 2, t = lane & 3, mi = lane >> 3, ri = lane & 7;
        uint32_t qf[MT][KS][4];
        float o[MT][D / 8][4], mx[MT][2], sum[MT][2];
        int lim[MT][2];
        int joins = 0;
        auto cons_sync = [&]() -> bool {
            __syncwarp();
            if (lane == 0) mbar_arrive(join);
            const bool ok = mbar_wait_or_abort(join, (uint32_t)(joins & 1), abort);
            ++joins;
            return __all_sync(0xFFFFFFFFu, ok);
        };
        for (int j = 0;; ++j) {
            const int k = j % NS;
            bool ok = *abort == 0 && mbar_wait_or_abort(&full[k], (uint32_t)((j / NS) & 1), abort);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                if (lane == 0) {
                    *abort = 1;
                    raise_error(a.err, ERR_TIMEOUT);
                }
                break;
            }
            const StepDesc s = desc[k];
            if (s.flags & PG_END) break;
            if (s.flags & PG_FIRST) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = mt * 16 + g + 8 * e, jj = r / a.G, hh = r - jj * a.G;
                        const bool real = jj < s.nq;
                        lim[mt][e] = real ? s.lim0 + s.limd * jj : 0;
                        mx[mt][e] = -INFINITY;
                        sum[mt][e] = 0.0f;
                        const uint16_t *qr = a.q + (long long)(s.q0 + (real ? jj : 0)) * a.q_ts + (long long)(s.head * a.G + hh) * a.q_hs;
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks) {
                            qf[mt][ks][e] = real ? *reinterpret_cast<const uint32_t *>(qr + ks * 16 + 2 * t) : 0u;
                            qf[mt][ks][2 + e] = real ? *reinterpret_cast<const uint32_t *>(qr + ks * 16 + 8 + 2 * t) : 0u;
                        }
                    }
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.0f;
                }
            }
            const int w0 = warp * 16;
            if (w0 < s.valid) {
                unsigned char *st = pg_smem + (size_t)k * LY::STAGE;
                const uint32_t kb = smem_addr(st), vb = kb + LY::HALVES * LY::BOX;
                if (w0 + 16 > s.valid) {
                    // V rows that nothing sees may hold anything, NaN too: a weight of 0 would keep it
                    for (int r = s.valid; r < w0 + 16; ++r)
                        if (lane < 8 * LY::HALVES)
                            *reinterpret_cast<uint4 *>(st + (LY::HALVES + (lane >> 3)) * LY::BOX + r * 128 + (lane & 7) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                    __syncwarp();
                }
                float sc[MT][2][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 8; ++e) sc[mt][e >> 2][e & 3] = 0.0f;
                {
                    const int r = w0 + (mi >> 1) * 8 + ri;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        uint32_t b[4];
                        ldsm_x4(b, kb + (ks / 4) * LY::BOX + r * 128 + ((((ks % 4) * 2 + (mi & 1)) ^ (r & 7)) << 4));
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            T::mma(sc[mt][0], qf[mt][ks], b[0], b[1]);
                            T::mma(sc[mt][1], qf[mt][ks], b[2], b[3]);
                        }
                    }
                }
                uint32_t pf[MT][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int tok = s.tok0 + w0 + nt * 8 + 2 * t + (e & 1);
                            float x = sc[mt][nt][e] * a.scale_log2;
                            x = tok < lim[mt][e >> 1] ? x : -INFINITY;
                            sc[mt][nt][e] = x;
                            top[e >> 1] = fmaxf(top[e >> 1], x);
                        }
                    bool rises = false;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], 1));
                        top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], 2));
                        rises |= top[e] > mx[mt][e];
                    }
                    if (__any_sync(0xFFFFFFFFu, rises)) {
                        float f[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float m = fmaxf(mx[mt][e], top[e]);
                            f[e] = m == mx[mt][e] ? 1.0f : exp2_fast(mx[mt][e] - m);  // (-inf: nothing summed yet)
                            mx[mt][e] = m;
                            sum[mt][e] *= f[e];
                        }
#pragma unroll
                        for (int n = 0; n < D / 8; ++n) {
                            o[mt][n][0] *= f[0];
                            o[mt][n][1] *= f[0];
                            o[mt][n][2] *= f[1];
                            o[mt][n][3] *= f[1];
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float m = mx[mt][e] == -INFINITY ? 0.0f : mx[mt][e];  // a row that sees nothing so far
                        float p[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            p[i] = exp2_fast(sc[mt][i >> 1][2 * e + (i & 1)] - m);
                            sum[mt][e] += p[i];
                        }
                        pf[mt][e] = T::pack(p[0], p[1]);
                        pf[mt][2 + e] = T::pack(p[2], p[3]);
                    }
                }
                const int r = w0 + (mi & 1) * 8 + ri;
#pragma unroll
                for (int c = 0; c < KS; ++c) {
                    uint32_t b[4];
                    ldsm_x4_t(b, vb + (c / 4) * LY::BOX + r * 128 + ((((c % 4) * 2 + (mi >> 1)) ^ (r & 7)) << 4));
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        T::mma(o[mt][2 * c], pf[mt], b[0], b[1]);
                        T::mma(o[mt][2 * c + 1], pf[mt], b[2], b[3]);
                    }
                }
                fence_proxy_async_smem();  // generic accesses before the slot's next copy
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[k]);

            if (s.flags & PG_LAST) {
                // Join the four warps' states: each scales its sums to the common maximum, then
                // 1 -> 0 and 3 -> 2, then 2 -> 0.
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        sum[mt][e] += __shfl_xor_sync(0xFFFFFFFFu, sum[mt][e], 1);
                        sum[mt][e] += __shfl_xor_sync(0xFFFFFFFFu, sum[mt][e], 2);
                        if (t == 0) {
                            float *p = ml + (warp * R + mt * 16 + g + 8 * e) * 2;
                            p[0] = mx[mt][e];
                            p[1] = sum[mt][e];
                        }
                    }
                if (!cons_sync()) break;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = mt * 16 + g + 8 * e;
                        float m = -INFINITY, z = 0.0f;
#pragma unroll
                        for (int w = 0; w < PG_CONS; ++w) m = fmaxf(m, ml[(w * R + r) * 2]);
                        const float ms = m == -INFINITY ? 0.0f : m;
#pragma unroll
                        for (int w = 0; w < PG_CONS; ++w) z += ml[(w * R + r) * 2 + 1] * exp2_fast(ml[(w * R + r) * 2] - ms);
                        const float f = exp2_fast(mx[mt][e] - ms);
#pragma unroll
                        for (int n = 0; n < D / 8; ++n) {
                            o[mt][n][2 * e] *= f;
                            o[mt][n][2 * e + 1] *= f;
                        }
                        mx[mt][e] = m;
                        sum[mt][e] = z;
                    }
                auto put = [&](float *buf) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int n = 0; n < D / 8; ++n)
                            reinterpret_cast<float4 *>(buf)[(mt * (D / 8) + n) * 32 + lane] =
                                make_float4(o[mt][n][0], o[mt][n][1], o[mt][n][2], o[mt][n][3]);
                };
                auto add = [&](const float *buf) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int n = 0; n < D / 8; ++n) {
                            const float4 v = reinterpret_cast<const float4 *>(buf)[(mt * (D / 8) + n) * 32 + lane];
                            o[mt][n][0] += v.x;
                            o[mt][n][1] += v.y;
                            o[mt][n][2] += v.z;
                            o[mt][n][3] += v.w;
                        }
                };
                if (warp & 1) put(red + (warp >> 1) * R * D);
                if (!cons_sync()) break;
                if (!(warp & 1)) add(red + (warp >> 1) * R * D);
                if (!cons_sync()) break;
                if (warp == 2) put(red);
                if (!cons_sync()) break;
                if (warp == 0) {
                    add(red);
                    if (s.slot >= 0) {
                        const int rows = s.nq * a.G;
                        float *po = l.part_o + (long long)s.slot * (l.tt * a.G) * D;
                        float *pm = l.part_ml + (long long)s.slot * (l.tt * a.G) * 2;
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int r = mt * 16 + g + 8 * e;
                                if (r >= rows) continue;
#pragma unroll
                                for (int n = 0; n < D / 8; ++n)
                                    *reinterpret_cast<float2 *>(po + r * D + n * 8 + 2 * t) =
                                        make_float2(o[mt][n][2 * e], o[mt][n][2 * e + 1]);
                                if (t == 0) *reinterpret_cast<float2 *>(pm + r * 2) = make_float2(mx[mt][e], sum[mt][e]);
                            }
                    }
                }
            }
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------------------------
// The last index i of 0 .. n with start[i] <= x (start ascending; -1: none).  The whole warp.
__device__ __forceinline__ int last_at_most(const int32_t *start, int n, int x) {
    int c = 0;
#pragma unroll 4
    for (int i = threadIdx.x & 31; i <= n; i += 32) c += start[i] <= x ? 1 : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xFFFFFFFFu, c, o);
    return c - 1;
}

constexpr int PM_NT = 128;

template <typename T, int D>
__global__ void __launch_bounds__(PM_NT) k_paged_merge(const PagedArgs a, const PagedLine l0, const PagedLine l1) {
    constexpr int V = D / 32;  // channels a lane holds
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int hq = a.hkv * a.G;
    const long long row = (long long)blockIdx.x * (PM_NT / 32) + (threadIdx.x >> 5);
    if (row >= (long long)a.q_tokens * hq) return;
    const int t = (int)(row / hq), hh = (int)(row - (long long)t * hq), head = hh / a.G, g = hh - head * a.G;
    const int s = a.q_start ? last_at_most(a.q_start, a.seqs, t) : t;
    const int grp = a.prefix.rows == 0 ? -1 : a.group_start ? last_at_most(a.group_start, a.prefix.rows, s) : 0;

    float m = -INFINITY, z = 0.0f, acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    // Join a state (maximum, sum, weighted values) whose values are at src, scaled by their sum's unit.
    auto join = [&](float m2, float z2, const float *src) {
        if (z2 == 0.0f) return;  // it summed nothing
        const float mn = fmaxf(m, m2), ms = mn == -INFINITY ? 0.0f : mn;
        const float f = exp2_fast(m - ms), f2 = exp2_fast(m2 - ms);
        z = z * f + z2 * f2;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = acc[i] * f + src[i] * f2;
        m = mn;
    };
#pragma unroll
    for (int x = 0; x < PAGED_LINES; ++x) {
        const PagedLine &l = x ? l1 : l0;
#pragma unroll
        for (int own = 0; own < 2; ++own) {
            if (!(own ? l.with_own : l.with_prefix)) continue;
            const int r = own ? s : grp;
            if (r < 0 || r >= (own ? a.own.rows : a.prefix.rows)) continue;
            const int i = r + (own && l.with_prefix ? a.prefix.rows : 0);
            bool bad = false;
            const PagedSeg sg = paged_segment(a, l, i, bad);
            const int j = t - sg.q0;
            if (j < 0 || j >= sg.qn) continue;
            const int nt = paged_row_tiles(sg, l.tt), mt = j / l.tt;
            const int steps = paged_steps(sg, l, mt);
            if (steps == 0) continue;
            const int per = l.rec[0].x;
            if (per == 0) continue;  // a bad segment: nothing was done
            const int2 before = l.rec[1 + i];
            const int w0 = before.x + head * paged_steps_before(sg, l, nt) + paged_steps_before(sg, l, mt);
            const int u = before.y + head * nt + mt;
            const int in = (j - mt * l.tt) * a.G + g, R = l.tt * a.G;
            const int c0 = w0 / per, c1 = (w0 + steps - 1) / per;
#pragma unroll 4
            for (int c = c0; c <= c1; ++c) {
                const long long at = c + u;
                if (at >= l.slots) break;
                const float2 mz = *reinterpret_cast<const float2 *>(l.part_ml + (at * R + in) * 2);
                float v[V];
                const float *src = l.part_o + at * R * D +
                                   (l.grouped ? (lane * V / 4) * R * 4 + in * 4 + lane * V % 4 : in * D + lane * V);
                if (V == 4) {
                    const float4 q = *reinterpret_cast<const float4 *>(src);
                    v[0] = q.x; v[1] = q.y; v[V - 2] = q.z; v[V - 1] = q.w;
                } else {
                    const float2 q = *reinterpret_cast<const float2 *>(src);
                    v[0] = q.x; v[1] = q.y;
                }
                join(mz.x, mz.y, v);
            }
        }
    }
    if (a.prior_lse) {
        const float pl = a.prior_lse[row];
        if (pl != -INFINITY) {
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = a.prior_o[row * D + lane * V + i];
            join(pl * 1.4426950408889634f, 1.0f, v);
        }
    }
    const float inv = z == 0.0f ? 0.0f : 1.0f / z;
    uint32_t *dst = reinterpret_cast<uint32_t *>(a.o + row * D + lane * V);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) dst[i] = T::pack(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    if (a.lse && lane == 0) a.lse[row] = z == 0.0f ? -INFINITY : (m + log2f(z)) * 0.6931471805599453f;
}

}  // namespace

// The pool as rows of K then V (2 d channels); boxes of 64 channels x box_rows tokens, 128-byte swizzle.
cudaError_t paged_tensor_map(CUtensorMap *map, const void *kv, int dtype, long long rows, int d, int box_rows) {
    const EncodeTiledFn encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)(2 * d), (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)d * 4};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = encode(map, dtype == VERKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                              const_cast<void *>(kv), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t launch_paged(const PagedArgs &a, const PagedLine &l, const CUtensorMap &map, int dtype, int d,
                         cudaStream_t s) {
    const int mt = l.tt * a.G / 16;
#define VERKV_PAGED(TT, DT, DD, MM)                                                            \
    if (dtype == DT && d == DD && mt == MM) {                                                  \
        const size_t smem = PagedLayout<DD, MM>::BYTES;                                        \
        const cudaError_t e = ensure_smem((const void *)k_paged<TT, DD, MM>, smem);            \
        if (e != cudaSuccess) return e;                                                        \
        return launch_pdl(k_paged<TT, DD, MM>, dim3(l.ctas), dim3(PG_NT), smem, s, a, l, map); \
    }
    VERKV_PAGED(PgBf16, VERKV_BF16, 128, 1) VERKV_PAGED(PgBf16, VERKV_BF16, 128, 2)
    VERKV_PAGED(PgBf16, VERKV_BF16, 64, 1) VERKV_PAGED(PgBf16, VERKV_BF16, 64, 2)
    VERKV_PAGED(PgF16, VERKV_F16, 128, 1) VERKV_PAGED(PgF16, VERKV_F16, 128, 2)
    VERKV_PAGED(PgF16, VERKV_F16, 64, 1) VERKV_PAGED(PgF16, VERKV_F16, 64, 2)
#undef VERKV_PAGED
    return cudaErrorInvalidValue;
}

cudaError_t launch_paged_merge(const PagedArgs &a, const PagedLine *lines, int dtype, int d, cudaStream_t s) {
    const long long rows = (long long)a.q_tokens * a.hkv * a.G, blocks = (rows + PM_NT / 32 - 1) / (PM_NT / 32);
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
#define VERKV_PM(TT, DT, DD) \
    if (dtype == DT && d == DD) return launch_pdl(k_paged_merge<TT, DD>, dim3((unsigned)blocks), dim3(PM_NT), 0, s, a, lines[0], lines[1]);
    VERKV_PM(PgBf16, VERKV_BF16, 128) VERKV_PM(PgBf16, VERKV_BF16, 64)
    VERKV_PM(PgF16, VERKV_F16, 128) VERKV_PM(PgF16, VERKV_F16, 64)
#undef VERKV_PM
    return cudaErrorInvalidValue;
}

}  // namespace verkv
