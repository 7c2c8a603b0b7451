// k_paged.cu -- attention over the paged cache for few query rows, and the merge of partial sums.
//
//   o = sum_i 2^(l_i - m) v_i / sum_i 2^(l_i - m),   l_i = q . k_i scale log2(e), m the running maximum
//
// k_paged: 16 or 32 query rows (query tokens x heads of one KV head) against a run of cached tokens.
// Bound by the bytes of K and V: a decode step has q_per_kv rows a sequence, a few flops per byte.
// One warp walks the CTA's run of the line (paged.cuh) and copies 64-token steps of K and V into
// a shared-memory ring by TMA (boxes of one page's tokens x 64 channels, 128-byte swizzle), with a
// unit's queries beside its first step; what a step is (which rows, which tokens, whether a unit
// begins or ends with it) travels with it, so one warp's walk drives the CTA and runs ahead of it.
// Four warps take 16 tokens of a step each (with 32 rows: two take each half of the rows, 32 tokens
// each): S = Q K^T with the rows as the m16 of mma.m16n8k16 (K by ldmatrix), the softmax in registers
// -- each warp keeps its own running maximum and sum and rescales only when some row's maximum rises --
// and P, already in the A operand's layout, times V (ldmatrix, transposed).  A weight is multiplied as
// two 16-bit parts, its rounding and what that leaves out, so that o is off by its own rounding only (one
// part: 1.33 times that, behind 32K tokens in bf16).  That doubles the products of P V, or, where no unit
// has more than 8 rows (a decode step's own tokens), the second parts take the rows that are free.  (256
// sequences behind 32K tokens: products of their own 156 us, free rows 148.)  At a unit's
// end the four warps' states are joined in the step's own shared memory, which nothing reads any more,
// and written as one partial.
//
// Measured (d 128, 8 heads, bf16): 32 sequences of up to 16384 tokens (1.1 GB) 168 us a call, 0.97 of a
// plain copy's bandwidth; 4 behind 128K tokens 94 us, 0.85; 256 sequences of up to 256 tokens 44 us
// (41 without any arithmetic: their copies, of whole steps, and the start bound it); 8 of up to 512
// tokens 10.8 us, two launches.  At d 128 ptxas spills 4 to 16 bytes a thread of its 168 registers.
//
// k_paged_merge: a warp, or with few rows four, per query token and head joins the partials of its
// prefix and its own pages, and the caller's prior state, in a fixed order.
#include <math.h>

#include <algorithm>

#include "paged.cuh"
#include "pivotal_mma.cuh"
#include "verkv_common.cuh"

namespace verkv {

namespace {

constexpr int PG_CONS = 4;                     // consumer warps: 16 tokens of a step each
constexpr int PG_NT = 32 * (PG_CONS + 1);      // and one warp that walks and copies
constexpr int PG_CTAS = 2;                     // an SM

struct StepDesc {
    int flags;       // PG_FIRST | PG_LAST | PG_END
    int valid;       // tokens of the step that some row of the unit sees
    int tok0;        // the step's first token
    int rows;        // real rows
    int q;           // where the unit's queries are: slot of their ring
    int lim0, limd;  // tokens the tile's first query sees, and how many more each next one does
    int slot;        // partial slot, or -1
};
enum { PG_FIRST = 1, PG_LAST = 2, PG_END = 4 };

// RH: halves of 16 rows.
template <int D, int RH>
struct PagedLayout {
    static constexpr int HALVES = D / 64;
    static constexpr int BOX = PAGED_TILE * 128;
    static constexpr int STAGE = 2 * HALVES * BOX;
    static constexpr int NS = D == 128 ? 3 : 6;
    static constexpr int R = 16 * RH;
    static constexpr int QN = RH == 1 ? NS : 2;                  // units whose queries are held
    static constexpr int QROW = 2 * D + (RH == 1 ? 16 : 0);      // (padded where there is room: ldmatrix's banks)
    static constexpr int Q = NS * STAGE;                         // [QN][R][QROW]
    static constexpr int ML = Q + QN * R * QROW;                 // float [4][16][2]
    static constexpr int DESC = ML + PG_CONS * 16 * 2 * 4;
    static constexpr int BARS = (DESC + NS * (int)sizeof(StepDesc) + 7) / 8 * 8;  // full, empty [NS], join
    static constexpr int BYTES = BARS + (2 * NS + 1) * 8 + 8;
    static_assert(PG_CONS * 16 * D * 4 <= STAGE, "a stage holds the four warps' sums");
    static_assert((BYTES + 1024) * PG_CTAS <= 228 * 1024, "CTAs an SM");
};

// A piece of the walk, and the ids of its first 32 pages (lane i: page ids0 + i).
struct Piece {
    const int32_t *row;
    int t0, t1, vis, head, q0, rows, lim0, limd, slot, ids0, ids;
};

// The ids of pages p .. p + 31 of a sequence that is seen up to `vis`, one a lane.
__device__ __forceinline__ int page_ids(const PagedArgs &a, const int32_t *row, int p, int vis) {
    p += threadIdx.x & 31;
    int id = 0;
    if (p <= (vis - 1) >> a.page_shift) {
        id = row[p];
        if (id < 0 || id >= a.num_pages) {
            raise_error(a.err, ERR_PAGE);
            id = 0;
        }
    }
    return id;
}

// SPARE: no unit has more than 8 rows.  Rows 8 .. 15 of the products then take what rounding the weights
// of rows 0 .. 7 has left out, in place of products of their own.
template <typename T, int D, int RH, bool SPARE>
__global__ void __launch_bounds__(PG_NT, PG_CTAS)
    k_paged(const __grid_constant__ PagedArgs a, const __grid_constant__ PagedLine l, const int second,
            const __grid_constant__ CUtensorMap map) {
    using LY = PagedLayout<D, RH>;
    constexpr int KS = D / 16, NS = LY::NS, R = LY::R;
    extern __shared__ __align__(1024) unsigned char pg_smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(pg_smem + LY::BARS), *empty = full + NS, *join = empty + NS;
    volatile int *abort = reinterpret_cast<volatile int *>(join + 1);
    StepDesc *desc = reinterpret_cast<StepDesc *>(pg_smem + LY::DESC);
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
    if (warp == PG_CONS) {
        if (lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map)) : "memory");
        // Before the CTA's barrier: no wait's limit counts what the kernels ahead still take.
        paged_begin(a, second != 0);
    }
    __syncthreads();

    if (warp == PG_CONS) {
        const int box = min(1 << a.page_shift, PAGED_TILE);  // tokens of a page in one step
        PagedWalk<false> wk;
        // (the queries' place holds nothing yet)
        wk.start(a, l, blockIdx.x, reinterpret_cast<int2 *>(pg_smem + LY::Q), LY::QN * R * LY::QROW / 8);
        fence_proxy_async_smem();  // these accesses before the queries' copies to the same place
        __syncwarp();
        // The walk is one piece ahead of the copies, so that a piece's page ids are there when its
        // first step is.
        auto fetch = [&](Piece &p) -> bool {
            if (!wk.next(a, l, blockIdx.x)) return false;
            const PagedLevel &lv = a.level[wk.s.own ? 1 : 0];
            const int first = wk.m << l.tt_shift;
            p.row = lv.table + (long long)wk.s.row * lv.stride;
            p.t0 = wk.t0;
            p.t1 = wk.t1;
            p.vis = paged_visible(wk.s, l, wk.m);
            p.head = wk.head;
            p.q0 = wk.s.q0 + first;
            p.rows = min(1 << l.tt_shift, wk.s.qn - first) << a.g_shift;
            p.lim0 = wk.s.own ? wk.s.len - (wk.s.qn - 1 - first) : wk.s.len;
            p.limd = wk.s.own ? 1 : 0;
            p.slot = wk.slot < l.slots ? wk.slot : -1;
            p.ids0 = p.t0 * PAGED_TILE >> a.page_shift;
            p.ids = page_ids(a, p.row, p.ids0, p.vis);
            return true;
        };
        Piece cur = {}, nxt = {};
        bool have = true, go = true;
        int j = 0, np = 0;      // steps and pieces so far
        int begun[2] = {-1, -1};  // first steps of the last two pieces
        while (have && go) {
            have = fetch(nxt);
#pragma unroll 1
            for (int t = cur.t0; t < cur.t1; ++t, ++j) {
                const int k = j % NS;
                if (j >= NS) go = __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(&empty[k], (uint32_t)((j / NS - 1) & 1), abort, a.wait_ns));
                if (!go) break;
                const int tok0 = t * PAGED_TILE, valid = min(PAGED_TILE, cur.vis - tok0);
                const int pages = (valid + box - 1) / box, p0 = tok0 >> a.page_shift;
                if (p0 + pages > cur.ids0 + 32) {
                    cur.ids0 = p0;
                    cur.ids = page_ids(a, cur.row, p0, cur.vis);
                }
                const bool first = t == cur.t0;
                if (first && LY::QN < NS) {
                    // The queries' slot: the piece before the last one has begun to be worked on.  (Of a step
                    // NS back that is known, and its barrier may be phases ahead.)
                    const int b = begun[0];
                    if (b >= 0 && b > j - NS) go = __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(&empty[b % NS], (uint32_t)((b / NS) & 1), abort, a.wait_ns));
                    if (!go) break;
                    begun[0] = begun[1];
                    begun[1] = j;
                }
                if (lane == 0) {
                    StepDesc s;
                    s.flags = (first ? PG_FIRST : 0) | (t + 1 == cur.t1 ? PG_LAST : 0);
                    s.valid = valid;
                    s.tok0 = tok0;
                    s.rows = cur.rows;
                    s.q = np % LY::QN;
                    s.lim0 = cur.lim0;
                    s.limd = cur.limd;
                    s.slot = cur.slot;
                    if (s.slot < 0) raise_error(a.err, ERR_PAGE);
                    desc[k] = s;
                    mbar_expect_tx(&full[k], (uint32_t)(pages * box * 4 * D + (first ? cur.rows * 2 * D : 0)));
                }
                __syncwarp();
                const int id = __shfl_sync(0xFFFFFFFFu, cur.ids, (p0 + lane - cur.ids0) & 31);
                const bool stalled = a.stall && blockIdx.x == 0 && j == 0;
                if (lane < pages && !stalled) {
                    // a page of more than one step is read at the step's offset in it
                    const int y = (((id * a.hkv + cur.head) << a.page_shift) + ((tok0 + lane * box) & ((1 << a.page_shift) - 1)));
                    unsigned char *st = pg_smem + (size_t)k * LY::STAGE + lane * box * 128;
#pragma unroll
                    for (int b = 0; b < 2 * LY::HALVES; ++b) tma_load_2d(st + b * LY::BOX, &map, b * 64, y, &full[k]);
                }
                if (first && lane < cur.rows && !stalled) {
                    const int jj = lane >> a.g_shift, hh = (cur.head << a.g_shift) + lane - (jj << a.g_shift);
                    bulk_g2s(pg_smem + LY::Q + (np % LY::QN * R + lane) * LY::QROW, a.q + (cur.q0 + jj) * a.q_ts + hh * a.q_hs, 2 * D, &full[k]);
                }
                __syncwarp();
            }
            if (cur.t0 < cur.t1) ++np;
            cur = nxt;
        }
        if (go) {  // tell the consumers that the run is over
            const int k = j % NS;
            if (j >= NS) go = __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(&empty[k], (uint32_t)((j / NS - 1) & 1), abort, a.wait_ns));
            if (go && lane == 0) {
                desc[k].flags = PG_END;
                mbar_arrive(&full[k]);
            }
        }
        if (lane == 0) {
            if (!go) {  // a wait ran out
                *abort = 1;
                raise_error(a.err, ERR_TIMEOUT);
            }
            // The copies in flight land before the CTA gives its shared memory back, also where another
            // warp's wait ran out after the last of them was issued.  They are of the last NS steps; the
            // place of the first of those holds the end of the run by now, if that has been told.
            for (int i = max(0, j - NS + (go ? 1 : 0)); i < j; ++i) mbar_wait_bounded(&full[i % NS], (uint32_t)((i / NS) & 1), a.wait_ns);
        }
        __syncwarp();
    } else {
        const int g = lane >> 2, t = lane & 3, mi = lane >> 3, ri = lane & 7;
        const int rb = RH == 1 ? 0 : (warp >> 1) * 16;            // this warp's rows
        const int wt = RH == 1 ? warp * 16 : (warp & 1) * 32;     // and tokens of a step
        constexpr int NW = PG_CONS / RH;                           // warps with the same rows
        uint32_t qf[KS][4];
        float o[D / 8][4], mx[2], sum[2];
        int lim[2];
        int joins = 0;
        auto cons_sync = [&]() -> bool {
            __syncwarp();
            if (lane == 0) mbar_arrive(join);
            const bool ok = mbar_wait_or_abort(join, (uint32_t)(joins & 1), abort, a.wait_ns);
            ++joins;
            if (__all_sync(0xFFFFFFFFu, ok)) return true;
            if (lane == 0) {
                *abort = 1;
                raise_error(a.err, ERR_TIMEOUT);
            }
            return false;
        };
        for (int j = 0;; ++j) {
            const int k = j % NS;
            const bool ok = mbar_wait_or_abort(&full[k], (uint32_t)((j / NS) & 1), abort, a.wait_ns);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                if (lane == 0) {
                    *abort = 1;
                    raise_error(a.err, ERR_TIMEOUT);
                }
                break;
            }
            const StepDesc s = desc[k];
            if (s.flags & PG_END) break;
            unsigned char *st = pg_smem + (size_t)k * LY::STAGE;
            if (s.flags & PG_FIRST) {
                const uint32_t qb = smem_addr(pg_smem + LY::Q) + (s.q * R + rb + (mi & 1) * 8 + ri) * LY::QROW + (mi >> 1) * 16;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) ldsm_x4(qf[ks], qb + ks * 32);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = rb + g + 8 * e;
                    lim[e] = r < s.rows ? s.lim0 + s.limd * (r >> a.g_shift) : 0;
                    mx[e] = -INFINITY;
                    sum[e] = 0.0f;
                }
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
            }
#pragma unroll 1
            for (int w0 = wt; w0 < wt + 16 * RH; w0 += 16) {
                if (w0 >= s.valid || rb >= s.rows) break;
                const uint32_t kb = smem_addr(st), vb = kb + LY::HALVES * LY::BOX;
                if (w0 + 16 > s.valid) {
                    // V rows that nothing sees may hold anything, NaN too: a weight of 0 would keep it
#pragma unroll 1
                    for (int r = s.valid; r < w0 + 16; ++r)
                        if (lane < 8 * LY::HALVES)
                            *reinterpret_cast<uint4 *>(st + (LY::HALVES + (lane >> 3)) * LY::BOX + r * 128 + (lane & 7) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                    __syncwarp();
                }
                float sc[2][4] = {}, sd[2][4] = {};  // even and odd k-steps: shorter chains
                {
                    const int r = w0 + (mi >> 1) * 8 + ri;
                    uint32_t b[KS][4];
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
                        ldsm_x4(b[ks], kb + (ks / 4) * LY::BOX + r * 128 + ((((ks % 4) * 2 + (mi & 1)) ^ (r & 7)) << 4));
#pragma unroll
                    for (int ks = 0; ks < KS; ks += 2) {
                        T::mma(sc[0], qf[ks], b[ks][0], b[ks][1]);
                        T::mma(sc[1], qf[ks], b[ks][2], b[ks][3]);
                        T::mma(sd[0], qf[ks + 1], b[ks + 1][0], b[ks + 1][1]);
                        T::mma(sd[1], qf[ks + 1], b[ks + 1][2], b[ks + 1][3]);
                    }
                }
                float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int tok = s.tok0 + w0 + nt * 8 + 2 * t + (e & 1);
                        float x = (sc[nt][e] + sd[nt][e]) * a.scale_log2;
                        x = tok < lim[e >> 1] ? x : -INFINITY;
                        sc[nt][e] = x;
                        top[e >> 1] = fmaxf(top[e >> 1], x);
                    }
                bool rises = false;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], 1));
                    top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], 2)) - T::SHIFT;
                    rises |= top[e] > mx[e];
                }
                if (__any_sync(0xFFFFFFFFu, rises)) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float m = fmaxf(mx[e], top[e]);
                        f[e] = m == mx[e] ? 1.0f : exp2_fast(mx[e] - m);  // (-inf: nothing summed yet)
                        mx[e] = m;
                        sum[e] *= f[e];
                    }
                    if (SPARE) f[1] = f[0];
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[n][0] *= f[0];
                        o[n][1] *= f[0];
                        o[n][2] *= f[1];
                        o[n][3] *= f[1];
                    }
                }
                uint32_t pf[4], pr[4];  // the weights in 16 bits, and what that leaves out
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float m = mx[e] == -INFINITY ? 0.0f : mx[e];  // a row that sees nothing so far
                    float p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        p[i] = exp2_fast(sc[i >> 1][2 * e + (i & 1)] - m);
                        sum[e] += p[i];
                    }
                    pf[e] = T::pack(p[0], p[1]);
                    pf[2 + e] = T::pack(p[2], p[3]);
                    pr[e] = pack_rest<T>(pf[e], p[0], p[1]);
                    pr[2 + e] = pack_rest<T>(pf[2 + e], p[2], p[3]);
                }
                if (SPARE) {
                    pf[1] = pr[0];
                    pf[3] = pr[2];
                }
                const int r = w0 + (mi & 1) * 8 + ri;
#pragma unroll
                for (int c0 = 0; c0 < KS; c0 += 4) {
                    uint32_t b[4][4];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        ldsm_x4_t(b[c], vb + (c0 / 4) * LY::BOX + r * 128 + (((c * 2 + (mi >> 1)) ^ (r & 7)) << 4));
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        T::mma(o[2 * (c0 + c)], pf, b[c][0], b[c][1]);
                        T::mma(o[2 * (c0 + c) + 1], pf, b[c][2], b[c][3]);
                    }
#pragma unroll
                    for (int c = 0; c < 4 && !SPARE; ++c) {
                        T::mma(o[2 * (c0 + c)], pr, b[c][0], b[c][1]);
                        T::mma(o[2 * (c0 + c) + 1], pr, b[c][2], b[c][3]);
                    }
                }
            }
            if (s.flags & PG_LAST) {
                // Join the four warps' states: each scales its sums to the common maximum and lays
                // them in the slot, and all threads add the four and write the partial.
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 1);
                    sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 2);
                    if (t == 0) *reinterpret_cast<float2 *>(ml + (warp * 16 + g + 8 * e) * 2) = make_float2(mx[e], sum[e]);
                }
#pragma unroll
                for (int n = 0; n < D / 8 && SPARE; ++n) {
                    o[n][0] += o[n][2];
                    o[n][1] += o[n][3];
                }
                if (!cons_sync()) break;  // and no warp reads the slot's K and V any more
                float *buf = reinterpret_cast<float *>(st);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = g + 8 * e;
                    float m = -INFINITY, z = 0.0f;
                    const float *mz = ml + (rb / 16 * NW * 16 + r) * 2;  // of the warps with these rows
#pragma unroll
                    for (int w = 0; w < NW; ++w) m = fmaxf(m, mz[w * 32]);
                    const float ms = m == -INFINITY ? 0.0f : m;
#pragma unroll
                    for (int w = 0; w < NW; ++w) z += mz[w * 32 + 1] * exp2_fast(mz[w * 32] - ms);
                    if (rb + r < s.rows) {
                        const float f = exp2_fast(mx[e] - ms);
#pragma unroll
                        for (int n = 0; n < D / 8; ++n)
                            *reinterpret_cast<float2 *>(buf + (warp * 16 + r) * D + ((n * 8 + 2 * t) ^ (g << 3))) =
                                make_float2(o[n][2 * e] * f, o[n][2 * e + 1] * f);
                        if (t == 0 && warp % NW == 0 && s.slot >= 0)
                            *reinterpret_cast<float2 *>(l.part_ml + ((long long)s.slot * R + rb + r) * 2) = make_float2(m, z);
                    }
                }
                if (!cons_sync()) break;
                if (s.slot >= 0) {
                    float *po = l.part_o + (long long)s.slot * R * D;
#pragma unroll 1
                    for (int x = tid * 4; x < s.rows * D; x += PG_CONS * 32 * 4) {
                        // as laid: 8 channels' groups turned by the row, and the half's first warp
                        const int y = (x ^ (((x / D) & 7) << 3)) + x / (16 * D) * (NW - 1) * 16 * D;
                        float4 v = *reinterpret_cast<const float4 *>(buf + y);
#pragma unroll
                        for (int w = 1; w < NW; ++w) {
                            const float4 u = *reinterpret_cast<const float4 *>(buf + w * 16 * D + y);
                            v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
                        }
                        *reinterpret_cast<float4 *>(po + x) = v;
                    }
                }
            }
            fence_proxy_async_smem();  // generic accesses before the slot's next copy
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[k]);
        }
        pdl_wait();  // the launch before this one is done when this one is
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------------------------
// The last index i of 0 .. n with start[i] <= x (start ascending; -1: none).  The whole warp: 32 probes a
// turn, so that 65536 sequences take four.  (Starts out of order end at some index of the range.)
__device__ __forceinline__ int last_at_most(const int32_t *start, int n, int x) {
    const int lane = threadIdx.x & 31;
    int at = -1, left = n + 1;  // start[at] <= x; how many behind it are left to look at
#pragma unroll 1
    while (left > 0) {
        const int step = (left + 31) >> 5;
        const int c = __popc(__ballot_sync(0xFFFFFFFFu, lane * step < left && start[at + 1 + lane * step] <= x));
        if (c == 0) break;
        at += 1 + (c - 1) * step;
        left = min(step, left - (c - 1) * step) - 1;
    }
    return at;
}

constexpr int PM_NT = 128;

// start[0 .. n] ascends from 0 to `end`, or the call is reported; all threads of the grid, whose number may
// pass 32 bits.
__device__ __forceinline__ void check_starts(const PagedArgs &a, const int32_t *start, int n, int end) {
    for (long long i = (long long)blockIdx.x * PM_NT + threadIdx.x; i <= n; i += (long long)gridDim.x * PM_NT) {
        const int x = start[i];
        if (i == n ? x != end : x > start[i + 1] || (i == 0 && x != 0)) raise_error(a.err, ERR_PAGE);
    }
}
// (A call: most launches have nothing of the kind, and pay for the code they pass.)
static __device__ __noinline__ void check_unseen(const PagedArgs &a) {
    if (a.check_q_start) check_starts(a, a.q_start, a.seqs, a.q_tokens);
    if (a.check_group_start) check_starts(a, a.group_start, a.zero_rows[0], a.seqs);
    for (int x = 0; x < 2; ++x)
        for (long long i = (long long)blockIdx.x * PM_NT + threadIdx.x; i < a.zero_rows[x]; i += (long long)gridDim.x * PM_NT)
            if (a.zero_length[x][i] != 0) raise_error(a.err, ERR_PAGE);
}

template <typename T, int D, int WPR>
__global__ void __launch_bounds__(PM_NT) k_paged_merge(const __grid_constant__ PagedArgs a, const __grid_constant__ PagedLines lines) {
    constexpr int V = D / 32;  // channels a lane holds
    const int lane = threadIdx.x & 31;
    const int hq = a.hkv << a.g_shift;
    __shared__ float states[PM_NT / 32][D + 2];
    pdl_wait();
    pdl_trigger();
    if (a.ready && blockIdx.x == 0 && threadIdx.x == 0) *a.ready = 0ull;  // (see paged_begin)
    if (a.unseen) check_unseen(a);
    const int warp = threadIdx.x >> 5, wi = warp % WPR;  // of the row's warps
    const long long row = (long long)blockIdx.x * (PM_NT / 32 / WPR) + warp / WPR;
    if (row >= (long long)a.q_tokens * hq) return;
    const int t = (int)(row / hq), hh = (int)(row - (long long)t * hq), head = hh >> a.g_shift, g = hh - (head << a.g_shift);
    const int s = a.q_start ? last_at_most(a.q_start, a.seqs, t) : t;

    // Where the row's partials are: of its prefix, then of its own pages.
    const float *po[2] = {}, *pm[2] = {};
    int count[2] = {0, 0}, rows[2] = {0, 0};  // a slot's rows
    bool grouped[2] = {false, false};
#pragma unroll
    for (int own = 0; own < 2; ++own) {
        const int at = lines.l[1].with[own] ? 1 : 0;
        const PagedLine &l = lines.l[at];
        if (!l.with[own]) continue;
        const int r = own ? s : a.group_start ? last_at_most(a.group_start, a.level[0].rows, s) : 0;
        if (r < 0 || r >= a.level[own].rows) continue;
        const int i = r + (own && l.with[0] ? a.level[0].rows : 0);
        const int per = l.rec[0].x, room = l.rec[0].y;
        const int2 before = l.rec[1 + i];
        bool bad = false;
        const PagedSeg sg = paged_segment(a, l, i, bad);
        const int j = t - sg.q0;
        if (j < 0 || j >= sg.qn || per <= 0) continue;  // (per 0: a bad segment, nothing was done)
        const int mt = j >> l.tt_shift, steps = paged_steps(sg, l, mt);
        if (steps == 0) continue;
        const int w0 = before.x + paged_steps_before(sg, l, mt, room) * a.hkv + head * (room ? room : steps);
        const int c0 = (unsigned)w0 / (unsigned)per, c1 = (unsigned)(w0 + steps - 1) / (unsigned)per;
        const int in = ((j - (mt << l.tt_shift)) << a.g_shift) + g;
        const int slot = clampi(c0 + before.y + mt * a.hkv + head, 0, l.slots - 1);
        count[own] = clampi(c1 - c0 + 1, 0, l.slots - slot);
        rows[own] = 1 << (l.tt_shift + a.g_shift);
        grouped[own] = l.grouped != 0;
        po[own] = l.part_o + (long long)slot * rows[own] * D + (l.grouped ? (in >> 2) * (D * 4) + (in & 3) * 4 : in * D);
        pm[own] = l.part_ml + ((long long)slot * rows[own] + in) * 2;
    }
    float prior = -INFINITY;
    if (a.prior_lse) prior = a.prior_lse[row] * 1.4426950408889634f;

    // 32 partials a turn, a lane each: its state, and where its values are.  A partial whose sum is 0
    // summed nothing, and its values are not used.
    const int n = count[0] + count[1];
    const int turns = (n + WPR - 1 - wi) / WPR;  // this warp's: every WPR-th
    const int flat = lane * V, quad = (lane * V / 4) * 16 + lane * V % 4;  // this lane's channels in either order
    float m = wi == 0 ? prior : -INFINITY, z = 0.0f, acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    if (m != -INFINITY) {
        z = lane == 0 ? 1.0f : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = a.prior_o[row * D + flat + i];
    }
#pragma unroll 1
    for (int x0 = 0; x0 < turns; x0 += 32) {
        const int x = (x0 + lane) * WPR + wi, v = x < count[0] ? 0 : 1, k = x - (v ? count[0] : 0);
        float2 mine = make_float2(-INFINITY, 0.0f);
        unsigned long long at = 0;
        if (x < n) {
            mine = *reinterpret_cast<const float2 *>((v ? pm[1] : pm[0]) + (long long)k * (v ? rows[1] : rows[0]) * 2);
            at = reinterpret_cast<unsigned long long>((v ? po[1] : po[0]) + (long long)k * (v ? rows[1] : rows[0]) * D);
        }
        const unsigned in_quads = __ballot_sync(0xFFFFFFFFu, v ? grouped[1] : grouped[0]);
        const float mn = fmaxf(m, warp_max(mine.x)), ms = mn == -INFINITY ? 0.0f : mn;
        const float f = exp2_fast(m - ms), w = exp2_fast(mine.x - ms);
        z = z * f + (mine.y == 0.0f ? 0.0f : mine.y * w);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] *= f;
        m = mn;
        const unsigned some = __ballot_sync(0xFFFFFFFFu, mine.y != 0.0f);
        const int c = min(32, turns - x0);
#pragma unroll 4
        for (int y = 0; y < c; ++y) {
            const float wy = __shfl_sync(0xFFFFFFFFu, w, y);
            const float *src = reinterpret_cast<const float *>(__shfl_sync(0xFFFFFFFFu, at, y)) + ((in_quads >> y & 1) ? quad : flat);
            float u[V];
            if (V == 4) {
                const float4 q = *reinterpret_cast<const float4 *>(src);
                u[0] = q.x; u[1] = q.y; u[V - 2] = q.z; u[V - 1] = q.w;
            } else {
                const float2 q = *reinterpret_cast<const float2 *>(src);
                u[0] = q.x; u[1] = q.y;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = (some >> y & 1) ? fmaf(u[i], wy, acc[i]) : acc[i];
        }
    }
    z = warp_sum(z);
    if (WPR > 1) {
        // The row's warps join in shared memory, in their order.
        if (lane == 0) {
            states[warp][D] = m;
            states[warp][D + 1] = z;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) states[warp][flat + i] = acc[i];
        __syncthreads();
        float mn = -INFINITY;
#pragma unroll
        for (int w = 0; w < WPR; ++w) mn = fmaxf(mn, states[w][D]);
        const float ms = mn == -INFINITY ? 0.0f : mn;
        m = mn;
        z = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) {
            const float f = exp2_fast(states[w][D] - ms), zw = states[w][D + 1];
            if (zw == 0.0f) continue;
            z = fmaf(zw, f, z);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(states[w][flat + i], f, acc[i]);
        }
    }
    if (wi) return;
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

cudaError_t launch_paged(const PagedArgs &a, const PagedLine &l, const CUtensorMap &map, bool second, int dtype, int d,
                         cudaStream_t s) {
    const int rows = 1 << (l.tt_shift + a.g_shift);
#define VERKV_PAGED(TT, DT, DD, RR, SP)                                                    \
    if (dtype == DT && d == DD && rows == 16 * RR && (l.spare != 0) == SP) {               \
        const size_t smem = PagedLayout<DD, RR>::BYTES;                                    \
        const cudaError_t e = ensure_smem((const void *)k_paged<TT, DD, RR, SP>, smem);    \
        if (e != cudaSuccess) return e;                                                    \
        return launch_pdl(k_paged<TT, DD, RR, SP>, dim3(l.ctas), dim3(PG_NT), smem, s, a, l, second ? 1 : 0, map); \
    }
#define VERKV_PAGED_D(TT, DT, DD) VERKV_PAGED(TT, DT, DD, 1, true) VERKV_PAGED(TT, DT, DD, 1, false) VERKV_PAGED(TT, DT, DD, 2, false)
    VERKV_PAGED_D(PgBf16, VERKV_BF16, 128) VERKV_PAGED_D(PgBf16, VERKV_BF16, 64)
    VERKV_PAGED_D(PgF16, VERKV_F16, 128) VERKV_PAGED_D(PgF16, VERKV_F16, 64)
#undef VERKV_PAGED_D
#undef VERKV_PAGED
    return cudaErrorInvalidValue;
}

cudaError_t launch_paged_merge(const PagedArgs &a, const PagedLines &lines, int dtype, int d, cudaStream_t s) {
    const long long rows = (long long)a.q_tokens * (a.hkv << a.g_shift);
    // Few rows with many partials each (128 rows with 39 each, 128K tokens: 101.6 -> 94.3 us a call) have warps to spare.
    double partials = 0.0;  // of a row, about
    for (const PagedLine &l : lines.l)
        if (l.units > 0) partials = std::max(partials, (double)l.ctas / l.units);
    const int wpr = rows <= 1024 && partials >= 7.0 ? 4 : 1;
    const long long blocks = (rows * wpr + PM_NT / 32 - 1) / (PM_NT / 32);
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
#define VERKV_PM(TT, DT, DD)                                                                                               \
    if (dtype == DT && d == DD) {                                                                                          \
        if (wpr == 4) return launch_pdl(k_paged_merge<TT, DD, 4>, dim3((unsigned)blocks), dim3(PM_NT), 0, s, a, lines);    \
        return launch_pdl(k_paged_merge<TT, DD, 1>, dim3((unsigned)blocks), dim3(PM_NT), 0, s, a, lines);                  \
    }
    VERKV_PM(PgBf16, VERKV_BF16, 128) VERKV_PM(PgBf16, VERKV_BF16, 64)
    VERKV_PM(PgF16, VERKV_F16, 128) VERKV_PM(PgF16, VERKV_F16, 64)
#undef VERKV_PM
    return cudaErrorInvalidValue;
}

}  // namespace verkv
