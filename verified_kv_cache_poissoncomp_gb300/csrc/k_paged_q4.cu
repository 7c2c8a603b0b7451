// k_paged_q4.cu -- attention over pages of 4-bit codes, and a pool's values.
//
//   o = sum_i 2^(l_i - m) v_i / sum_i 2^(l_i - m),   l_i = q . k_i scale log2(e),   k, v = floor + code step
//
// k_paged_q4: units of up to 8, 16 or 32 query rows (query tokens x heads of one KV head) against a run of
// cached tokens, on the line of paged.cuh; the partials are joined by k_paged_merge.  A step is 64 tokens,
// a block of 16 for each of the CTA's four warps.  A warp has a ring of blocks of its own, each brought by
// one bulk copy (a block is one piece of memory), so that warps wait for nothing but their copies until
// the unit's end.
//
//     S = K Q^T      16 tokens x 8 rows, exact codes (q4.cuh), steps and floors after it in float32
//     P = 2^(S c - ref), rounded to binary16 and turned into a B operand by a transpose of 8 x 8 tiles
//         (movmatrix); times the step of each group of V's channels, rounded again: an operand a group.  Of
//         bfloat16 results that is all: a weight is off by up to 2^-11, and 2^-11 more where it meets codes, little
//         beside the result's own 2^-8 (1.66e-3 of o's root mean square, 1.65e-3 without).  Binary16 results
//         would show it (5.5e-4 for 2.1e-4): there what either rounding leaves out goes along in an operand of
//         its own (REST), and all codes are 16 n (q4.cuh; with n, results near 0 were off by 1.4e-5 for 2e-6 of
//         values of 1).  The sum that they are divided by is of the float32 weights
//     O += V^T P     channels x rows, exact codes
//     B += F^T P     groups x rows: the floors' part, the same for all channels of a group
//
// `ref` of a row is its running maximum at some step, and is raised, with O scaled, only where the
// maximum has risen by more than SLACK since: a vote a block, and shuffles in the rare other case.  P is below
// 2^14, the largest one so far 2^8 at least, and the last bit of a binary16 2^-24.  Steps meet it as step 2^k, with a k for each
// group of V's channels that makes the largest one so far 1/2 to 2 (k <= 15, all that one product makes of binary16:
// a group whose steps are all below 2^-16 stays below 1/2).  Where larger steps come k is lowered, with O scaled, by
// the same vote.  So products are below 2^15, and as many bits of them remain in small values as in large ones: a
// rounding of one loses 2^-32 at most of the row's largest weight times its group's largest step, for each of up to 15
// of a code.  (With steps as they are, codes of values of 0.01 behind a token of 2^20 times the others' weight were lost.)
//
// Bound: with few rows the bytes and, beside them, each CTA's start, end and changes of unit, where its ring stands
// empty: 32 sequences of up to 16384 tokens (346 MB) 82 us, 0.62 of a plain copy's rate (over 16-bit pages 0.97).  With
// many rows the dependences within a block -- codes to products to weights to products -- with the few warps that
// the sums' registers leave: of 32 rows at d = 128 8 warps an SM issue in a quarter of the slots, and 32 rows behind 32K
// tokens take 48 us, 128 rows 116.  Each unit spreads its codes again, so that from about 32 rows of a sequence or prefix on 16-bit
// pages take less time.  Five CTAs an SM, rings of three blocks and two blocks at a time gained nothing, nor
// did the groups' 2^k in shared memory.
#include <math.h>

#include <algorithm>

#include "paged.cuh"
#include "pivotal_mma.cuh"
#include "q4.cuh"
#include "verkv_common.cuh"

namespace verkv {

namespace {

constexpr int PQ_WARPS = 4, PQ_NT = 32 * PQ_WARPS;
constexpr int PQ_NS = 4;  // blocks of a warp's ring
constexpr float PQ_ROOM = 14.0f;  // log2 that a weight may be above ref
constexpr float PQ_SLACK = 6.0f;  // log2 that a maximum may rise by until ref does
constexpr uint32_t PQ_SCALE = 0x78007800u;  // 2^15, twice: of a group before its first steps
constexpr float PQ_NONE = -1e30f;                // ref of a row that has seen nothing

struct Q4Piece {
    const int32_t *row;  // its page ids
    int steps;           // 0: the run is over
    int t0, vis, head, q0, rows, lim0, limd, slot;
};

template <int D, int NT>
struct Q4Layout {
    static constexpr int BLOCK = Q4<D>::BLOCK;
    static constexpr int RING = 0;  // [PQ_WARPS][PQ_NS][BLOCK]; at a unit's end [PQ_WARPS][8 NT][D] float
    static constexpr int RING_BYTES = PQ_WARPS * PQ_NS * BLOCK;
    static constexpr int JOIN_BYTES = PQ_WARPS * 8 * NT * D * 4;
    static constexpr int ML = RING_BYTES > JOIN_BYTES ? RING_BYTES : JOIN_BYTES;  // float [PQ_WARPS][8 NT][2]
    static constexpr int PIECE = ML + PQ_WARPS * 8 * NT * 2 * 4;
    static constexpr int WALK = (PIECE + 2 * (int)sizeof(Q4Piece) + 15) / 16 * 16;  // warp 0's walk between pieces
    static constexpr int Q = WALK + ((int)sizeof(PagedWalk<false>) + 15) / 16 * 16;  // the queries' B operands, uint4 [NT][D / 32][32]
    static constexpr int UNITS = Q + NT * (D / 32) * 512;                            // and what goes with them: uint2 [NT][32], float [NT][8]
    static constexpr int BARS = UNITS + NT * (256 + 32);
    static constexpr int BYTES = BARS + PQ_WARPS * PQ_NS * 8 + 8;
};

__device__ __forceinline__ uint32_t mul_f16(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t fma_f16(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t max_f16(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

template <typename T>
struct Parts;
template <>
struct Parts<PgBf16> {
    static constexpr bool REST = false;
};
template <>
struct Parts<PgF16> {
    static constexpr bool REST = true;
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(PQ_NT, NT == 1 ? 4 : NT == 2 ? 3 : 2)
    k_paged_q4(const __grid_constant__ PagedArgs a, const __grid_constant__ PagedLine l, const int second) {
    using F = Q4<D>;
    using LY = Q4Layout<D, NT>;
    constexpr int R = 8 * NT, NG = F::GROUPS;
    constexpr bool REST = Parts<T>::REST;
    typedef typename Q4Vec<D>::Key KeyVec;
    typedef typename Q4Vec<D>::Value ValueVec;
    extern __shared__ __align__(128) unsigned char pq_smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(pq_smem + LY::BARS);
    volatile int *abort = reinterpret_cast<volatile int *>(bars + PQ_WARPS * PQ_NS);
    volatile Q4Piece *pieces = reinterpret_cast<volatile Q4Piece *>(pq_smem + LY::PIECE);  // [2]: this one and the next
    float *ml = reinterpret_cast<float *>(pq_smem + LY::ML), *units_at = reinterpret_cast<float *>(pq_smem + LY::UNITS + NT * 256);
    uint4 *q_at = reinterpret_cast<uint4 *>(pq_smem + LY::Q);
    uint2 *sums_at = reinterpret_cast<uint2 *>(pq_smem + LY::UNITS);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    if (tid == 0) {
        for (int k = 0; k < PQ_WARPS * PQ_NS; ++k) mbar_init(&bars[k], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *abort = 0;
    }
    // The walk's state is in registers only while warp 0 walks.
    PagedWalk<false> *walk = reinterpret_cast<PagedWalk<false> *>(pq_smem + LY::WALK);
    auto next_piece = [&](PagedWalk<false> wk, volatile Q4Piece *p) {
        const bool more = wk.next(a, l, blockIdx.x);
        if (lane == 0) {
            if (more) {
                const PagedLevel &lv = a.level[wk.s.own ? 1 : 0];
                const int first = wk.m << l.tt_shift;
                p->row = lv.table + (long long)wk.s.row * lv.stride;
                p->t0 = wk.t0;
                p->vis = paged_visible(wk.s, l, wk.m);
                p->head = wk.head;
                p->q0 = wk.s.q0 + first;
                p->rows = min(1 << l.tt_shift, wk.s.qn - first) << a.g_shift;
                p->lim0 = wk.s.own ? wk.s.len - (wk.s.qn - 1 - first) : wk.s.len;
                p->limd = wk.s.own ? 1 : 0;
                p->slot = wk.slot < l.slots ? wk.slot : -1;
                if (wk.slot >= l.slots) raise_error(a.err, ERR_PAGE);
            }
            p->steps = more ? wk.t1 - wk.t0 : 0;
            *walk = wk;
        }
        __syncwarp();
    };
    if (warp == 0) {
        // The other warps touch the caller's data only behind a barrier.
        paged_begin(a, second != 0);
        // (the ring holds nothing yet)
        PagedWalk<false> wk;
        wk.start(a, l, blockIdx.x, reinterpret_cast<int2 *>(pq_smem), LY::RING_BYTES / 8);
        fence_proxy_async_smem();  // these accesses before the copies to the same place
        next_piece(wk, &pieces[0]);
    }
    unsigned char *ring = pq_smem + warp * PQ_NS * F::BLOCK;
    uint64_t *full = bars + warp * PQ_NS;
    const unsigned char *pool = reinterpret_cast<const unsigned char *>(a.pages);
    const uint32_t sign = a.scale_log2 < 0.0f ? 0x80008000u : 0u;  // a negative scale turns Q round
    const float c = fabsf(a.scale_log2);
    // Tokens 2 t and 2 t + 1 (and 8 more) are this lane's columns of V's product; odd lanes read them in
    // the other order, so that fewer of a load's rows are in the same banks.
    const int odd = t & 1;
    const uint32_t byte0 = odd ? BYTE0_TURNED : BYTE0;

    int j = 0;  // blocks this warp has taken, of all units
    bool ok = true;
#pragma unroll 1
    for (int np = 0;; ++np) {
        __syncthreads();
        if (np == 0 && second) asm volatile("fence.proxy.async;" ::: "memory");  // the copies' reads behind paged_begin's
        volatile Q4Piece *piece = &pieces[np & 1];
        const int steps = piece->steps;
        if (steps == 0) break;
        const int tok0 = piece->t0 * PAGED_TILE + warp * 16, vis = piece->vis, head = piece->head, rows = piece->rows;
        const int lim0 = piece->lim0, limd = piece->limd, q0 = piece->q0;
        const int32_t *ids_row = piece->row;
        // this warp's blocks: the step's 16 tokens, where some row sees one of them
        const int blocks = min(steps, max(0, (vis - tok0 + PAGED_TILE - 1) >> 6));

        // Lane i: where block (of 32) i is, in blocks of the pool.
        int places = 0;
        auto fetch = [&](int b) {
            const int i = b + lane;
            int id = 0;
            const int at = tok0 + i * PAGED_TILE;
            if (i < blocks) {
                id = ids_row[at >> a.page_shift];
                if (id < 0 || id >= a.num_pages) {
                    raise_error(a.err, ERR_PAGE);
                    id = 0;
                }
            }
            places = (((id * a.hkv + head) << a.page_shift) + (at & ((1 << a.page_shift) - 1))) >> 4;
        };
        auto issue = [&](int b, int k, bool send) {  // block b of the unit, into place k of the ring
            if ((b & 31) == 0) fetch(b);
            const int place = __shfl_sync(0xFFFFFFFFu, places, b & 31);
            if (lane == 0) {
                mbar_expect_tx(&full[k], F::BLOCK);
                if (send) bulk_g2s(ring + k * F::BLOCK, pool + (long long)place * F::BLOCK, F::BLOCK, &full[k]);
            }
        };
        int k = j % PQ_NS;  // place and turn of the next block
        uint32_t turn = (uint32_t)(j / PQ_NS) & 1u;
#pragma unroll 1
        for (int b = 0; b < min(PQ_NS, blocks); ++b) issue(b, (k + b) % PQ_NS, !(a.stall && blockIdx.x == 0 && j + b == 0));
        // While these are on their way: the queries as operands, for all warps, and the next piece.
        if (warp >= PQ_WARPS - NT) {
            const int n = PQ_WARPS - 1 - warp, r = 8 * n + g, jj = r >> a.g_shift, hh = r - (jj << a.g_shift);
            Queries8<T, D> q;
            q.load(r < rows ? a.q + (long long)(q0 + jj) * a.q_ts + (long long)((head << a.g_shift) + hh) * a.q_hs : nullptr, sign);
#pragma unroll
            for (int x = 0; x < NG; ++x) q_at[(n * NG + x) * 32 + lane] = q.at(x);
            sums_at[n * 32 + lane] = make_uint2(q.sum[0], q.sum[1]);
            if (t == 0) units_at[n * 8 + g] = q.units_of(c);
        }
        if (warp == 0) next_piece(*walk, &pieces[(np + 1) & 1]);
        __syncthreads();

        uint2 qsum[NT];
        float unit[NT][2];  // of a logit, of this lane's rows
        int lim[NT][2];
        float ref[NT][2], sum[NT][2], o[NT][D / 16][4];
        float ob[NT][4];  // group g (the first two: rows 2 t and 2 t + 1)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            qsum[n] = sums_at[n * 32 + lane];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                unit[n][e] = units_at[n * 8 + 2 * t + e];
                lim[n][e] = lim0 + limd * ((8 * n + 2 * t + e) >> a.g_shift);  // (also of rows that are not there)
                ref[n][e] = PQ_NONE;
                sum[n][e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) ob[n][e] = 0.0f;
#pragma unroll
            for (int x = 0; x < D / 16; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][x][e] = 0.0f;
        }
        uint32_t scale[NG];  // of a group's steps, 2^k twice: o is 2^k times what it stands for
#pragma unroll
        for (int x = 0; x < NG; ++x) scale[x] = PQ_SCALE;

        int b = 0;
#pragma unroll 1
        for (; b < blocks; ++b) {
            ok = __all_sync(0xFFFFFFFFu, paged_wait(smem_addr(&full[k]), turn, abort, a.wait_ns));
            if (!ok) break;
            const unsigned char *st = ring + k * F::BLOCK;
            const int tok = tok0 + b * PAGED_TILE;
            // V's floors and steps of tokens 2 t and 2 t + 1, and of 8 more: pairs of tokens, [8 more][group]
            uint32_t steps2[2][NG], floors2[2];
            auto load_steps = [&]() {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const unsigned char *par = st + F::SIDE + F::PARS + (2 * t + 8 * i) * F::PAR;
                    const KeyVec x = *reinterpret_cast<const KeyVec *>(par), y = *reinterpret_cast<const KeyVec *>(par + F::PAR);
#pragma unroll
                    for (int z = 0; z < NG; ++z) steps2[i][z] = byte_pair(word_of(x, z), word_of(y, z), 0x7632u);
                }
            };
            // what lies behind the tokens that are seen may be anything, not a number too
            auto seen = [&](int i) -> uint32_t {
                const int left = vis - (tok + 2 * t + 8 * i);
                return left <= 0 ? 0u : left == 1 ? 0xFFFFu : 0xFFFFFFFFu;
            };
            load_steps();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const unsigned char *par = st + F::SIDE + F::PARS + (2 * t + 8 * i) * F::PAR + (g & (NG - 1)) * 4;
                floors2[i] = byte_pair(*reinterpret_cast<const uint32_t *>(par), *reinterpret_cast<const uint32_t *>(par + F::PAR), 0x5410u);
            }
            float s[NT][4], y[NT][4];
            {
                KeyCodes<D> kc;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const unsigned char *par = st + F::PARS + (g + 8 * i) * F::PAR;
                    kc.codes(i, *reinterpret_cast<const KeyVec *>(st + (g + 8 * i) * F::CODE + t * (F::CODE / 4)));
                    kc.scales(i, *reinterpret_cast<const KeyVec *>(par), *reinterpret_cast<const uint32_t *>(par + (t & (NG - 1)) * 4));
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) q4_logits<D>(s[n], kc, qsum[n].x, qsum[n].y, [&](int x) { return q_at[(n * NG + x) * 32 + lane]; });
            }
            if (tok + 16 > lim0) {  // not every row sees every token
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][e] = tok + g + 8 * (e >> 1) < lim[n][e & 1] ? s[n][e] : -INFINITY;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    floors2[i] &= seen(i);
#pragma unroll
                    for (int z = 0; z < NG; ++z) steps2[i][z] &= seen(i);
                }
            }
            // Does any step reach 2?  Its bit 14 says so (of one that has become infinite too); the largest ones are looked
            // for only then.
            uint32_t step = 0;
#pragma unroll
            for (int z = 0; z < 2 * NG; ++z) {
                steps2[z / NG][z % NG] = mul_f16(steps2[z / NG][z % NG], scale[z % NG]);
                step |= steps2[z / NG][z % NG];
            }
            step &= 0x40004000u;
            float above = -INFINITY;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[n][e] = fmaf(s[n][e], unit[n][e & 1], -ref[n][e & 1]);
                    above = fmaxf(above, y[n][e]);
                }
            if (__any_sync(0xFFFFFFFFu, above > PQ_ROOM || step)) {
                if (__any_sync(0xFFFFFFFFu, step)) {
                    load_steps();
#pragma unroll
                    for (int z = 0; z < NG; ++z) {
                        if (tok + 16 > lim0) {
                            steps2[0][z] &= seen(0);
                            steps2[1][z] &= seen(1);
                        }
                        uint32_t top = max_f16(steps2[0][z], steps2[1][z]);
                        top = max(top & 0xFFFFu, top >> 16) >> 10;  // exponent bits
                        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                        // (all lanes hold the same.  2^-15 is the one power below binary16's normal numbers that may be
                        // needed: its exponent bits are 0, as the k that they stand for has it)
                        const int was = (int)(scale[z] >> 10 & 31u) - 15, k = (int)top + was >= 16 ? max(14 - (int)top, -15) : was;
                        scale[z] = k == -15 ? 0x02000200u : (uint32_t)(k + 15) * 0x04000400u;
                        const float f = __uint_as_float((uint32_t)(127 + k - was) << 23);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                o[n][2 * z][e] *= f;
                                o[n][2 * z + 1][e] *= f;
                            }
                        steps2[0][z] = mul_f16(steps2[0][z], scale[z]);
                        steps2[1][z] = mul_f16(steps2[1][z], scale[z]);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(s[n][e], s[n][e + 2]);
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
                        const float m = fmaxf(ref[n][e], fmaf(top, unit[n][e], PQ_SLACK - PQ_ROOM));
                        f[e] = exp2_fast(ref[n][e] - m);  // (nothing summed yet: 0 or 1)
                        ref[n][e] = m;
                        sum[n][e] *= f[e];
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[n][e] = fmaf(s[n][e], unit[n][e & 1], -ref[n][e & 1]);
                        ob[n][e] *= f[e & 1];
#pragma unroll
                        for (int x = 0; x < D / 16; ++x) o[n][x][e] *= f[e & 1];
                    }
                }
            }
            uint32_t p[NT][2], rest[NT][2];  // of pairs of tokens, query g
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[n][e] = exp2_fast(y[n][e]);
                    sum[n][e & 1] += y[n][e];
                }
                const uint32_t fa[4] = {floors2[0], 0u, floors2[1], 0u};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    p[n][i] = PgF16::pack(y[n][2 * i], y[n][2 * i + 1]);
                    if (REST) {
                        const float2 f = PgF16::unpack(p[n][i]);
                        rest[n][i] = movmatrix_t(PgF16::pack(y[n][2 * i] - f.x, y[n][2 * i + 1] - f.y));
                    }
                    p[n][i] = movmatrix_t(p[n][i]);
                }
                mma_f16(ob[n], fa, p[n][0], p[n][1]);
                if (REST) mma_f16(ob[n], fa, rest[n][0], rest[n][1]);
            }
            // V's words of the lane's four tokens, two of them each time
            constexpr int VW = D / 64;
            ValueVec v[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const unsigned char *vr = st + F::SIDE + (2 * t + 8 * i) * F::CODE + g * (F::CODE / 8);
                v[i][0] = *reinterpret_cast<const ValueVec *>(vr + odd * F::CODE);
                v[i][1] = *reinterpret_cast<const ValueVec *>(vr + (odd ^ 1) * F::CODE);
            }
#pragma unroll
            for (int x = 0; x < NG; ++x) {
                // The channels of two products.  Of d = 128, bytes x of the lane's two words: their lower codes, their
                // upper ones.  Of d = 64, byte 2 x of its word, byte 2 x + 1.
                uint32_t va[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (D == 128) {
#pragma unroll
                        for (int w = 0; w < VW; ++w) {
                            const uint32_t z = byte_pair(word_of(v[i][0], w), word_of(v[i][1], w), byte0 + x * NEXT_BYTE);
                            va[0][2 * i + (w & 1)] = REST ? z << 4 & HIGH4 : z & LOW4;
                            va[1][2 * i + (w & 1)] = z & HIGH4;
                        }
                    } else {
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const uint32_t z = byte_pair(word_of(v[i][0], 0), word_of(v[i][1], 0), byte0 + (2 * x + m) * NEXT_BYTE);
                            va[m][2 * i] = REST ? z << 4 & HIGH4 : z & LOW4;
                            va[m][2 * i + 1] = z & HIGH4;
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint32_t b0 = mul_f16(p[n][0], steps2[0][x]), b1 = mul_f16(p[n][1], steps2[1][x]);
                    mma_f16(o[n][2 * x], va[0], b0, b1);
                    mma_f16(o[n][2 * x + 1], va[1], b0, b1);
                    if (REST) {
                        // the product's own rest, which is exact, and the weight's
                        const uint32_t r0 = fma_f16(rest[n][0], steps2[0][x], fma_f16(p[n][0], steps2[0][x], b0 ^ 0x80008000u));
                        const uint32_t r1 = fma_f16(rest[n][1], steps2[1][x], fma_f16(p[n][1], steps2[1][x], b1 ^ 0x80008000u));
                        mma_f16(o[n][2 * x], va[0], r0, r1);
                        mma_f16(o[n][2 * x + 1], va[1], r0, r1);
                    }
                }
            }
            fence_proxy_async_smem();  // this block's reads before the next copy to its place
            __syncwarp();
            if (b + PQ_NS < blocks) issue(b + PQ_NS, k, true);
            if (++k == PQ_NS) {
                k = 0;
                turn ^= 1u;
            }
        }
        if (!ok) {
            if (lane == 0) {
                *abort = 1;
                raise_error(a.err, ERR_TIMEOUT);
                // the copies in flight land before the CTA gives its shared memory back
                for (int i = b; i < min(blocks, b + PQ_NS); ++i) mbar_wait_bounded(&full[(j + i) % PQ_NS], (uint32_t)(((j + i) / PQ_NS) & 1), a.wait_ns);
            }
            __syncwarp();
        }
        j += blocks;
        if (__syncthreads_or(!ok)) break;

        // The four warps' states: each scales its sums to the common maximum and lays them in the ring,
        // which holds nothing any more, and all threads add the four and write the partial.
        float *buf = reinterpret_cast<float *>(pq_smem);
        float base[NT][2][NG];  // the floors' part
        float back[NG];         // 2^-k
#pragma unroll
        for (int x = 0; x < NG; ++x) back[x] = __uint_as_float((254u << 23) - __float_as_uint(floor_of(scale[x])));
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int x = 0; x < NG; ++x) base[n][e][x] = __shfl_sync(0xFFFFFFFFu, ob[n][e], 4 * x + t);
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) sum[n][e] += __shfl_xor_sync(0xFFFFFFFFu, sum[n][e], x);
                if (ref[n][e] <= 0.5f * PQ_NONE) ref[n][e] = -INFINITY;
                if (g == 0) *reinterpret_cast<float2 *>(ml + (warp * R + 8 * n + 2 * t + e) * 2) = make_float2(ref[n][e], sum[n][e]);
            }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * n + 2 * t + e;
                float m = -INFINITY, z = 0.0f;
#pragma unroll
                for (int w = 0; w < PQ_WARPS; ++w) m = fmaxf(m, ml[(w * R + r) * 2]);
                const float ms = m == -INFINITY ? 0.0f : m;
#pragma unroll
                for (int w = 0; w < PQ_WARPS; ++w) z += ml[(w * R + r) * 2 + 1] * exp2_fast(ml[(w * R + r) * 2] - ms);
                const float f = exp2_fast(ref[n][e] - ms);
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    // channels 16 x + 2 g and the next one, or of d = 64 16 x + g and 8 more; codes of upper bits are 16 n, with
                    // REST all
                    float *at = buf + (warp * R + r) * D + 16 * x;
                    const float lu = REST || (D == 128 && (x & 1)) ? CODE_UNIT / 16 : CODE_UNIT, hu = REST || D == 64 || (x & 1) ? CODE_UNIT / 16 : CODE_UNIT;
                    const float lo = fmaf(o[n][x][e], lu * back[x / 2], base[n][e][x / 2]) * f, hi = fmaf(o[n][x][e + 2], hu * back[x / 2], base[n][e][x / 2]) * f;
                    if (D == 128) {
                        *reinterpret_cast<float2 *>(at + 2 * g) = make_float2(lo, hi);
                    } else {
                        at[g] = lo;
                        at[g + 8] = hi;
                    }
                }
                if (warp == 0 && g == 0 && r < rows && piece->slot >= 0)
                    *reinterpret_cast<float2 *>(l.part_ml + ((long long)piece->slot * R + r) * 2) = make_float2(m, z);
            }
        __syncthreads();
        if (piece->slot >= 0) {
            float *po = l.part_o + (long long)piece->slot * R * D;
#pragma unroll 1
            for (int x = tid * 4; x < rows * D; x += PQ_NT * 4) {
                float4 u = *reinterpret_cast<const float4 *>(buf + x);
#pragma unroll
                for (int w = 1; w < PQ_WARPS; ++w) {
                    const float4 y = *reinterpret_cast<const float4 *>(buf + w * R * D + x);
                    u = make_float4(u.x + y.x, u.y + y.y, u.z + y.z, u.w + y.w);
                }
                *reinterpret_cast<float4 *>(po + x) = u;
            }
        }
        fence_proxy_async_smem();  // the sums' accesses before the ring's next copies
    }
    pdl_wait();  // the launch before this one is done when this one is
}

// The values of a pool's pages: out [pages][kv_heads][page_tokens][2][d] in 16 bits, one rounding each.
// A thread takes two words: eight pairs of channels d / 8 apart, so that neighbours' stores fill sectors; bound by
// the bytes: 32768 tokens of 8 heads of 128 (42 MB read, 134 written) 28 us, 6.3 TB/s, 0.93 of a plain copy's rate.
template <typename T, int D>
__global__ void __launch_bounds__(256) k_q4_values(const unsigned char *__restrict__ pool, uint16_t *__restrict__ out, long long words) {
    using F = Q4<D>;
    constexpr int W = F::WORDS;
    pdl_wait();
    pdl_trigger();
    for (long long x = (long long)blockIdx.x * 256 + threadIdx.x; x < words; x += (long long)gridDim.x * 256) {
        // pairs of words: [block][side][token][W / 2]
        const int w = (int)(x % (W / 2)) * 2;
        const long long row = x / (W / 2);
        const int token = (int)(row & 15), side = (int)(row >> 4) & 1;
        const long long block = row >> 5;
        const unsigned char *src = pool + block * F::BLOCK + side * F::SIDE;
        const uint2 code = *reinterpret_cast<const uint2 *>(src + token * F::CODE + w * 4);
        const uint32_t *par = reinterpret_cast<const uint32_t *>(src + F::PARS + token * F::PAR);
        uint16_t *dst = out + ((block * 16 + token) * 2 + side) * D + w;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(par + i * W / 32));
            const float lo = fmaf((float)((code.x >> (4 * i)) & 15u), p.y, p.x), hi = fmaf((float)((code.y >> (4 * i)) & 15u), p.y, p.x);
            *reinterpret_cast<uint32_t *>(dst + i * W) = T::pack(lo, hi);
        }
    }
}

}  // namespace

cudaError_t launch_paged_q4(const PagedArgs &a, const PagedLine &l, bool second, int dtype, int d, cudaStream_t s) {
    const int rows = 1 << (l.tt_shift + a.g_shift);
#define VERKV_PQ(TT, DT, DD, NN)                                                                              \
    if (dtype == DT && d == DD && rows == 8 * NN) {                                                            \
        const cudaError_t e = ensure_smem((const void *)k_paged_q4<TT, DD, NN>, Q4Layout<DD, NN>::BYTES);      \
        if (e != cudaSuccess) return e;                                                                        \
        return launch_pdl(k_paged_q4<TT, DD, NN>, dim3(l.ctas), dim3(PQ_NT), Q4Layout<DD, NN>::BYTES, s, a, l, second ? 1 : 0); \
    }
    VERKV_PQ(PgBf16, VERKV_BF16, 128, 1) VERKV_PQ(PgBf16, VERKV_BF16, 128, 2) VERKV_PQ(PgBf16, VERKV_BF16, 128, 4)
    VERKV_PQ(PgBf16, VERKV_BF16, 64, 1) VERKV_PQ(PgBf16, VERKV_BF16, 64, 2)
    VERKV_PQ(PgF16, VERKV_F16, 128, 1) VERKV_PQ(PgF16, VERKV_F16, 128, 2) VERKV_PQ(PgF16, VERKV_F16, 128, 4)
    VERKV_PQ(PgF16, VERKV_F16, 64, 1) VERKV_PQ(PgF16, VERKV_F16, 64, 2)
#undef VERKV_PQ
    return cudaErrorInvalidValue;
}

cudaError_t launch_q4_values(const void *pool, void *out, int dtype, long long rows, int d, cudaStream_t s) {
    const long long words = rows * 2 * (d / 16);
    const unsigned blocks = (unsigned)std::max(1LL, std::min((words + 255) / 256, 152LL * 16));
#define VERKV_QV(TT, DT, DD) \
    if (dtype == DT && d == DD) return launch_pdl(k_q4_values<TT, DD>, dim3(blocks), dim3(256), 0, s, (const unsigned char *)pool, (uint16_t *)out, words);
    VERKV_QV(PgBf16, VERKV_BF16, 128) VERKV_QV(PgBf16, VERKV_BF16, 64)
    VERKV_QV(PgF16, VERKV_F16, 128) VERKV_QV(PgF16, VERKV_F16, 64)
#undef VERKV_QV
    return cudaErrorInvalidValue;
}

}  // namespace verkv
