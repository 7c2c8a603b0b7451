// k_paged_wide.cu -- attention over the paged cache for many query rows: a prefix that a batch
// shares, or a sequence with many queries, on the fifth-generation tensor cores.
//
// With R rows a KV head, a token costs 4 R d flops and 4 d bytes: from about 280 rows on the
// products bound it, below that K and V's bytes.  A unit is 128 or 256 rows (query tokens x heads of
// one KV head); it streams 128-token steps of K and V by TMA into a shared-memory ring, and for
// every step
//     S = Q K^T   128 x 128, Q and K in shared memory,       float32 in tensor memory
//     P = 2^(S c - ref), 16 bits, written over S in tensor memory; with 128 rows in two parts, the
//         rounded weights and what rounding leaves out, which fill S's place between them
//     O += P V    128 x d, P in tensor memory, V in shared memory
// Two such chains run side by side so that one's softmax hides behind the other's products: with
// 256 rows, the two halves of the rows on the same step; with 128 rows, even and odd steps, joined
// at the unit's end.  Items n = 0, 1, ... alternate between the chains; the products are issued in
// the order S(0) S(1) | P V(0) S(2) | P V(1) S(3) | ..., in which the tensor core executes them, so
// that S(n + 2) may overwrite the P that P V(n) reads.
//
// One warp issues all products, an elected lane of it, in step: its descriptors and barriers stay in
// uniform registers, and a step's 32 instructions are issued while the tensor core works.  (Issued by
// a thread in a branch of its own, 256 sequences behind 32K tokens took 178 us a call instead of 158;
// two such threads, one a chain, taking turns at a barrier: 157, and 8 % more with few queries.)
//
// Warps: 0-3 and 4-7 hold the rows of the chains, a thread a row (no shuffles); 8 issues the
// products; 9 walks the line and copies.  The reference `ref` of a row's weights is its running
// maximum less SHIFT, and is raised -- with O scaled in tensor memory -- only when the maximum has
// risen by more than SLACK since: rarely after the first steps, and no weight passes
// 2^(SHIFT + SLACK) <= 2^14.  fp16 weights sit 2^8 up, away from its subnormals.
//
// Weights in two parts leave o off by its own rounding alone (32K tokens, bf16: 1.64e-3 of its root mean
// square) at twice the products of P V.  With 128 rows the bytes bound a step and that costs little (8
// sequences behind 32K tokens 40.9 -> 43.9 us).  With 256 rows the products bound it: 256 sequences behind
// 32K tokens would go from 148 to 214 us, a prompt of 32768 from 9.0 to 11.4 ms.  There the weights are
// rounded once, as o is (2.2e-3 in all); the sum they are divided by is not.
//
// Measured (8 heads, d 128, bf16; whole calls): 1024 rows a head behind 128K tokens 405 us,
// 1.36 PFLOP/s, 0.71 of a library matrix product's rate; behind 32K tokens 120 us; 32 rows behind 128K
// 93 us, 0.85 of a plain copy's bandwidth.  A step of 256 rows takes about 3300 cycles.  Its products
// need 2050 at the tensor core's rate and some 2500 with their operands' reads from shared memory
// (Q K^T: 82 cycles for 64), and it is they that bound it: a faster maximum, or P announced in smaller
// parts, changed nothing or lost (the smaller parts 4 %), and Q K^T in two halves lost 25 %.  With
// d 64 the products halve and the exponentials do not (32K tokens, 1024 rows: 98 to 109 us).  A thread has 168
// registers (ten warps an SM), a softmax row takes 128 of them, and ptxas spills 84 to 120 bytes.
#include <float.h>
#include <math.h>

#include <algorithm>

#include "paged.cuh"
#include "pivotal_mma.cuh"
#include "tcgen05.cuh"
#include "verkv_common.cuh"

namespace verkv {

namespace {

constexpr int PW_NT = 320;
constexpr int PW_MMA = 8, PW_COPY = 9;  // warps
constexpr int PW_PIECES = 8;            // ring of pieces: the copies are at most a ring of slots ahead

struct PieceDesc {
    int steps;       // 0: the run is over
    int tok0;        // first token
    int vis;         // tokens some row of the unit sees
    int q0, nq;      // query tokens of the row tile
    int head;        // KV head
    int lim0, limd;  // tokens the tile's first query sees, and how many more each next one does
    int slot;        // partial slot, or -1
};

template <int D, int TILES>
struct WideLayout {
    static constexpr int HALVES = D / 64;
    static constexpr int BOX = PAGED_WIDE_TILE * 128;   // 128 tokens (or rows) x 64 channels
    static constexpr int SLOT = HALVES * BOX;           // K or V of a step; also a tile of Q
    static constexpr int NS = D == 128 ? (TILES == 2 ? 5 : 6) : 10;
    static constexpr int R = TILES * 128;
    static constexpr bool REST = TILES == 1;            // weights in two parts (see above)
    static constexpr int Q = 0;
    static constexpr int RING = TILES * SLOT;
    static constexpr int ML = RING + NS * SLOT;                          // float [2][128][2]
    static constexpr int PIECES = ML + 2 * 128 * 2 * 4;                  // PieceDesc [PW_PIECES]
    static constexpr int BARS = (PIECES + PW_PIECES * (int)sizeof(PieceDesc) + 7) / 8 * 8;
    // full, empty [NS]; piece [PW_PIECES]; s_full, h_full, p_full [2]; q_full, o_full, ml_full, drain
    static constexpr int NBARS = 2 * NS + PW_PIECES + 6 + 4;
    static constexpr int BYTES = BARS + NBARS * 8 + 16;
};

// The order of a piece's 2 n slots, which is that of their use: with two tiles on the same step K(0)
// V(0) K(1) V(1) ..; with even and odd steps side by side K(0) K(1) V(0) K(2) V(1) .. V(n - 2) V(n - 1).
// (A slot loaded earlier than it is used is one less in flight: in the first order for both, 8
// sequences behind 32K tokens took 40.5 us for 39.3.)
template <int TILES>
struct WideOrder {
    static __device__ __forceinline__ bool is_v(int x, int n) { return TILES == 2 ? x & 1 : x == 2 * n - 1 || (x > 0 && (x & 1) == 0); }
    static __device__ __forceinline__ int step(int x, int n) {
        return TILES == 2 ? x >> 1 : x == 2 * n - 1 ? n - 1 : x & 1 ? (x + 1) >> 1 : x > 0 ? (x - 2) >> 1 : 0;
    }
    static __device__ __forceinline__ int k(int step) { return TILES == 2 ? 2 * step : step == 0 ? 0 : 2 * step - 1; }
    static __device__ __forceinline__ int v(int step, int n) { return TILES == 2 ? 2 * step + 1 : step < n - 1 ? 2 * step + 2 : 2 * n - 1; }
};

template <typename T>
struct Weights;
template <>
struct Weights<PgBf16> {
    static constexpr float SLACK = 8.0f;
    static constexpr bool BF = true;
};
template <>
struct Weights<PgF16> {
    static constexpr float SLACK = 6.0f;
    static constexpr bool BF = false;
};

// a * b + c on two floats in one instruction.
__device__ __forceinline__ void fma2(float &x, float &y, float b, float c) {
    unsigned long long v, bb, cc;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
    asm("mov.b64 %0, {%1, %1};" : "=l"(bb) : "f"(b));
    asm("mov.b64 %0, {%1, %1};" : "=l"(cc) : "f"(c));
    asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(v) : "l"(bb), "l"(cc));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}

// The pair (x, y) added to the pair v.
__device__ __forceinline__ void add2(unsigned long long &v, float x, float y) {
    unsigned long long w;
    asm("mov.b64 %0, {%1, %2};" : "=l"(w) : "f"(x), "f"(y));
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(w));
}
__device__ __forceinline__ float lo2(unsigned long long v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi2(unsigned long long v) { return __uint_as_float((uint32_t)(v >> 32)); }

template <typename T, int D, int TILES>
__global__ void __launch_bounds__(PW_NT, 1)
    k_paged_wide(const __grid_constant__ PagedArgs a, const __grid_constant__ PagedLine l, const int second,
                 const __grid_constant__ CUtensorMap map) {
    using LY = WideLayout<D, TILES>;
    using W = Weights<T>;
    constexpr int NS = LY::NS, R = LY::R;
    extern __shared__ __align__(1024) unsigned char pw_smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(pw_smem + LY::BARS), *empty = full + NS, *piece = empty + NS;
    uint64_t *s_full = piece + PW_PIECES, *h_full = s_full + 2, *p_full = h_full + 2, *q_full = p_full + 2, *o_full = q_full + 1;
    uint64_t *ml_full = o_full + 1, *drain = ml_full + 1;
    uint32_t *tmem_at = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_at + 1);
    PieceDesc *pieces = reinterpret_cast<PieceDesc *>(pw_smem + LY::PIECES);
    float *ml = reinterpret_cast<float *>(pw_smem + LY::ML);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int k = 0; k < NS; ++k) {
            mbar_init(&full[k], 1);
            mbar_init(&empty[k], 1);
        }
        for (int k = 0; k < PW_PIECES; ++k) mbar_init(&piece[k], 1);
        for (int k = 0; k < 2; ++k) {
            mbar_init(&s_full[k], 1);
            mbar_init(&h_full[k], 4);
            mbar_init(&p_full[k], 4);
        }
        mbar_init(q_full, 8);
        mbar_init(o_full, 1);
        mbar_init(ml_full, 8);
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *abort = 0;
    }
    if (warp == PW_MMA) tmem_alloc(tmem_at, 512);
    if (warp == PW_COPY) {
        if (lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map)) : "memory");
        // Before the CTA's barrier: no wait's limit counts what the kernels ahead still take.
        paged_begin(a, second != 0);
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tm = *tmem_at;
    // S (and P over it) of chain i in columns 128 i .., O in 256 + 128 i ..
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        const bool ok = paged_wait(smem_addr(bar), parity, abort, a.wait_ns);
        if (__all_sync(0xFFFFFFFFu, ok)) return true;
        if (lane == 0) {
            *abort = 1;
            raise_error(a.err, ERR_TIMEOUT);
        }
        return false;
    };

    if (warp == PW_COPY) {
        // The other warps touch the caller's data only after the first piece that this one announces.
        // (the chains' states have no use for their place yet)
        PagedWalk<true> wk;
        wk.start(a, l, blockIdx.x, reinterpret_cast<int2 *>(ml), 2 * 128);
        const int box = min(1 << a.page_shift, PAGED_WIDE_TILE);
        int j = 0, np = 0;  // slots and pieces so far
        bool go = true;
        while (go && wk.next(a, l, blockIdx.x)) {
            const PagedLevel &lv = a.level[wk.s.own ? 1 : 0];
            const int32_t *row = lv.table + (long long)wk.s.row * lv.stride;
            const int vis = paged_visible(wk.s, l, wk.m);
            const int steps = wk.t1 - wk.t0;
            int ids = 0, ids0 = 1, ids1 = 0;      // lane i: id of page ids0 + i of the sequence
            int y[2] = {0, 0}, pages[2] = {0, 0};  // row of this lane's page, pages: of the last two K steps
#pragma unroll 1
            for (int x = 0; x < 2 * steps; ++x, ++j) {
                // What the x-th slot of the piece takes (see WideOrder).
                const bool is_v = WideOrder<TILES>::is_v(x, steps);
                const int step = WideOrder<TILES>::step(x, steps), k = j % NS;
                if (!is_v) {
                    const int tok0 = (wk.t0 + step) * PAGED_WIDE_TILE, valid = min(PAGED_WIDE_TILE, vis - tok0);
                    const int p0 = tok0 >> a.page_shift;
                    y[0] = y[1];
                    pages[0] = pages[1];
                    pages[1] = (valid + box - 1) / box;
                    if (p0 < ids0 || p0 + pages[1] > ids1) {
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
                    const int id = __shfl_sync(0xFFFFFFFFu, ids, (p0 + lane - ids0) & 31);
                    y[1] = ((id * a.hkv + wk.head) << a.page_shift) + ((tok0 + lane * box) & ((1 << a.page_shift) - 1));
                }
                const int back = TILES == 1 && is_v && step < steps - 1 ? 0 : 1;
                const int n = back ? pages[1] : pages[0], at = back ? y[1] : y[0];
                if (j >= NS) go = wait(&empty[k], (uint32_t)(j / NS - 1));
                if (!go) break;
                if (lane == 0) {
                    if (x == 0) {
                        // A slot was free for this piece's first step, so at most NS / 2 pieces are ahead
                        // of the products: the entry reused here is long read.
                        PieceDesc s;
                        s.steps = steps;
                        s.tok0 = wk.t0 * PAGED_WIDE_TILE;
                        s.vis = vis;
                        s.q0 = wk.s.q0 + (wk.m << l.tt_shift);
                        s.nq = min(1 << l.tt_shift, wk.s.qn - (wk.m << l.tt_shift));
                        s.head = wk.head;
                        s.lim0 = wk.s.own ? wk.s.len - (wk.s.qn - 1 - (wk.m << l.tt_shift)) : wk.s.len;
                        s.limd = wk.s.own ? 1 : 0;
                        s.slot = wk.slot < l.slots ? wk.slot : -1;
                        if (s.slot < 0) raise_error(a.err, ERR_PAGE);
                        pieces[np % PW_PIECES] = s;
                        mbar_arrive(&piece[np % PW_PIECES]);
                    }
                    mbar_expect_tx(&full[k], (uint32_t)(n * box * 2 * D));
                }
                __syncwarp();
                if (lane < n && !(a.stall && blockIdx.x == 0 && j == 0)) {
                    unsigned char *st = pw_smem + LY::RING + (size_t)k * LY::SLOT + lane * box * 128;
#pragma unroll
                    for (int b = 0; b < LY::HALVES; ++b)
                        tma_load_2d(st + b * LY::BOX, &map, (is_v ? D : 0) + b * 64, at, &full[k]);
                }
                __syncwarp();
            }
            ++np;
        }
        if (go && lane == 0) {
            pieces[np % PW_PIECES].steps = 0;
            mbar_arrive(&piece[np % PW_PIECES]);
        }
        if (lane == 0) {
            // The copies in flight land here even where another warp's wait ran out: they are the last NS
            // slots issued.
            for (int i = max(0, j - NS); i < j; ++i) mbar_wait_bounded(&full[i % NS], (uint32_t)((i / NS) & 1), a.wait_ns);
        }
        __syncwarp();
    } else if (warp == PW_MMA) {
        // One lane issues every product, in one order; the warp runs in step (elect_one).  A descriptor is
        // its slot's plus a constant (its address field counts 16 bytes).
        const uint32_t it = elect_one();
        {
            const uint64_t ring = smem_desc(smem_addr(pw_smem + LY::RING), LY::BOX, 1024);
            const uint64_t qd = smem_desc(smem_addr(pw_smem + LY::Q), LY::BOX, 1024);
            constexpr uint32_t IS = mma_desc(128, 128, W::BF, false), IO = mma_desc(128, D, W::BF, true);
            using Order = WideOrder<TILES>;
            auto await = [&](uint64_t *bar, uint32_t parity) -> bool {
                if (__all_sync(0xFFFFFFFFu, paged_wait(smem_addr(bar), parity, abort, a.wait_ns))) return true;
                *abort = 1;
                raise_error(a.err, ERR_TIMEOUT);
                return false;
            };
            int j0 = 0;                // slots used before the piece
            uint32_t ns[2] = {0, 0};   // items of each chain so far
            bool go = true;
            for (int np = 0; go; ++np) {
                if (!await(&piece[np % PW_PIECES], (uint32_t)(np / PW_PIECES))) break;
                const PieceDesc pd = pieces[np % PW_PIECES];
                if (pd.steps == 0) break;
                const int items = pd.steps * TILES;
                go = await(q_full, (uint32_t)np);
                tcgen05_after_sync();
                // K's slot of an item, filled; S of the item; and what waits for it: the softmax, and the
                // copies after the step's last item.
                auto k_slot = [&](int n) { return j0 + Order::k(n / TILES); };
                auto k_there = [&](int n) -> bool {
                    const int x = k_slot(n);
                    return n % TILES != 0 || await(&full[x % NS], (uint32_t)(x / NS));
                };
                auto do_s = [&](int n) {
                    const uint64_t kd = ring + (uint32_t)(k_slot(n) % NS * (LY::SLOT >> 4));
                    const uint64_t q = qd + (uint32_t)(n % TILES * (LY::SLOT >> 4));
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        const int off = ((x / 4) * LY::BOX + (x % 4) * 32) >> 4;
                        mma_ss(tm + (n & 1) * 128, q + off, kd + off, IS, x > 0, it);
                    }
                    tcgen05_commit(&s_full[n & 1], it);
                    if (n % TILES == TILES - 1) tcgen05_commit(&empty[k_slot(n) % NS], it);
                };
#pragma unroll 1
                for (int n = 0; n < min(2, items) && go; ++n) {
                    if ((go = k_there(n))) do_s(n);
                }
#pragma unroll 1
                for (int n = 0; n < items && go; ++n) {
                    const int step = n / TILES, tile = n % TILES, i = n & 1;
                    const int valid = min(PAGED_WIDE_TILE, pd.vis - (pd.tok0 + step * PAGED_WIDE_TILE));
                    const int vx = j0 + Order::v(step, pd.steps), vs = vx % NS;
                    if (tile == 0) {
                        if (!(go = await(&full[vs], (uint32_t)(vx / NS)))) break;
                        if (valid & 15) {
                            // V rows of the last 16 tokens that nothing sees may hold anything, NaN too: a
                            // weight of 0 would keep it.
                            unsigned char *v = pw_smem + LY::RING + vs * LY::SLOT;
#pragma unroll 1
                            for (int x = valid * 8 + lane; x < ((valid + 15) & ~15) * 8; x += 32)
#pragma unroll
                                for (int h = 0; h < LY::HALVES; ++h)
                                    *reinterpret_cast<uint4 *>(v + h * LY::BOX + x * 16) = make_uint4(0u, 0u, 0u, 0u);
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                    }
                    const bool more = n + 2 < items;
                    if (more && !(go = k_there(n + 2))) break;
                    const uint32_t pt = tm + i * 128, ot = tm + 256 + i * 128;
                    const uint64_t vd = ring + (uint32_t)(vs * (LY::SLOT >> 4));
                    const bool add = step >= (TILES == 2 ? 1 : 2);
                    if (!(go = await(&h_full[i], ns[i]))) break;
                    tcgen05_after_sync();
                    // The first half of P's tokens, while the softmax writes the second.
                    if (valid > PAGED_WIDE_TILE - 16) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            mma_ts(ot, pt + x * 8, vd + x * 128, IO, add || x > 0, it);
                            if (LY::REST) mma_ts(ot, pt + 64 + x * 8, vd + x * 128, IO, true, it);
                        }
                        if (!(go = await(&p_full[i], ns[i]))) break;
                        tcgen05_after_sync();
#pragma unroll
                        for (int x = 4; x < 8; ++x) {
                            mma_ts(ot, pt + x * 8, vd + x * 128, IO, true, it);
                            if (LY::REST) mma_ts(ot, pt + 64 + x * 8, vd + x * 128, IO, true, it);
                        }
                    } else {
                        if (!(go = await(&p_full[i], ns[i]))) break;
                        tcgen05_after_sync();
#pragma unroll 1
                        for (int x = 0; x < (valid + 15) / 16; ++x) {
                            mma_ts(ot, pt + x * 8, vd + x * 128, IO, add || x > 0, it);
                            if (LY::REST) mma_ts(ot, pt + 64 + x * 8, vd + x * 128, IO, true, it);
                        }
                    }
                    ++ns[i];
                    if (more) do_s(n + 2);
                    if (tile == TILES - 1) tcgen05_commit(&empty[vs], it);
                }
                if (!go) break;
                tcgen05_commit(o_full, it);
                j0 += 2 * pd.steps;
            }
            // Nothing is in flight when the CTA gives its tensor memory back.
            tcgen05_commit(drain, it);
            if (!mbar_wait_bounded(drain, 0u, a.wait_ns)) raise_error(a.err, ERR_TIMEOUT);
        }
        __syncwarp();
    } else {
        const int i = warp >> 2;                       // chain
        const int r = (warp & 3) * 32 + lane;          // row of the tile
        const int row = TILES == 2 ? i * 128 + r : r;  // row of the unit
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t ts = tm + lanes + i * 128;
        const float c = fabsf(a.scale_log2);
        const uint32_t sign = a.scale_log2 < 0.0f ? 0x80008000u : 0u;  // a negative scale turns Q round
        uint32_t ns = 0;
        for (int np = 0;; ++np) {
            if (!wait(&piece[np % PW_PIECES], (uint32_t)(np / PW_PIECES))) break;
            const PieceDesc pd = pieces[np % PW_PIECES];
            if (pd.steps == 0) break;
            const int jj = row >> a.g_shift, hh = row - (jj << a.g_shift);
            const bool real = jj < pd.nq;
            const bool busy = __any_sync(0xFFFFFFFFu, real);  // a warp without rows only keeps step
            const int lim = real ? pd.lim0 + pd.limd * jj : 0;
            const int count = TILES == 2 ? pd.steps : (pd.steps + 1 - i) / 2;
            {
                // Q, swizzled as the copies are: a thread a row; with one tile the chains halve it.
                const uint16_t *src = a.q + (long long)(pd.q0 + (real ? jj : 0)) * a.q_ts + (long long)((pd.head << a.g_shift) + hh) * a.q_hs;
                unsigned char *dst = pw_smem + LY::Q + (TILES == 2 ? i * LY::SLOT : 0);
                constexpr int N = TILES == 2 ? D / 8 : D / 16;
                const int c0 = TILES == 2 ? 0 : i * N;
#pragma unroll 4
                for (int x = 0; x < N; ++x) {
                    const int ch = c0 + x;
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (real) v = *reinterpret_cast<const uint4 *>(src + ch * 8);
                    v = make_uint4(v.x ^ sign, v.y ^ sign, v.z ^ sign, v.w ^ sign);
                    *reinterpret_cast<uint4 *>(dst + (ch >> 3) * LY::BOX + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v;
                }
                fence_proxy_async_smem();
                tcgen05_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }
            float ref = -INFINITY, sum = 0.0f;
            bool ok = true;
#pragma unroll 1
            for (int n = 0; n < count; ++n) {
                if (!(ok = wait(&s_full[i], ns))) break;
                tcgen05_after_sync();
                if (busy) {
                    uint32_t s[128];
                    tmem_ld128(s, ts);
                    const int tok0 = pd.tok0 + (TILES == 2 ? n : 2 * n + i) * PAGED_WIDE_TILE;
                    if (__any_sync(0xFFFFFFFFu, tok0 + PAGED_WIDE_TILE > lim)) {
#pragma unroll
                        for (int x = 0; x < 128; ++x) s[x] = tok0 + x < lim ? s[x] : 0xFF800000u;
                    }
                    float top[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) top[x] = __uint_as_float(s[x]);
#pragma unroll
                    for (int x = 4; x < 128; ++x) top[x & 3] = fmaxf(top[x & 3], __uint_as_float(s[x]));
                    const float want = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c - T::SHIFT;
                    if (__any_sync(0xFFFFFFFFu, want > ref + W::SLACK || (ref == -INFINITY && want != -INFINITY))) {
                        const float m = fmaxf(ref, want);
                        const float f = m == ref ? 1.0f : exp2_fast(ref - m);
                        ref = m;
                        sum *= f;
                        if (n > 0) {
                            // P V(n - 1) of this chain is done: S(n) was issued after it.
#pragma unroll 1
                            for (int x = 0; x < D; x += 32) {
                                uint32_t o[32];
                                tmem_ld32(o, tm + lanes + 256 + i * 128 + x);
#pragma unroll
                                for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                                tmem_st32(tm + lanes + 256 + i * 128 + x, o);
                            }
                        }
                    }
                    const float base = ref == -INFINITY ? 0.0f : ref;  // a row that sees nothing so far
                    unsigned long long part[2] = {0ull, 0ull};  // pairs of floats
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t p[32], rest[32];
#pragma unroll
                        for (int x = 0; x < 32; ++x) {
                            float u = __uint_as_float(s[64 * h + 2 * x]), v = __uint_as_float(s[64 * h + 2 * x + 1]);
                            fma2(u, v, c, -base);
                            u = exp2_fast(u);
                            v = exp2_fast(v);
                            p[x] = T::pack(u, v);
                            if (LY::REST) rest[x] = pack_rest<T>(p[x], u, v);
                            add2(part[x & 1], u, v);
                        }
                        tmem_st32(ts + 32 * h, p);
                        if (LY::REST) tmem_st32(ts + 64 + 32 * h, rest);
                        tmem_wait_st();
                        if (h == 0) {
                            tcgen05_before_sync();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&h_full[i]);
                        }
                    }
                    sum += (lo2(part[0]) + hi2(part[0])) + (lo2(part[1]) + hi2(part[1]));
                }
                tcgen05_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (!busy) mbar_arrive(&h_full[i]);
                    mbar_arrive(&p_full[i]);
                }
                ++ns;
            }
            if (!ok) break;
            if (TILES == 1) {
                // Each chain tells the other its rows' reference and sum, once all eight warps have read those
                // of the unit before: a first product of this unit says so, and a chain without one asks.
                if (count == 0 && !wait(q_full, (uint32_t)np)) break;
                ml[(i * 128 + r) * 2] = ref;
                ml[(i * 128 + r) * 2 + 1] = sum;
                __syncwarp();
                if (lane == 0) mbar_arrive(ml_full);
                if (!wait(ml_full, (uint32_t)np)) break;
            }
            if (!wait(o_full, (uint32_t)np)) break;
            tcgen05_after_sync();
            if (busy) {
                // Partials lie [slot][group of 4 rows][group of 4 channels][4 rows][4]: lanes (rows) write
                // whole sectors, and a reader of one row shares its lines with its neighbours'.
                float *po = l.part_o + (long long)max(pd.slot, 0) * R * D + (row >> 2) * (D * 4) + (row & 3) * 4;
                float *pm = l.part_ml + ((long long)max(pd.slot, 0) * R + row) * 2;
                const bool put = real && pd.slot >= 0;
                if (TILES == 2) {
#pragma unroll 1
                    for (int x = 0; x < D; x += 32) {
                        uint32_t o[32];
                        tmem_ld32(o, tm + lanes + 256 + i * 128 + x);
                        if (put) {
#pragma unroll
                            for (int y = 0; y < 8; ++y)
                                *reinterpret_cast<uint4 *>(po + (x / 4 + y) * 16) =
                                    make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
                        }
                    }
                    if (put) *reinterpret_cast<float2 *>(pm) = make_float2(ref, sum);
                } else {
                    const float m0 = ml[r * 2], z0 = ml[r * 2 + 1], m1 = ml[(128 + r) * 2], z1 = ml[(128 + r) * 2 + 1];
                    const float m = fmaxf(m0, m1), ms = m == -INFINITY ? 0.0f : m;
                    const float f0 = exp2_fast(m0 - ms), f1 = exp2_fast(m1 - ms);
                    const bool both = pd.steps > 1;  // else chain 1's columns hold nothing of this unit
#pragma unroll 1
                    for (int x0 = 0; x0 < D / 2; x0 += 32) {
                        const int x = i * (D / 2) + x0;
                        uint32_t o[32], o1[32];
                        tmem_ld32(o, tm + lanes + 256 + x);
                        if (both) tmem_ld32(o1, tm + lanes + 384 + x);
#pragma unroll
                        for (int y = 0; y < 32; ++y) {
                            float v = __uint_as_float(o[y]) * f0;
                            if (both) v = fmaf(__uint_as_float(o1[y]), f1, v);
                            o[y] = __float_as_uint(v);
                        }
                        if (put) {
#pragma unroll
                            for (int y = 0; y < 8; ++y)
                                *reinterpret_cast<uint4 *>(po + (x / 4 + y) * 16) =
                                    make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
                        }
                    }
                    if (put && i == 0) *reinterpret_cast<float2 *>(pm) = make_float2(m, z0 * f0 + z1 * f1);
                }
            }
            tcgen05_before_sync();
            // The next unit's Q overwrites this one's, and its products these sums: it is announced by
            // all eight warps (q_full), each after its reads here.
        }
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (warp == PW_MMA) tmem_free(tm, 512);
    pdl_wait();  // the launch before this one is done when this one is
}

}  // namespace

cudaError_t launch_paged_wide(const PagedArgs &args, const PagedLine &l, const CUtensorMap &map, bool second, int dtype,
                              int d, cudaStream_t s) {
    PagedArgs a = args;
    // a scale that rounds to 0 would make the masked logits' -infinity not a number
    if (fabsf(a.scale_log2) < FLT_MIN) a.scale_log2 = copysignf(FLT_MIN, a.scale_log2);
    const int tiles = (1 << (l.tt_shift + a.g_shift)) / 128;
#define VERKV_WIDE(TT, DT, DD, NN)                                                              \
    if (dtype == DT && d == DD && tiles == NN) {                                                \
        const size_t smem = WideLayout<DD, NN>::BYTES;                                          \
        const cudaError_t e = ensure_smem((const void *)k_paged_wide<TT, DD, NN>, smem);        \
        if (e != cudaSuccess) return e;                                                         \
        return launch_pdl(k_paged_wide<TT, DD, NN>, dim3(l.ctas), dim3(PW_NT), smem, s, a, l, second ? 1 : 0, map); \
    }
    VERKV_WIDE(PgBf16, VERKV_BF16, 128, 1) VERKV_WIDE(PgBf16, VERKV_BF16, 128, 2)
    VERKV_WIDE(PgBf16, VERKV_BF16, 64, 1) VERKV_WIDE(PgBf16, VERKV_BF16, 64, 2)
    VERKV_WIDE(PgF16, VERKV_F16, 128, 1) VERKV_WIDE(PgF16, VERKV_F16, 128, 2)
    VERKV_WIDE(PgF16, VERKV_F16, 64, 1) VERKV_WIDE(PgF16, VERKV_F16, 64, 2)
#undef VERKV_WIDE
    return cudaErrorInvalidValue;
}

}  // namespace verkv
