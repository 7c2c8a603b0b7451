// k_weigh.cu -- the attention weight that each cached token gets, added up over queries and heads:
//
//   out[s][h][i] = in[s][h][i] + sum_{j, g} 2^(q_jhg . k_i scale log2(e) - lse_jhg log2(e)),  j sees i
//
// One pass over the keys (the values are not read): no maximum is needed, since lse is at hand.  Tokens are
// the rows (m16) of mma.m16n8k16 and query rows (query tokens x heads of one KV head) its columns, so that
// a token's sum is over its own row of the product: additions in registers, and two shuffles for the four
// lanes of a row at its end.  A token's keys go from memory to the A operand without a shuffle: a product
// does not mind the order of its channels, and the order here is the memory's.  Every sum has one owner
// and a fixed order.  What lies behind a sequence's length is copied in pieces of 512 places a warp.
//
// k_weigh_few: up to about 8 rows a sequence (a decode step).  Bound by the keys' bytes (16 sequences of 16384 tokens, 550 MB:
// 90 us, 6.1 TB/s, 0.90 of a plain copy's rate), over 4-bit pages by its copies and its chains of products alike, with
// 16 warps an SM and 48 % of the issue slots (32 of up to 16384, 190 MB: 61 us, 0.46).  All sequences'
// blocks of 16 tokens, end to end, are cut into equal runs, one a warp, which has a ring of blocks in shared
// memory: its next two are on their way while it works on two (chains of products and exponentials side by side), or of 4-bit
// pages seven while it works on one.  (One in place of two, 32 sequences of 2000-2048 tokens: 32.4 us, 27.1; two of 4-bit
// pages, which leaves three CTAs of four an SM, 32 of up to 16384: 65.3 us, 61.5.)
//
// k_weigh_many: more rows (drafts; over 4-bit pages any number).  16 rows, four sequences of 8192 tokens: 20.5 us, waiting
// for an item's loads (lengths, table, keys), which are not on their way during the item before; over 4-bit pages 27.7,
// and about 1 us for each row more (64 queries, 256 rows: 256 us for 28 over 16-bit pages), chains of mma.sync and
// float32 sums with 12 warps an SM: 46 % of the issue slots, 15 % of the tensor pipe.  Nothing stands against a form of
// k_weigh_wide over codes, which are exact there too; it has not been written.  A CTA takes 128 tokens
// of one KV head, 32 a warp, whose keys stay in registers while 32 rows at a time pass through shared
// memory, the next ones on their way meanwhile.
//
// k_weigh_wide: many rows over 16-bit pages (the last queries of a prompt, a whole one), on the
// fifth-generation tensor cores.  An item is 256 tokens of one KV head, whose keys come once by TMA; 128 query
// rows a tile pass by, also by TMA (a box of all a KV head's query heads of 128 / q_per_kv tokens), through a
// ring, and S = K Q^T, twice 128 tokens x 128 rows, goes to tensor memory, two places for either half.  There
// a thread has a token: it reads its own lane, and its sum needs no other thread.  Two groups of four
// warps take the tiles of a half in turn, one place each, and join their sums at the item's end; one warp
// copies, one issues the products.  Bound by the turn of a place (product, read, arithmetic, handing
// back): 64 queries of four prompts of 8192 tokens 28.7 us, 2048 queries 584 us, 828 TFLOP/s, 0.42 of a
// library product's burst.  (Of the latter: 1/8 or 1/4 of the exponentials as polynomials 582 and 625 us;
// reads in pieces ahead of the arithmetic 626; one group a half, which takes all 128 columns to registers
// at once and so frees the place before it makes the exponentials 597.)
#include <math.h>

#include <algorithm>

#include "paged.cuh"
#include "pivotal_mma.cuh"
#include "q4.cuh"
#include "tcgen05.cuh"
#include "verkv_common.cuh"

namespace verkv {

namespace {

constexpr int WF_NT = 128, WM_NT = 128;
constexpr int WM_ROWS = 32;    // query rows in shared memory at a time
constexpr int WM_TOKENS = 128;  // tokens of an item
// k_weigh_wide: more rows a sequence than these, on average.  (32 rows, four sequences of 8192 tokens: 24.0 us, k_weigh_many
// 28.5; 32 of up to 2000 27.9 and 29.3; 8 of up to 300 7.6 and 6.8.  20 rows: 24.2 and 24.0, 28.1 and 26.9, 7.6 and 6.4.)
constexpr int WW_ROWS = 24;

// A sequence's place in the call, clamped to its range; `bad` is set where that changed something.
struct Seq {
    int len, q0, qn;
};
__device__ __forceinline__ Seq weigh_seq(const WeighArgs &a, int s, bool &bad) {
    Seq x;
    const int len = a.length[s], r0 = a.q_start ? a.q_start[s] : s, r1 = a.q_start ? a.q_start[s + 1] : s + 1;
    x.len = clampi(len, 0, a.max_length);
    x.q0 = clampi(r0, 0, a.q_tokens);
    const int q1 = clampi(r1, x.q0, a.q_tokens);
    x.qn = q1 - x.q0;
    bad |= x.len != len || x.q0 != r0 || q1 != r1 || (s == 0 && r0 != 0) || (s == a.seqs - 1 && r1 != a.q_tokens);
    return x;
}

// Items -- pieces of 2^SHIFT tokens of one head -- in the order (sequence, head, piece).  All lanes of a warp
// hold the same values but `end`, the running count of items behind sequence base + lane.
template <int SHIFT>
struct Items {
    int base;         // first sequence of the window
    long long before;  // items before it
    long long end;

    __device__ __forceinline__ void window(const WeighArgs &a) {
        const int s = base + (threadIdx.x & 31);
        bool bad = false;
        long long n = s < a.seqs ? (long long)((weigh_seq(a, s, bad).len + (1 << SHIFT) - 1) >> SHIFT) * a.hkv : 0;
        if (bad) raise_error(a.err, ERR_PAGE);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long p = __shfl_up_sync(0xFFFFFFFFu, n, o);
            if ((threadIdx.x & 31) >= o) n += p;
        }
        end = before + n;
    }
    __device__ __forceinline__ void start(const WeighArgs &a) {
        base = 0;
        before = 0;
        window(a);
    }
    // All items; the window is the last one's then.
    __device__ __forceinline__ long long total(const WeighArgs &a) {
        for (;;) {
            const long long n = __shfl_sync(0xFFFFFFFFu, end, 31);
            if (base + 32 >= a.seqs) return n;
            base += 32;
            before = n;
            window(a);
        }
    }
    // The sequence of item x (not before an item found earlier; less than the total), and the items before it.
    __device__ __forceinline__ int find(const WeighArgs &a, long long x, long long &at) {
        for (;;) {
            const long long n = __shfl_sync(0xFFFFFFFFu, end, 31);
            if (x < n || base + 32 >= a.seqs) break;
            base += 32;
            before = n;
            window(a);
        }
        const int i = min(__popc(__ballot_sync(0xFFFFFFFFu, end <= x)), 31);
        at = i ? __shfl_sync(0xFFFFFFFFu, end, i - 1) : before;
        return base + i;
    }
};

__device__ __forceinline__ void cp_async(void *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}

// The keys of 16 tokens, one block or slot group of a page, as a lane of the A operand holds them (tokens g
// and g + 8), and their products with eight queries.
template <typename T, int D, bool PACKED>
struct Keys;
template <typename T, int D>
struct Keys<T, D, false> {
    uint4 w[2][D / 32];  // channels 32 b + 8 t .. + 7
    // A ring's place: rows 64 bytes past a multiple of 128 apart, so that the lanes of two rows meet no bank twice.
    static constexpr int ROW = 2 * D + 64, PLACE = 16 * ROW, AHEAD = 4, TURN = 2, CTAS = 2;
    // row: of the first of the tokens in the pool's order of pages, heads and places
    static __device__ __forceinline__ void copy(unsigned char *to, const WeighArgs &a, int row) {
        const int lane = threadIdx.x & 31;
        constexpr int CH = D / 8, RPT = 32 / CH;  // chunks of a row, rows a turn
        const unsigned char *p = reinterpret_cast<const unsigned char *>(a.pages) + (long long)row * (4 * D) + lane / CH * (4 * D) + lane % CH * 16;
        to += lane / CH * ROW + lane % CH * 16;
#pragma unroll
        for (int x = 0; x < 16 / RPT; ++x) cp_async(to + x * RPT * ROW, p + x * RPT * (4 * D));
    }
    __device__ __forceinline__ void load(const unsigned char *from) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int b = 0; b < D / 32; ++b) w[i][b] = *reinterpret_cast<const uint4 *>(from + (g + 8 * i) * ROW + 64 * b + 16 * t);
    }
    __device__ __forceinline__ void load(const WeighArgs &a, int id, int head, int tok) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const uint16_t *p = reinterpret_cast<const uint16_t *>(a.pages) +
                            ((((long long)id * a.hkv + head) << a.page_shift) + (tok & ((1 << a.page_shift) - 1)) + g) * (2 * D) + 8 * t;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int b = 0; b < D / 32; ++b) w[i][b] = ldg_stream(reinterpret_cast<const uint4 *>(p + i * 8 * 2 * D + 32 * b));
    }
    struct Queries {
        uint4 b[D / 32];
        __device__ __forceinline__ void load(const uint16_t *row, uint32_t sign) {
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
                b[x] = make_uint4(0u, 0u, 0u, 0u);
                if (row) b[x] = *reinterpret_cast<const uint4 *>(row + 32 * x + 8 * (threadIdx.x & 3));
                b[x] = make_uint4(b[x].x ^ sign, b[x].y ^ sign, b[x].z ^ sign, b[x].w ^ sign);
            }
        }
    };
    struct Ready {
        __device__ __forceinline__ void make(const Keys &) {}
    };
    static __device__ __forceinline__ float unit(const Queries &, float c, int) { return c; }
    static __device__ __forceinline__ void logits(float (&s)[4], const Keys &k, const Ready &, const Queries &q) {
        float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // odd k-steps: shorter chains
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = 0.0f;
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
            const uint32_t a0[4] = {k.w[0][b].x, k.w[1][b].x, k.w[0][b].y, k.w[1][b].y};
            const uint32_t a1[4] = {k.w[0][b].z, k.w[1][b].z, k.w[0][b].w, k.w[1][b].w};
            T::mma(s, a0, q.b[b].x, q.b[b].y);
            T::mma(o, a1, q.b[b].z, q.b[b].w);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += o[e];
    }
};
template <typename T, int D>
struct Keys<T, D, true> {
    typedef typename Q4Vec<D>::Key Vec;
    Vec code[2], par[2];
    uint32_t mine[2];  // floor and step of the lane's group
    static constexpr int PLACE = Q4<D>::SIDE, AHEAD = 8, TURN = 1, CTAS = 4;
    static __device__ __forceinline__ const unsigned char *at(const WeighArgs &a, int id, int head, int tok) {
        return reinterpret_cast<const unsigned char *>(a.pages) +
               (((((long long)id * a.hkv + head) << a.page_shift) + (tok & ((1 << a.page_shift) - 1))) >> 4) * Q4<D>::BLOCK;
    }
    static __device__ __forceinline__ void copy(unsigned char *to, const WeighArgs &a, int row) {
        const int lane = threadIdx.x & 31;
        const unsigned char *p = reinterpret_cast<const unsigned char *>(a.pages) + (long long)(row >> 4) * Q4<D>::BLOCK + lane * 16;
        to += lane * 16;
#pragma unroll
        for (int x = 0; x < PLACE / 16; x += 32)
            if (x + 32 <= PLACE / 16 || x + lane < PLACE / 16) cp_async(to + x * 16, p + x * 16);
    }
    __device__ __forceinline__ void load(const WeighArgs &a, int id, int head, int tok) { load(at(a, id, head, tok)); }
    __device__ __forceinline__ void load(const unsigned char *p) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const unsigned char *q = p + Q4<D>::PARS + (g + 8 * i) * Q4<D>::PAR;
            code[i] = *reinterpret_cast<const Vec *>(p + (g + 8 * i) * Q4<D>::CODE + t * (Q4<D>::CODE / 4));
            par[i] = *reinterpret_cast<const Vec *>(q);
            mine[i] = *reinterpret_cast<const uint32_t *>(q + (t & (D / 32 - 1)) * 4);
        }
    }
    typedef Queries8<T, D> Queries;
    struct Ready {
        KeyCodes<D> kc;
        __device__ __forceinline__ void make(const Keys &k) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                kc.codes(i, k.code[i]);
                kc.scales(i, k.par[i], k.mine[i]);
            }
        }
    };
    static __device__ __forceinline__ float unit(const Queries &q, float c, int e) { return q.units(c, e); }
    static __device__ __forceinline__ void logits(float (&s)[4], const Keys &, const Ready &r, const Queries &q) { 
        q4_logits<D>(s, r.kc, q.sum[0], q.sum[1], [&](int j) { return q.at(j); });
    }
};

// Adds the weights of a product's logits: z[i] of token g + 8 i, of rows 2 t and 2 t + 1, whose lse2 is +infinity
// where a row counts nothing.
__device__ __forceinline__ void add_weights(float (&z)[2], const float (&s)[4], const float (&c)[2], const float (&lse2)[2]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e >> 1] += exp2_fast(fmaf(s[e], c[e & 1], -lse2[e & 1]));
}
// The same where not every row sees every token: tok with the lane's g in it, rows see tokens before lim[e].
__device__ __forceinline__ void add_weights(float (&z)[2], const float (&s)[4], const float (&c)[2], const float (&lse2)[2], int tok, const int (&lim)[2]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float w = exp2_fast(fmaf(s[e], c[e & 1], -lse2[e & 1]));
        z[e >> 1] += tok + 8 * (e >> 1) < lim[e & 1] ? w : 0.0f;
    }
}

// lse in units of log 2; a row that saw nothing counts nothing.  (Its weights are 2^(s - infinity) = 0 where its channels are
// numbers.  They need not be, in a padded batch, so it is masked as well: where a tile has such a row, it goes the way
// of those whose rows do not see every token.)
__device__ __forceinline__ float lse_log2(float lse) { return lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f; }

__device__ __forceinline__ int page_of(const WeighArgs &a, int s, int tok) {
    const int id = a.table[(long long)s * a.stride + (tok >> a.page_shift)];
    if (id >= 0 && id < a.num_pages) return id;
    raise_error(a.err, ERR_PAGE);
    return 0;
}

// Places behind the sequences' lengths, where out is not in: warps take pieces of 512 places in turn, all of whose
// loads are on their way together.
__device__ __forceinline__ void weigh_behind(const WeighArgs &a, long long warp, long long warps) {
    if (a.in == a.out) return;
    const int lane = threadIdx.x & 31, each = (a.places + 511) / 512;
    const long long pieces = (long long)a.seqs * a.hkv * each;
    for (long long x = warp; x < pieces; x += warps) {
        const long long u = x / each;
        const int i0 = (int)(x - u * each) * 512, len = clampi(a.length[u / a.hkv], 0, a.max_length);
        if (i0 + 512 <= len) continue;
        const long long row = u * a.places;
        float v[16];
#pragma unroll
        for (int y = 0; y < 16; ++y) {
            const int i = i0 + y * 32 + lane;
            v[y] = a.in && i >= len && i < a.places ? a.in[row + i] : 0.0f;
        }
#pragma unroll
        for (int y = 0; y < 16; ++y) {
            const int i = i0 + y * 32 + lane;
            if (i >= len && i < a.places) a.out[row + i] = v[y];
        }
    }
}

template <typename T, int D, bool PACKED>
__global__ void __launch_bounds__(WF_NT, PACKED ? 4 : 2) k_weigh_few(const __grid_constant__ WeighArgs a) {
    using K = Keys<T, D, PACKED>;
    constexpr int NB = K::AHEAD, NU = K::TURN;  // blocks on their way and worked on, and of them worked on
    extern __shared__ __align__(16) unsigned char wf_smem[];
    unsigned char *ring = wf_smem + (threadIdx.x >> 5) * (NB * K::PLACE);
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const long long warp = (long long)blockIdx.x * (WF_NT / 32) + (threadIdx.x >> 5), warps = (long long)gridDim.x * (WF_NT / 32);
    const uint32_t sign = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
    const float c = fabsf(a.scale_log2);
    Items<4> items;
    items.start(a);
    const long long total = items.total(a);
    if (items.base) items.start(a);
    const long long x1 = (warp + 1) * total / warps;
    long long x = warp * total / warps;
    while (x < x1) {
        long long at;
        const int s = items.find(a, x, at);
        bool bad = false;
        const Seq sq = weigh_seq(a, s, bad);
        const int blocks = (sq.len + 15) >> 4;
        if (blocks == 0) break;  // (lengths changed under the kernel)
        const int head = (int)((x - at) / blocks), b0 = (int)((x - at) - (long long)head * blocks);
        if (head >= a.hkv) break;
        const int b1 = (int)min((long long)blocks, b0 + (x1 - x));
        x += b1 - b0;

        const int rows = sq.qn << a.g_shift, first = sq.len - sq.qn + 1;  // tokens the first query sees
        typename K::Queries q;
        float lse2[2], unit[2];
        int lim[2];
        bool dead = false;  // some of the rows count nothing
        auto take = [&](int r0) {  // rows r0 .. r0 + 7
            const int r = r0 + g, jj = r >> a.g_shift;
            q.load(r < rows ? a.q + (long long)(sq.q0 + jj) * a.q_ts + (long long)((head << a.g_shift) + r - (jj << a.g_shift)) * a.q_hs : nullptr, sign);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                unit[e] = K::unit(q, c, e);
                const int y = r0 + 2 * t + e, j = y >> a.g_shift;
                lim[e] = first + j;
                lse2[e] = y < rows ? lse_log2(a.lse[((long long)(sq.q0 + j) * a.hkv << a.g_shift) + (head << a.g_shift) + y - (j << a.g_shift)]) : INFINITY;
                if (lse2[e] == INFINITY) lim[e] = 0;
            }
            dead = __any_sync(0xFFFFFFFFu, (lim[0] == 0 && r0 + 2 * t < rows) || (lim[1] == 0 && r0 + 2 * t + 1 < rows));
        };
        // Rows in the pool of 32 blocks at a time, one a lane.
        int ids0 = b0, ids = 0;
        auto fetch = [&](int b) {
            ids0 = b;
            const int tok = (b + lane) * 16;
            const int id = b + lane < b1 ? page_of(a, s, tok) : 0;
            ids = ((id * a.hkv + head) << a.page_shift) + (tok & ((1 << a.page_shift) - 1));
        };
        fetch(b0);
        unsigned char *to = ring;  // place of the next copy
        auto copy = [&](int b) {
            if (b < b1) {
                if (b >= ids0 + 32) fetch(b);
                K::copy(to, a, __shfl_sync(0xFFFFFFFFu, ids, b - ids0));
            }
            to = to == ring + (NB - 1) * K::PLACE ? ring : to + K::PLACE;
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // Lanes t = 0 and 1 have the sums of tokens g and g + 8.
        const int odd = t & 1;
        const long long mine = ((long long)s * a.hkv + head) * a.places + b0 * 16 + g + 8 * odd;
        const float *in = a.in ? a.in + mine : nullptr;
        float *out = a.out + mine;
        int left = t < 2 ? sq.len - (b0 * 16 + g + 8 * odd) : 0;  // tokens from this lane's on
        __syncwarp();  // nobody reads the last unit's blocks any more
#pragma unroll 1
        for (int u = 0; u < NB - NU; ++u) copy(b0 + u);
        take(0);
        const unsigned char *from = ring;
        // NU blocks a turn: chains of products and exponentials side by side.  (What the place of a block that is not
        // there holds goes nowhere: left says so.)
#pragma unroll 1
        for (int b = b0; b < b1; b += NU) {
            __syncwarp();  // nor the last blocks
#pragma unroll
            for (int u = 0; u < NU; ++u) copy(b + NB - NU + u);
            asm volatile("cp.async.wait_group %0;" ::"n"(NB - NU) : "memory");
            __syncwarp();
            K key[NU];
            typename K::Ready ready[NU];
            float was[NU], z[NU][2];
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                was[u] = in && left > 16 * u && b + u < b1 ? in[16 * u] : 0.0f;
                key[u].load(from);
                from = from == ring + (NB - 1) * K::PLACE ? ring : from + K::PLACE;
                ready[u].make(key[u]);
                z[u][0] = z[u][1] = 0.0f;
            }
            // from the first row on that sees any of the blocks
            const int r1 = max(0, b * 16 - first + 1) << a.g_shift;
#pragma unroll 1
            for (int r0 = r1 & ~7; r0 < rows; r0 += 8) {
                if (rows > 8) take(r0);
                float lg[NU][4];
#pragma unroll
                for (int u = 0; u < NU; ++u) K::logits(lg[u], key[u], ready[u], q);
                if (b * 16 + 16 * NU <= first + (r0 >> a.g_shift) && !dead) {
#pragma unroll
                    for (int u = 0; u < NU; ++u) add_weights(z[u], lg[u], unit, lse2);
                } else {
#pragma unroll
                    for (int u = 0; u < NU; ++u) add_weights(z[u], lg[u], unit, lse2, (b + u) * 16 + g, lim);
                }
            }
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                float sum = odd ? z[u][1] : z[u][0];
                sum += __shfl_xor_sync(0xFFFFFFFFu, odd ? z[u][0] : z[u][1], 1);
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
                if (left > 16 * u && b + u < b1) out[16 * u] = was[u] + sum;
            }
            if (in) in += 16 * NU;
            out += 16 * NU;
            left -= 16 * NU;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    weigh_behind(a, warp, warps);
}

// A row of queries in shared memory: 64 bytes past a multiple of 128, so that two rows' 64 bytes are in
// different banks.
template <int D>
struct ManyLayout {
    static constexpr int ROW = 2 * D + 64;
    static constexpr int LSE = 2 * WM_ROWS * ROW;                     // float [2][WM_ROWS]
    static constexpr int ITEM = LSE + 2 * WM_ROWS * 4;
    static constexpr int BYTES = ITEM + 16;
};

template <typename T, int D, bool PACKED>
__global__ void __launch_bounds__(WM_NT, PACKED ? 3 : 4) k_weigh_many(const __grid_constant__ WeighArgs a) {
    using K = Keys<T, D, PACKED>;
    using LY = ManyLayout<D>;
    extern __shared__ __align__(16) unsigned char wm_smem[];
    float *lse_at = reinterpret_cast<float *>(wm_smem + LY::LSE);
    volatile int *item = reinterpret_cast<volatile int *>(wm_smem + LY::ITEM);  // sequence (-1: none), head, piece
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t sign = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
    const float c = fabsf(a.scale_log2);
    Items<7> items;
    long long total = 0;
    if (warp == 0) {
        items.start(a);
        total = items.total(a);
        if (items.base) items.start(a);
    }
    for (long long x = blockIdx.x;; x += gridDim.x) {
        __syncthreads();
        if (warp == 0) {
            int s = -1, head = 0, piece = 0;
            if (x < total) {
                long long at;
                s = items.find(a, x, at);
                bool bad = false;
                const int pieces = (weigh_seq(a, s, bad).len + WM_TOKENS - 1) / WM_TOKENS;
                head = pieces ? (int)((x - at) / pieces) : a.hkv;
                piece = (int)((x - at) - (long long)head * pieces);
                if (head >= a.hkv) s = -1;  // (lengths changed under the kernel)
            }
            if (lane == 0) {
                item[0] = s;
                item[1] = head;
                item[2] = piece;
            }
        }
        __syncthreads();
        const int s = item[0], head = item[1];
        if (s < 0) break;
        bool bad = false;
        const Seq sq = weigh_seq(a, s, bad);
        const int rows = sq.qn << a.g_shift, first = sq.len - sq.qn + 1;
        const int piece0 = item[2] * WM_TOKENS, tok0 = piece0 + warp * 32;
        const int ra = (max(0, piece0 - first + 1) << a.g_shift) & ~7;  // the first row that sees any of the piece

        auto stage = [&](int r0, int buf) {
#pragma unroll
            for (int y = 0; y < WM_ROWS * D / 8 / WM_NT; ++y) {
                const int at = tid + y * WM_NT, r = at / (D / 8), ch = at % (D / 8) * 8, rr = r0 + r;
                if (rr < rows) {
                    const int jj = rr >> a.g_shift;
                    const uint16_t *src = a.q + (long long)(sq.q0 + jj) * a.q_ts + (long long)((head << a.g_shift) + rr - (jj << a.g_shift)) * a.q_hs + ch;
                    cp_async(wm_smem + (buf * WM_ROWS + r) * LY::ROW + ch * 2, src);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (tid < WM_ROWS) {
                const int rr = r0 + tid, jj = rr >> a.g_shift;
                lse_at[buf * WM_ROWS + tid] =
                    rr < rows ? lse_log2(a.lse[((long long)(sq.q0 + jj) * a.hkv << a.g_shift) + (head << a.g_shift) + rr - (jj << a.g_shift)]) : INFINITY;
            }
        };
        if (ra < rows) stage(ra, 0);
        K k[2];
        typename K::Ready ready[2];
        float z[2][2] = {}, was[2][2] = {};
        const long long row = ((long long)s * a.hkv + head) * a.places;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            if (tok0 + 16 * m < sq.len) {
                k[m].load(a, page_of(a, s, tok0 + 16 * m), head, tok0 + 16 * m);
                ready[m].make(k[m]);
            } else {
                k[m] = K{};
                ready[m].make(k[m]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int tok = tok0 + 16 * m + g + 8 * i;
                if (a.in && t == 0 && tok < sq.len) was[m][i] = a.in[row + tok];
            }
        }
        int buf = 0;
#pragma unroll 1
        for (int r0 = ra; r0 < rows; r0 += WM_ROWS, buf ^= 1) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();  // these rows are there, and nobody reads the other buffer any more
            if (r0 + WM_ROWS < rows) stage(r0 + WM_ROWS, buf ^ 1);
            const unsigned char *qb = wm_smem + buf * WM_ROWS * LY::ROW;
#pragma unroll 1
            for (int n = 0; n < WM_ROWS; n += 8) {
                if (r0 + n >= rows || tok0 >= sq.len) break;
                const int seen = first + ((min(rows, r0 + n + 8) - 1) >> a.g_shift);  // tokens the last of the rows sees
                if (seen <= tok0) continue;
                typename K::Queries q;
                q.load(reinterpret_cast<const uint16_t *>(qb + (n + g) * LY::ROW), sign);
                float lse2[2], unit[2];
                int lim[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    unit[e] = K::unit(q, c, e);
                    lse2[e] = lse_at[buf * WM_ROWS + n + 2 * t + e];
                    // (what is in the place of a row that is not there may be no number; its lse is infinite)
                    lim[e] = lse2[e] != INFINITY ? first + ((r0 + n + 2 * t + e) >> a.g_shift) : 0;
                }
                const bool live = __all_sync(0xFFFFFFFFu, lse2[0] != INFINITY && lse2[1] != INFINITY);
                const int all = live ? first + ((r0 + n) >> a.g_shift) : 0;  // tokens every one of the rows sees
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    float lg[4];
                    K::logits(lg, k[m], ready[m], q);
                    if (tok0 + 16 * m + 16 <= all) add_weights(z[m], lg, unit, lse2);
                    else add_weights(z[m], lg, unit, lse2, tok0 + 16 * m + g, lim);
                }
            }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                z[m][i] += __shfl_xor_sync(0xFFFFFFFFu, z[m][i], 1);
                z[m][i] += __shfl_xor_sync(0xFFFFFFFFu, z[m][i], 2);
                const int tok = tok0 + 16 * m + g + 8 * i;
                if (t == 0 && tok < sq.len) a.out[row + tok] = was[m][i] + z[m][i];
            }
    }
    weigh_behind(a, (long long)blockIdx.x * (WM_NT / 32) + warp, (long long)gridDim.x * (WM_NT / 32));
}

constexpr int WW_GROUPS = 4;            // of four warps that add up: two a half
constexpr int WW_NT = WW_GROUPS * 128 + 64;
constexpr int WW_MMA = WW_GROUPS * 4, WW_COPY = WW_MMA + 1;  // warps: issues the products, copies
constexpr int WW_ITEMS = 4;             // items on their way
constexpr int WW_TOKENS = 256;          // of an item, in halves of 128

struct WideItem {
    int s, head, piece0;  // s < 0: the last one was the one before
    int len, first, rows, q0;
    int n0, tiles;        // the first row tile that sees any of the piece, and how many
    int halves;           // with tokens
};

template <int D>
struct WeighWide {
    static constexpr int HALVES = D / 64;         // of the channels
    static constexpr int BOX = 128 * 128;         // 128 rows x 64 channels
    static constexpr int TILE = HALVES * BOX;
    // Halves of items' keys in their ring, and query tiles in theirs.  (4 and 2: four prompts of 8192 by 64 queries 29.7 us, by
    // 2048 641; 3 and 3: 28.7, 584; 2 and 4: 29.3, 561.)  No two CTAs fit on an SM, nor its tensor memory.
    static constexpr int NK = 3, NQ = D == 128 ? 3 : 6;
    static constexpr int K = 0;                   // [NK][TILE]
    static constexpr int Q = NK * TILE;           // [NQ][TILE]
    static constexpr int LSE = Q + NQ * TILE;                // float [warps of the groups][128]: less lse
    static constexpr int PART = LSE + WW_GROUPS * 4 * 512;   // float [WW_ITEMS][2][128]: a half's second group's sums
    static constexpr int ITEM = PART + WW_ITEMS * 2 * 512;
    static constexpr int BARS = (ITEM + WW_ITEMS * (int)sizeof(WideItem) + 7) / 8 * 8;
    // item full, empty [WW_ITEMS], part [WW_ITEMS][2]; keys full, empty [NK]; queries full, empty [NQ]; S full, empty [4]; drain
    static constexpr int NBARS = 4 * WW_ITEMS + 2 * NK + 2 * NQ + 8 + 1;
    static constexpr int BYTES = BARS + NBARS * 8 + 16;
    static_assert(BYTES <= 227 * 1024, "shared memory of a CTA");
};

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ unsigned long long two(float x, float y) {
    unsigned long long v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
    return v;
}

__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ void add2(unsigned long long &v, float x, float y) {
    const unsigned long long w = two(x, y);
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(w));
}

template <bool BF, int D>
__global__ void __launch_bounds__(WW_NT, 1)
    k_weigh_wide(const __grid_constant__ WeighArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qmap) {
    using LY = WeighWide<D>;
    extern __shared__ __align__(1024) unsigned char ww_smem[];
    uint64_t *item_full = reinterpret_cast<uint64_t *>(ww_smem + LY::BARS), *item_empty = item_full + WW_ITEMS;
    uint64_t *part_full = item_empty + WW_ITEMS, *k_full = part_full + 2 * WW_ITEMS, *k_empty = k_full + LY::NK;
    uint64_t *q_full = k_empty + LY::NK, *q_empty = q_full + LY::NQ, *s_full = q_empty + LY::NQ, *s_empty = s_full + 4;
    uint64_t *drain = s_empty + 4;
    uint32_t *tmem_at = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_at + 1);
    WideItem *items = reinterpret_cast<WideItem *>(ww_smem + LY::ITEM);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < WW_ITEMS; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], WW_GROUPS * 4 + 1);  // the warps that read it
            mbar_init(&part_full[2 * i], 4);
            mbar_init(&part_full[2 * i + 1], 4);
        }
        for (int i = 0; i < LY::NK; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < LY::NQ; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], 4);
        }
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *abort = 0;
    }
    if (warp == WW_MMA) tmem_alloc(tmem_at, 512);
    if (warp == WW_COPY && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&qmap)) : "memory");
    }
    pdl_wait();
    pdl_trigger();
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tm = *tmem_at;
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        if (__all_sync(0xFFFFFFFFu, paged_wait(smem_addr(bar), parity, abort, a.wait_ns))) return true;
        if (lane == 0) {
            *abort = 1;
            raise_error(a.err, ERR_TIMEOUT);
        }
        return false;
    };

    if (warp == WW_COPY) {
        Items<8> walk;
        walk.start(a);
        const long long total = walk.total(a);
        if (walk.base) walk.start(a);
        const int box = min(1 << a.page_shift, 128);
        int tiles = 0, keys = 0;  // so far: query tiles, halves of keys
        bool go = true;
        Seq sq{};
        int sq_of = -1;
        // Item n, and in lane i the page of its i-th box (as the table has it: it is on its way, and looked at a turn later).
        auto prepare = [&](int n, WideItem &it, int &id) {
            const long long x = blockIdx.x + (long long)n * gridDim.x;
            it.s = -1;
            id = 0;
            if (x >= total) return;
            long long at;
            it.s = walk.find(a, x, at);
            if (it.s != sq_of) {
                bool bad = false;
                sq = weigh_seq(a, it.s, bad);
                sq_of = it.s;
            }
            const int pieces = (sq.len + WW_TOKENS - 1) / WW_TOKENS;
            it.head = pieces ? (int)((x - at) / pieces) : a.hkv;
            if (it.head >= a.hkv) {  // lengths changed under the kernel
                it.s = -1;
                return;
            }
            it.piece0 = (int)((x - at) - (long long)it.head * pieces) * WW_TOKENS;
            it.halves = sq.len - it.piece0 > 128 ? 2 : 1;
            it.len = sq.len;
            it.q0 = sq.q0;
            it.rows = sq.qn << a.g_shift;
            it.first = sq.len - sq.qn + 1;
            it.n0 = (max(0, it.piece0 - it.first + 1) << a.g_shift) >> 7;
            it.tiles = max(0, (it.rows + 127) / 128 - it.n0);
            const int tok = it.piece0 + lane * box;
            if (it.tiles && lane * box < WW_TOKENS && tok < it.len) id = a.table[(long long)it.s * a.stride + (tok >> a.page_shift)];
        };
        WideItem it, after;
        int id, id_after;
        prepare(0, after, id_after);
        for (int n = 0; go; ++n) {
            it = after;
            id = id_after;
            if (it.s >= 0) prepare(n + 1, after, id_after);
            const int i = n % WW_ITEMS;
            if (n >= WW_ITEMS && !(go = wait(&item_empty[i], (uint32_t)(n / WW_ITEMS - 1)))) break;
            if (lane == 0) {
                items[i] = it;
                mbar_arrive(&item_full[i]);
            }
            if (it.s < 0) break;
            if (it.tiles == 0) continue;
            // The keys of the tokens that there are; what the other rows hold stays in its own lanes.
            for (int m = 0; m < it.halves && go; ++m, ++keys) {
                const int kb = keys % LY::NK, tok0 = it.piece0 + 128 * m, pages = (min(128, it.len - tok0) + box - 1) / box;
                if (keys >= LY::NK && !(go = wait(&k_empty[kb], (uint32_t)(keys / LY::NK - 1)))) break;
                const int tok = tok0 + lane * box;
                int page = __shfl_sync(0xFFFFFFFFu, id, (lane + (m ? 128 / box : 0)) & 31);
                if (lane < pages && (page < 0 || page >= a.num_pages)) {
                    raise_error(a.err, ERR_PAGE);
                    page = 0;
                }
                if (lane == 0) mbar_expect_tx(&k_full[kb], (uint32_t)(pages * box * 2 * D));
                __syncwarp();
                if (lane < pages && !(a.stall && blockIdx.x == 0 && keys == 0)) {
                    const int y = ((page * a.hkv + it.head) << a.page_shift) + (tok & ((1 << a.page_shift) - 1));
#pragma unroll
                    for (int b = 0; b < LY::HALVES; ++b) tma_load_2d(ww_smem + LY::K + kb * LY::TILE + b * LY::BOX + lane * box * 128, &kmap, b * 64, y, &k_full[kb]);
                }
                __syncwarp();
            }
            if (!go) break;
            for (int t = 0; t < it.tiles; ++t, ++tiles) {
                const int st = tiles % LY::NQ;
                if (tiles >= LY::NQ && !(go = wait(&q_empty[st], (uint32_t)(tiles / LY::NQ - 1)))) break;
                if (lane == 0) {
                    mbar_expect_tx(&q_full[st], LY::TILE);
                    // (rows behind the last query of the call come as zeros, those of other sequences count nothing)
#pragma unroll
                    for (int b = 0; b < LY::HALVES; ++b)
                        tma_load_3d(ww_smem + LY::Q + st * LY::TILE + b * LY::BOX, &qmap, b * 64, it.head << a.g_shift, it.q0 + ((it.n0 + t) << (7 - a.g_shift)), &q_full[st]);
                }
                __syncwarp();
            }
        }
        if (lane == 0) {
            // The copies in flight land here also where another warp's wait ran out.
            for (int i = max(0, keys - LY::NK); i < keys; ++i) mbar_wait_bounded(&k_full[i % LY::NK], (uint32_t)((i / LY::NK) & 1), a.wait_ns);
            for (int i = max(0, tiles - LY::NQ); i < tiles; ++i) mbar_wait_bounded(&q_full[i % LY::NQ], (uint32_t)((i / LY::NQ) & 1), a.wait_ns);
        }
        __syncwarp();
    } else if (warp == WW_MMA) {
        const uint32_t it1 = elect_one();
        const uint64_t kd = smem_desc(smem_addr(ww_smem + LY::K), LY::BOX, 1024), qd = smem_desc(smem_addr(ww_smem + LY::Q), LY::BOX, 1024);
        constexpr uint32_t IS = mma_desc(128, 128, BF, false);
        int tiles = 0, keys = 0, used[2] = {0, 0};  // so far: query tiles, halves of keys, and tiles of either half
        bool go = true;
        for (int n = 0; go; ++n) {
            const int i = n % WW_ITEMS;
            if (!(go = wait(&item_full[i], (uint32_t)(n / WW_ITEMS)))) break;
            const int s = items[i].s, count = items[i].tiles, halves = items[i].halves;
            __syncwarp();
            if (s < 0) break;
            if (lane == 0) mbar_arrive(&item_empty[i]);
            if (count == 0) continue;
            for (int t = 0; t < count && go; ++t, ++tiles) {
                const int st = tiles % LY::NQ;
                if (!(go = wait(&q_full[st], (uint32_t)(tiles / LY::NQ)))) break;
                const uint64_t q0 = qd + (uint32_t)(st * (LY::TILE >> 4));
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    if (m >= halves || !go) continue;
                    const int kb = (keys + m) % LY::NK, acc = 2 * m + (used[m] & 1);
                    if (t == 0 && !(go = wait(&k_full[kb], (uint32_t)((keys + m) / LY::NK)))) continue;
                    if (used[m] >= 2 && !(go = wait(&s_empty[acc], (uint32_t)(used[m] / 2 - 1)))) continue;
                    tcgen05_after_sync();
                    const uint64_t k0 = kd + (uint32_t)(kb * (LY::TILE >> 4));
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        const int off = ((x / 4) * LY::BOX + (x % 4) * 32) >> 4;
                        mma_ss(tm + acc * 128, k0 + off, q0 + off, IS, x > 0, it1);
                    }
                    tcgen05_commit(&s_full[acc], it1);
                    if (t == count - 1) tcgen05_commit(&k_empty[kb], it1);
                    ++used[m];
                }
                if (go) tcgen05_commit(&q_empty[st], it1);
            }
            keys += halves;
        }
        // Nothing is in flight when the CTA gives its tensor memory back.
        tcgen05_commit(drain, it1);
        if (!mbar_wait_bounded(drain, 0u, a.wait_ns)) raise_error(a.err, ERR_TIMEOUT);
        __syncwarp();
    } else {
        const int m = (warp >> 2) & 1, turn = warp >> 3, r = (warp & 3) * 32 + lane;  // half, which tiles of it, token
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        float *lse_at = reinterpret_cast<float *>(ww_smem + LY::LSE) + warp * 128, *part = reinterpret_cast<float *>(ww_smem + LY::PART);
        const float c = a.scale_log2;
        const unsigned long long cc = two(c, c);
        int tiles = 0;  // of this half so far
        bool go = true;
        for (int n = 0; go; ++n) {
            const int i = n % WW_ITEMS;
            if (!(go = wait(&item_full[i], (uint32_t)(n / WW_ITEMS)))) break;
            const WideItem it = items[i];
            if (it.s < 0) break;
            if (m >= it.halves) {
                __syncwarp();
                if (lane == 0) {
                    if (turn) mbar_arrive(&part_full[2 * i + m]);  // (as of every item)
                    mbar_arrive(&item_empty[i]);
                }
                continue;
            }
            const int tok = it.piece0 + 128 * m + r;
            const bool mine = tok < it.len;
            const long long at = ((long long)it.s * a.hkv + it.head) * a.places + tok;
            const int t0 = (turn ^ tiles) & 1;  // this group's first tile; that with the item's first one joins
            const float was = t0 == 0 && mine && a.in ? a.in[at] : 0.0f;
            // lse of the rows of tile t, four a lane; rows that are not there count nothing.  (As it lies: what is not
            // used until the next tile is not waited for in this one.)
            float lse[4];
            auto fetch = [&](int t) {
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int row = ((it.n0 + t) << 7) + 4 * lane + y, j = row >> a.g_shift;
                    lse[y] = -INFINITY;
                    if (row < it.rows) lse[y] = a.lse[((long long)(it.q0 + j) * a.hkv << a.g_shift) + (it.head << a.g_shift) + row - (j << a.g_shift)];
                }
            };
            if (t0 < it.tiles) fetch(t0);
            unsigned long long sum[4] = {0ull, 0ull, 0ull, 0ull};  // pairs
            for (int t = t0; t < it.tiles; t += 2) {
                __syncwarp();
                const bool live = lse[0] != -INFINITY && lse[1] != -INFINITY && lse[2] != -INFINITY && lse[3] != -INFINITY;
                reinterpret_cast<float4 *>(lse_at)[lane] = make_float4(-lse_log2(lse[0]), -lse_log2(lse[1]), -lse_log2(lse[2]), -lse_log2(lse[3]));
                __syncwarp();
                if (t + 2 < it.tiles) fetch(t + 2);
                const int acc = 2 * m + turn;
                if (!(go = wait(&s_full[acc], (uint32_t)((tiles + t) / 2)))) break;
                tcgen05_after_sync();
                // rows from `from` on see this token; those that are not there have an infinite lse
                const int row0 = (it.n0 + t) << 7, from = (max(0, tok - it.first + 1) << a.g_shift) - row0;
                const bool all = __all_sync(0xFFFFFFFFu, from <= 0 && live);
#pragma unroll 1
                for (int x = 0; x < 128; x += 32) {
                    uint32_t u[32];
                    tmem_ld32(u, tm + lanes + acc * 128 + x);
                    if (x == 96) {  // all of it has been read
                        tcgen05_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s_empty[acc]);
                    }
                    if (all) {
#pragma unroll
                        for (int y = 0; y < 32; y += 4) {
                            const ulonglong2 l = *reinterpret_cast<const ulonglong2 *>(lse_at + x + y);
                            const unsigned long long e0 = fma2(two(__uint_as_float(u[y]), __uint_as_float(u[y + 1])), cc, l.x);
                            const unsigned long long e1 = fma2(two(__uint_as_float(u[y + 2]), __uint_as_float(u[y + 3])), cc, l.y);
                            add2(sum[y / 2 & 2], exp2_fast(__uint_as_float((uint32_t)e0)), exp2_fast(__uint_as_float((uint32_t)(e0 >> 32))));
                            add2(sum[(y / 2 & 2) + 1], exp2_fast(__uint_as_float((uint32_t)e1)), exp2_fast(__uint_as_float((uint32_t)(e1 >> 32))));
                        }
                    } else {
#pragma unroll
                        for (int y = 0; y < 32; ++y) {
                            const float l = lse_at[x + y], e = exp2_fast(fmaf(__uint_as_float(u[y]), c, l));
                            add2(sum[y & 3], x + y < from || l == -INFINITY ? 0.0f : e, 0.0f);
                        }
                    }
                }
            }
            if (!go) break;
            float z = 0.0f;
#pragma unroll
            for (int y = 0; y < 4; ++y) z += __uint_as_float((uint32_t)sum[y]) + __uint_as_float((uint32_t)(sum[y] >> 32));
            tiles += it.tiles;
            float *other = part + (2 * i + m) * 128 + r;
            if (t0) {
                *other = z;
                __syncwarp();
                if (lane == 0) mbar_arrive(&part_full[2 * i + m]);
            } else {
                if (!(go = wait(&part_full[2 * i + m], (uint32_t)(n / WW_ITEMS)))) break;
                if (mine) a.out[at] = was + (z + *other);
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(&item_empty[i]);
        }
        weigh_behind(a, (long long)blockIdx.x * (WW_GROUPS * 4) + warp, (long long)gridDim.x * (WW_GROUPS * 4));
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (warp == WW_MMA) tmem_free(tm, 512);
}

// The queries as [tokens][heads][d], boxes of a KV head's query heads of 128 rows; false where they do not
// lie in a way that copies can follow (one row for many).
bool query_map(CUtensorMap *map, const WeighArgs &a, int dtype, int d) {
    const EncodeTiledFn encode = tensor_map_encoder();
    const int g = 1 << a.g_shift, hq = a.hkv * g;
    if (!encode || (a.q_hs == 0 && hq > 1) || (a.q_ts == 0 && a.q_tokens > 1)) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)hq, (cuuint64_t)a.q_tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)(hq > 1 ? a.q_hs : d) * 2, (cuuint64_t)(a.q_tokens > 1 ? a.q_ts : (long long)hq * d) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)g, (cuuint32_t)(128 / g)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode(map, dtype == VERKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<uint16_t *>(a.q), dims,
                  strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BF, int D>
cudaError_t launch_wide(const WeighArgs &a, const CUtensorMap &kmap, const CUtensorMap &qmap, unsigned blocks, cudaStream_t s) {
    const cudaError_t e = ensure_smem((const void *)k_weigh_wide<BF, D>, WeighWide<D>::BYTES);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_weigh_wide<BF, D>, dim3(blocks), dim3(WW_NT), WeighWide<D>::BYTES, s, a, kmap, qmap);
}

template <typename T, int D, bool PACKED>
cudaError_t launch_few(const WeighArgs &a, long long items, long long units, cudaStream_t s) {
    using K = Keys<T, D, PACKED>;
    constexpr size_t bytes = (size_t)WF_NT / 32 * K::AHEAD * K::PLACE;
    const cudaError_t e = ensure_smem((const void *)k_weigh_few<T, D, PACKED>, bytes);
    if (e != cudaSuccess) return e;
    const long long blocks = std::max(1LL, std::min(std::max(items, (units + 3) / 4), 152LL * K::CTAS));
    return launch_pdl(k_weigh_few<T, D, PACKED>, dim3((unsigned)blocks), dim3(WF_NT), bytes, s, a);
}

}  // namespace

cudaError_t launch_weigh(const WeighArgs &a, int dtype, bool packed, int d, cudaStream_t s) {
    // Rows of a sequence, on average.
    const long long rows = ((long long)a.q_tokens + a.seqs - 1) / a.seqs << a.g_shift;
    const long long units = (long long)a.seqs * a.hkv;
    const bool few = rows <= 8;
    const long long items = few ? (units * ((a.max_length + 15) / 16) + WF_NT / 32 - 1) / (WF_NT / 32) : units * ((a.max_length + WM_TOKENS - 1) / WM_TOKENS);
    CUtensorMap kmap, qmap;
    if (rows > WW_ROWS && !packed && query_map(&qmap, a, dtype, d) &&
        paged_tensor_map(&kmap, a.pages, dtype, (long long)a.num_pages * a.hkv << a.page_shift, d, std::min(1 << a.page_shift, WM_TOKENS)) == cudaSuccess) {
        const unsigned wide = (unsigned)std::max(1LL, std::min(std::max(items, (units + 15) / 16), 152LL));
        if (d == 128) return dtype == VERKV_BF16 ? launch_wide<true, 128>(a, kmap, qmap, wide, s) : launch_wide<false, 128>(a, kmap, qmap, wide, s);
        return dtype == VERKV_BF16 ? launch_wide<true, 64>(a, kmap, qmap, wide, s) : launch_wide<false, 64>(a, kmap, qmap, wide, s);
    }
    const unsigned blocks = (unsigned)std::max(1LL, std::min(std::max(items, (units + 3) / 4), 152LL * 4));
#define VERKV_WEIGH(TT, DT, DD, PP)                                                                                   \
    if (dtype == DT && d == DD && packed == PP) {                                                                     \
        if (few) return launch_few<TT, DD, PP>(a, items, units, s);                                                   \
        return launch_pdl(k_weigh_many<TT, DD, PP>, dim3(blocks), dim3(WM_NT), (size_t)ManyLayout<DD>::BYTES, s, a);  \
    }
    VERKV_WEIGH(PgBf16, VERKV_BF16, 128, false) VERKV_WEIGH(PgBf16, VERKV_BF16, 64, false)
    VERKV_WEIGH(PgF16, VERKV_F16, 128, false) VERKV_WEIGH(PgF16, VERKV_F16, 64, false)
    VERKV_WEIGH(PgBf16, VERKV_BF16, 128, true) VERKV_WEIGH(PgBf16, VERKV_BF16, 64, true)
    VERKV_WEIGH(PgF16, VERKV_F16, 128, true) VERKV_WEIGH(PgF16, VERKV_F16, 64, true)
#undef VERKV_WEIGH
    return cudaErrorInvalidValue;
}

}  // namespace verkv
