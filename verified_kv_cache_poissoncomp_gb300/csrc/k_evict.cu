// k_evict.cu -- eviction from a paged cache: of a sequence's tokens, each KV head keeps the first, the last
// and, of those between, the ones with the most weight; the kept rows move together in their pages.
//
// What is kept.  With len > keep: places 0 .. first - 1, len - last .. len - 1, and the keep - first - last
// places between with the largest weights, ties to the lower place.  The threshold is found by three
// rounds over the weights' bits (a map of float32 to integers of the same order), each a histogram of 2048
// bins in shared memory.
//
// What moves.  Order among old tokens does not matter to attention (a key carries its position), so rows
// move as little as they can: chosen ones below keep - last stay, and the holes between them are filled, in
// ascending order, by the chosen ones behind.  A sequence that has run over by 256 of 2048 moves some 230
// and the last ones, not 2048.  The last ones move together and keep their order, for the next eviction's
// sake.  Their new places may be among the old ones of either, hence two steps: holes first, then the last
// ones, a piece at a time held in registers between its loads and its stores.
//
// A cluster of 1 to 8 CTAs has a head of a sequence (as many as fill the GPU), a contiguous share of the
// places each; counts and histograms are exchanged through distributed shared memory.  One launch, bound by
// its latency: some 12 barriers, dependent loads (a length; weights; a list, a table, a row; a table, a row) and,
// since most of it runs once, the fetch of its instructions, hence loops that are not unrolled.  Measured: 32
// sequences x 8 heads of 2304 tokens down to 2048 (24 MB of rows read, 24 written) 17.1 us, of which choosing takes 5 and
// the lists 2; four prompts of 8192 tokens down to 1024 16.0; 64 sequences of 4096 down to 1024 (426 MB) 85, 5.0 TB/s.
#include <algorithm>

#include "paged.cuh"
#include "q4.cuh"
#include "verkv_common.cuh"

namespace verkv {

namespace {

constexpr int EV_NT = 512, EV_WARPS = EV_NT / 32;
// Keys of a CTA's share that stay in shared memory.  (More leave too little of it to the loads on their way: with 20480
// 64 sequences of 4096 tokens take 98 us for 82, with 12288 four of 131072 69 for 62.)
constexpr int EV_KEYS = 16384;
constexpr int EV_BINS = 2048;
constexpr int EV_AHEAD = 4;      // rows in flight a lane group

struct EvictShared {
    uint32_t keys[EV_KEYS];
    int hist[3][EV_BINS];
    int sums[5][EV_WARPS];     // of each round, then a warp's ties, and its holes and what may fill them
    int fills[EV_WARPS];
    int found[3][3];           // of each round: the bin, how many are above it and in it
    alignas(8) int counts[2];  // this CTA's holes, and what may fill them
};

// float32 in its order as integers; -0 is 0, and what is no number is above all.
__device__ __forceinline__ uint32_t ordered(float w) {
    if (w != w) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

// Sum of v's over a warp's lanes before this one, and this one.
__device__ __forceinline__ int scan_upto(int v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if ((threadIdx.x & 31) >= o) v += y;
    }
    return v;
}
// Sum over the CTA's warps (lanes 0 .. 15 hold theirs) before this one; total: over all.
__device__ __forceinline__ int sum_before(const int *of, int &total) {
    const int lane = threadIdx.x & 31, v = lane < EV_WARPS ? of[lane] : 0;
    total = __reduce_add_sync(0xFFFFFFFFu, v);
    return __reduce_add_sync(0xFFFFFFFFu, lane < (int)(threadIdx.x >> 5) ? v : 0);
}

// Where chunk c of a row is: of the pool's row `at`, in its order of pages, heads and places.
template <int D, bool PACKED>
struct EvictRow;
template <int D>
struct EvictRow<D, false> {
    typedef uint4 Vec;
    static constexpr int CHUNKS = 4 * D / 16;
    static __device__ __forceinline__ long long offset(int at, int c) { return (long long)at * (4 * D) + c * 16; }
};
template <int D>
struct EvictRow<D, true> {
    typedef typename Q4Vec<D>::Key Vec;  // four of codes and one of floors and steps a side
    static constexpr int CHUNKS = 10;
    static __device__ __forceinline__ long long offset(int at, int c) {
        const int side = c >= 5 ? 1 : 0, x = c - 5 * side, t = at & 15;
        return (long long)(at >> 4) * Q4<D>::BLOCK + side * Q4<D>::SIDE +
               (x < 4 ? t * Q4<D>::CODE + x * (int)sizeof(Vec) : Q4<D>::PARS + t * Q4<D>::PAR);
    }
};

// Of all threads of the cluster, and of what they have written.
__device__ __forceinline__ void cluster_barrier(int cl) {
    if (cl == 1) {
        __syncthreads();
        return;
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int D, bool PACKED>
__global__ void __launch_bounds__(EV_NT, 2) k_evict(const __grid_constant__ EvictArgs a) {
    using Row = EvictRow<D, PACKED>;
    typedef typename Row::Vec Vec;
    constexpr int NC = Row::CHUNKS, RPW = 32 / NC;
    extern __shared__ __align__(16) unsigned char ev_smem[];
    EvictShared &sh = *reinterpret_cast<EvictShared *>(ev_smem);
    cg::cluster_group cluster = cg::this_cluster();
    const int cl = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int unit = blockIdx.x / cl, s = unit / a.hkv, head = unit - s * a.hkv;
#pragma unroll
    for (int r = 0; r < 3; ++r) reinterpret_cast<int4 *>(sh.hist[r])[tid] = make_int4(0, 0, 0, 0);
    if (tid < 9) sh.found[tid / 3][tid % 3] = 0;  // (what weights that change under the kernel leave)
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int given = a.length[s], len = clampi(given, 0, a.max_length);
    if (given != len && tid == 0) raise_error(a.err, ERR_PAGE);
    const float *in = a.in + (long long)unit * a.places;
    float *out = a.out + (long long)unit * a.places;
    int32_t *kept = a.kept ? a.kept + (long long)unit * a.keep : nullptr;
    const bool apart = a.in != a.out;
    const int all = cl * EV_NT, me = rank * EV_NT + tid;

    if (len <= a.keep) {
        for (int i = me; kept && i < a.keep; i += all) kept[i] = i < len ? i : -1;
        for (int i = me; i < a.places; i += all)
            if (i >= len) out[i] = 0.0f;
            else if (apart) out[i] = in[i];
        return;
    }

    // This CTA's share of the places between the first and the last.
    const int need = a.keep - a.first - a.last, middle = len - a.last - a.first, zone = a.keep - a.last;
    const int per = ((middle + cl - 1) / cl + 3) & ~3;
    const int lo = a.first + min(middle, rank * per), hi = a.first + min(middle, (rank + 1) * per);
    // Keys of places i .. i + 3, i - lo a multiple of 4; behind hi: anything.
    auto keys_of = [&](uint32_t (&k)[4], int i) {
        if (i - lo < EV_KEYS) {
            const uint4 v = *reinterpret_cast<const uint4 *>(sh.keys + (i - lo));
            k[0] = v.x;
            k[1] = v.y;
            k[2] = v.z;
            k[3] = v.w;
        } else {
#pragma unroll
            for (int y = 0; y < 4; ++y) k[y] = i + y < hi ? ordered(in[i + y]) : 0u;
        }
    };

    uint32_t threshold = 0xFFFFFFFFu;
    int left = need;      // still to be taken, of those whose upper bits are the threshold's
    int same = 0;         // how many there are of those
    int bin = 0;
    if (need > 0) {
        threshold = 0;
#pragma unroll 1
        for (int r = 0; r < 3; ++r) {
            const int shift = r == 0 ? 21 : r == 1 ? 10 : 0, mask = r == 2 ? 1023 : 2047;
            int *hist = sh.hist[r];
            if (r == 0) {
                // (the loads of a turn are on their way together)
                for (int i0 = lo + tid; i0 < hi; i0 += 8 * EV_NT) {
                    float w[8];
#pragma unroll
                    for (int y = 0; y < 8; ++y) w[y] = i0 + y * EV_NT < hi ? in[i0 + y * EV_NT] : 0.0f;
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const int i = i0 + y * EV_NT;
                        if (i >= hi) break;
                        const uint32_t k = ordered(w[y]);
                        if (i - lo < EV_KEYS) sh.keys[i - lo] = k;
                        atomicAdd(&hist[k >> 21], 1);
                    }
                }
            } else {
                const int fixed = r == 1 ? 21 : 10;
#pragma unroll 1
                for (int i = lo + 4 * tid; i < hi; i += 4 * EV_NT) {
                    uint32_t k[4];
                    keys_of(k, i);
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        if (i + y < hi && k[y] >> fixed == threshold >> fixed) atomicAdd(&hist[(k[y] >> shift) & mask], 1);
                }
            }
            cluster_barrier(cl);
            // From the top: thread 0 has the highest bins.
            int n[4] = {0, 0, 0, 0};
            const int bins = EV_BINS / 4 - 1 - tid;
            if (cl == 1) {
                const int4 v = reinterpret_cast<const int4 *>(hist)[bins];
                n[0] = v.w;
                n[1] = v.z;
                n[2] = v.y;
                n[3] = v.x;
            } else {
                int4 v[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) v[c] = c < cl ? reinterpret_cast<const int4 *>(cluster.map_shared_rank(hist, c))[bins] : make_int4(0, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    n[0] += v[c].w;
                    n[1] += v[c].z;
                    n[2] += v[c].y;
                    n[3] += v[c].x;
                }
            }
            // The warp whose 128 bins hold the threshold looks for it.
            const int own = n[0] + n[1] + n[2] + n[3], sum = __reduce_add_sync(0xFFFFFFFFu, own);
            if (lane == 0) sh.sums[r][warp] = sum;
            __syncthreads();
            int total;
            const int before = sum_before(sh.sums[r], total);
            if (before < left && before + sum >= left) {
                int above = before + scan_upto(own) - own;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    if (above < left && above + n[y] >= left) {
                        sh.found[r][0] = bins * 4 + 3 - y;
                        sh.found[r][1] = above;
                        sh.found[r][2] = n[y];
                    }
                    above += n[y];
                }
            }
            __syncthreads();
            bin = sh.found[r][0];
            left -= sh.found[r][1];
            same = sh.found[r][2];
            threshold |= (uint32_t)bin << shift;
        }
    }
    // The share in equal runs, one a warp, four places a lane a turn.  (Few instructions: most of them run once, and wait
    // to be fetched.)
    constexpr int TURN = 128;
    const int run = ((hi - lo + EV_WARPS - 1) / EV_WARPS + 3) & ~3;
    const int w0 = min(hi, lo + warp * run), w1 = min(hi, w0 + run);
    // Of `same` places with the threshold's weight, the lowest `left` are kept: those in the shares before this one
    // come first.
    const bool some = need > 0 && left < same;
    int ties0 = 0;
    if (some) {
        if (cl > 1) ties0 = __reduce_add_sync(0xFFFFFFFFu, lane < rank ? cluster.map_shared_rank(sh.hist[2], lane)[bin] : 0);
        int n = 0;
#pragma unroll 1
        for (int i = w0 + 4 * lane; i < w1; i += TURN) {
            uint32_t k[4];
            keys_of(k, i);
#pragma unroll
            for (int y = 0; y < 4; ++y) n += i + y < w1 && k[y] == threshold ? 1 : 0;
        }
        n = __reduce_add_sync(0xFFFFFFFFu, n);
        if (lane == 0) sh.sums[3][warp] = n;
        __syncthreads();
        ties0 += sum_before(sh.sums[3], n);
    }
    // Which of places i .. i + 3 stay, and (f) which are holes or, behind the zone, fill one; `ties` have come before the
    // turn's first.  Where neither is asked for i is behind w1.
    auto turn = [&](int i, int &ties, uint32_t &stays, uint32_t &f) {
        uint32_t k[4] = {0u, 0u, 0u, 0u};
        if (i < w1) keys_of(k, i);
        int eq = 0;
        if (some) {
#pragma unroll
            for (int y = 0; y < 4; ++y) eq += i + y < w1 && k[y] == threshold ? 1 : 0;
            const int upto = scan_upto(eq);
            eq = ties + upto - eq;
            ties += __shfl_sync(0xFFFFFFFFu, upto, 31);
        }
        uint32_t set = 0;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            bool in_set = k[y] >= threshold;
            if (some && k[y] == threshold) in_set = eq++ < left;
            set |= in_set ? 1u << y : 0u;
        }
        if (need == 0) set = 0;
        const uint32_t there = (1u << clampi(w1 - i, 0, 4)) - 1u, low = (1u << clampi(zone - i, 0, 4)) - 1u;
        set &= there;
        stays = set & low;
        f = (set ^ low) & there;
    };
    // Holes, and the chosen ones behind that fill them, in two lists, in order.  How many there are first.
    int holes = 0, fills = 0, ties = ties0;
#pragma unroll 1
    for (int i0 = w0; i0 < w1; i0 += TURN) {
        const int i = i0 + 4 * lane;
        uint32_t stays, f;
        turn(i, ties, stays, f);
        const uint32_t low = (1u << clampi(zone - i, 0, 4)) - 1u;
        holes += __popc(f & low);
        fills += __popc(f & ~low);
    }
    holes = __reduce_add_sync(0xFFFFFFFFu, holes);
    fills = __reduce_add_sync(0xFFFFFFFFu, fills);
    if (lane == 0) {
        sh.sums[4][warp] = holes;
        sh.fills[warp] = fills;
    }
    __syncthreads();
    int moves, total_fills;
    int hole_at = sum_before(sh.sums[4], moves), fill_at = sum_before(sh.fills, total_fills);
    if (cl > 1) {
        if (tid == 0) {
            sh.counts[0] = moves;
            sh.counts[1] = total_fills;
        }
        cluster_barrier(cl);
        const int2 n = lane < cl ? *reinterpret_cast<const int2 *>(cluster.map_shared_rank(sh.counts, lane)) : make_int2(0, 0);
        moves = __reduce_add_sync(0xFFFFFFFFu, n.x);
        hole_at += __reduce_add_sync(0xFFFFFFFFu, lane < rank ? n.x : 0);
        fill_at += __reduce_add_sync(0xFFFFFFFFu, lane < rank ? n.y : 0);
    }
    moves = min(moves, a.room);
    int32_t *to = a.lists + (long long)unit * 2 * a.room, *from = to + a.room;
    ties = ties0;
#pragma unroll 1
    for (int i0 = w0; i0 < w1; i0 += TURN) {
        const int i = i0 + 4 * lane;
        uint32_t stays, f;
        turn(i, ties, stays, f);
        // Of the places that stay, 32 neighbours at a time: what a lane has of place i0 + 32 y + lane.  (w: on its way meanwhile)
        float w[4];
        bool here[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            here[y] = __shfl_sync(0xFFFFFFFFu, stays, 8 * y + (lane >> 2)) >> (lane & 3) & 1;
            w[y] = apart && here[y] ? in[i0 + 32 * y + lane] : 0.0f;
        }
        const uint32_t low = (1u << clampi(zone - i, 0, 4)) - 1u;
        // (128 of either at most)
        const int n = __popc(f & low) + (__popc(f & ~low) << 16), upto = scan_upto(n), total = __shfl_sync(0xFFFFFFFFu, upto, 31);
        int h = hole_at + ((upto - n) & 0xFFFF), m = fill_at + ((upto - n) >> 16);
        hole_at += total & 0xFFFF;
        fill_at += total >> 16;
#pragma unroll 1
        while (f) {
            const int y = __ffs(f) - 1;
            f &= f - 1;
            const bool hole = i + y < zone;
            const int at = hole ? h++ : m++;
            if (at < a.room) (hole ? to : from)[at] = i + y;
        }
#pragma unroll
        for (int y = 0; y < 4; ++y)
            if (here[y]) {
                const int at = i0 + 32 * y + lane;
                if (kept) kept[at] = at;
                if (apart) out[at] = w[y];
            }
    }
    for (int i = me; i < a.first; i += all) {
        if (kept) kept[i] = i;
        if (apart) out[i] = in[i];
    }
    cluster_barrier(cl);  // the lists are there, and nobody reads another's shared memory any more

    // Rows.  A lane group holds a row (of 16-bit pages a warp, or half of one), EV_AHEAD of them at a time; the lanes of a
    // warp look up the places of its next 32 together, one a lane.
    const int32_t *row = a.table + (long long)s * a.stride;
    const int c = lane % NC, sub = lane / NC, gw = rank * EV_WARPS + warp, gws = cl * EV_WARPS;
    unsigned char *pool = static_cast<unsigned char *>(a.pages);
    auto place = [&](int tok, bool there) -> int {  // a token's row of the pool, -1: none
        const int id = there ? row[tok >> a.page_shift] : -1;
        if (id >= 0 && id < a.num_pages) return ((id * a.hkv + head) << a.page_shift) + (tok & ((1 << a.page_shift) - 1));
        if (there) raise_error(a.err, ERR_PAGE);
        return -1;
    };
    const int shift = len - a.keep;
    // First into the holes.  (Weights that change under the kernel leave no list: places are kept in their range.)  Then
    // the last ones, a piece at a time: all its rows are in registers before one of them is written.  A piece's new
    // places are below the next one's old ones, so pieces need no more between them.
    constexpr int PIECE = EV_AHEAD * RPW;  // a warp's rows of a piece
#pragma unroll 1
    for (int lasts = 0; lasts < 2; ++lasts) {
        const int n = lasts ? a.last : moves;
        int src = 0, dst = 0, sat = -1, dat = -1, at = 32;
        float w = 0.0f;
#pragma unroll 1
        for (int k0 = 0; k0 < n || (lasts && k0 == 0); k0 += gws * PIECE) {
            if (at + PIECE > 32) {
                const int k = k0 + gw + lane * gws;
                const bool there = k < n && lane < 32 / PIECE * PIECE;
                src = zone + shift + k;
                dst = zone + k;
                if (!lasts && there) {
                    src = clampi(from[k], 0, len - 1);
                    dst = clampi(to[k], 0, zone - 1);
                }
                if (!there) src = dst = -1;
                sat = place(src, there);
                dat = place(dst, there);
                w = there ? in[src] : 0.0f;
                at = 0;
            }
            Vec v[EV_AHEAD];
#pragma unroll
            for (int y = 0; y < EV_AHEAD; ++y) {
                const int r = __shfl_sync(0xFFFFFFFFu, sat, (at + y * RPW + sub) & 31);
                v[y] = Vec{};
                if (sub < RPW && r >= 0) v[y] = *reinterpret_cast<const Vec *>(pool + Row::offset(r, c));
            }
            if (lasts) cluster_barrier(cl);
#pragma unroll
            for (int y = 0; y < EV_AHEAD; ++y) {
                const int r = __shfl_sync(0xFFFFFFFFu, dat, (at + y * RPW + sub) & 31);
                if (sub < RPW && r >= 0) *reinterpret_cast<Vec *>(pool + Row::offset(r, c)) = v[y];
            }
            if (lane >= at && lane < at + PIECE && dst >= 0) {
                out[dst] = w;
                if (kept) kept[dst] = src;
            }
            at += PIECE;
        }
    }
    // (every weight has been read: the last piece's barrier)
    for (int i = a.keep + me; i < a.places; i += all) out[i] = 0.0f;
}

template <int D, bool PACKED>
cudaError_t launch(const EvictArgs &a, cudaStream_t s) {
    const cudaError_t e = ensure_smem((const void *)k_evict<D, PACKED>, sizeof(EvictShared));
    if (e != cudaSuccess) return e;
    // As many CTAs a cluster as leave none waiting (two an SM), with 2048 places each at least: barriers of eight CTAs
    // cost more than shares of 1024 save (four prompts of 8192: 8 CTAs 32 us, 4 18.7, 2 22.0, 1 28.9).
    const long long units = (long long)a.seqs * a.hkv;
    int cl = 1;
    while (cl < 8 && units * cl * 2 <= 304 && a.max_length >= 2048 * cl * 2) cl *= 2;
    if (units * cl > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * cl));
    cfg.blockDim = dim3(EV_NT);
    cfg.dynamicSmemBytes = sizeof(EvictShared);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cl;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_evict<D, PACKED>, a);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, bool packed, int d, cudaStream_t s) {
    if (d == 128) return packed ? launch<128, true>(a, s) : launch<128, false>(a, s);
    return packed ? launch<64, true>(a, s) : launch<64, false>(a, s);
}

}  // namespace verkv
