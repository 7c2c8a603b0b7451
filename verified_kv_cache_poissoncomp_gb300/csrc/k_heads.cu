// k_heads.cu -- per-head norms and the position rotation of queries and keys in one pass, with the
// keys (and the values beside them) going to rows of the caller or into a paged cache.
//
//   y = x w / sqrt(mean(x^2) + eps);   (a, b) -> (a cos t - b sin t, b cos t + a sin t)
//
// The angle.  A float32 product position * frequency loses the angle of far positions (at 131072 a
// float32 step is 2^-7 of a radian).  The frequency is therefore kept in turns per position as a
// 64-bit fixed-point fraction: position * turns mod 2^64 is reduced to one turn exactly, by integer
// arithmetic that wraps.  Its upper 32 bits, read as a signed fraction of a turn in [-1/2, 1/2),
// give an argument in [-pi, pi), where the hardware sine and cosine are within 2^-21 of exact:
// far below half a step of the 16-bit result.
//
// Bound: the rows' bytes (2 d each way per head) for prompts, one launch for a decode step.  A row
// takes d / 8 lanes, each holding two groups of four channels: rotated in halves, a channel and its
// partner rotary_dim / 2 away are in the same lane, rotated in pairs, neighbours are, so that a
// rotation moves nothing between lanes and a lane makes four sines.  Only the square sums go by
// shuffle.  A warp takes PASSES rounds of 2 (d = 128) or 4 rows of one token, all queries, keys or
// values; it loads them all, makes the token's sines once, folds the norm's weights into them --
//   out_a = s (x_a (w_a cos) - x_b (w_b sin)),  out_b = s (x_b (w_b cos) + x_a (w_a sin)),  s = 1 / rms
// -- and then spends three packed operations a channel pair.
//
// Measured: 32768 tokens of 40 heads of 128 (671 MB) 104 us, 0.95 of a plain copy's bandwidth; 32768
// tokens' keys and values into pages (268 MB) 47 us, 0.85; 8 tokens 2.1 us and 1021 small ones 3.1, a
// launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.cuh"
#include "verkv_common.cuh"

namespace verkv {

namespace {

constexpr int HD_NT = 256;

struct Bf16 {
    static __device__ __forceinline__ float2 up(uint32_t x) { return make_float2(bf16lo(x), bf16hi(x)); }
    static __device__ __forceinline__ uint32_t down(float lo, float hi) {
        uint32_t y;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
        return y;
    }
};
struct F16 {
    static __device__ __forceinline__ float2 up(uint32_t x) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&x));
    }
    static __device__ __forceinline__ uint32_t down(float lo, float hi) {
        uint32_t y;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
        return y;
    }
};

// Two floats in one register pair: the packed arithmetic of this architecture.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float x, float y) {
    f32x2 v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
    return v;
}
__device__ __forceinline__ float2 split(f32x2 v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// A lane's eight channels as x[0..1] and their partners y[0..1], pairs of floats: in halves the
// channels of `a` and `b`; in pairs (IL) the even and the odd ones of both.
template <typename T, bool IL>
__device__ __forceinline__ void unpack(const uint2 &a, const uint2 &b, f32x2 (&x)[2], f32x2 (&y)[2]) {
    const float2 a0 = T::up(a.x), a1 = T::up(a.y), b0 = T::up(b.x), b1 = T::up(b.y);
    if (IL) {
        x[0] = pair(a0.x, a1.x);
        x[1] = pair(b0.x, b1.x);
        y[0] = pair(a0.y, a1.y);
        y[1] = pair(b0.y, b1.y);
    } else {
        x[0] = pair(a0.x, a0.y);
        x[1] = pair(a1.x, a1.y);
        y[0] = pair(b0.x, b0.y);
        y[1] = pair(b1.x, b1.y);
    }
}
template <typename T, bool IL>
__device__ __forceinline__ void repack(const f32x2 (&x)[2], const f32x2 (&y)[2], uint2 &a, uint2 &b) {
    const float2 x0 = split(x[0]), x1 = split(x[1]), y0 = split(y[0]), y1 = split(y[1]);
    if (IL) {
        a = make_uint2(T::down(x0.x, y0.x), T::down(x0.y, y0.y));
        b = make_uint2(T::down(x1.x, y1.x), T::down(x1.y, y1.y));
    } else {
        a = make_uint2(T::down(x0.x, x0.y), T::down(x1.x, x1.y));
        b = make_uint2(T::down(y0.x, y0.y), T::down(y1.x, y1.y));
    }
}

// sin and cos of position p's angle for the pair with `turns` (see the head of this file).
__device__ __forceinline__ void turn_sincos(int32_t pos, uint64_t turns, float &s, float &c) {
    const uint32_t lo = (uint32_t)turns, hi = (uint32_t)(turns >> 32), p = (uint32_t)pos;
    // upper word of pos * turns mod 2^64 (p is 2^32 more than a negative pos)
    const int32_t frac = (int32_t)(__umulhi(p, lo) + p * hi - (pos < 0 ? lo : 0u));
    const float x = (float)frac * 1.4629180792671596e-9f;      // 2 pi / 2^32
    s = __sinf(x);
    c = __cosf(x);
}

template <typename T, int D, int PASSES, bool IL>
__global__ void __launch_bounds__(HD_NT) k_heads(const __grid_constant__ HeadsArgs a) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;  // lanes a row, rows a warp holds at once
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, li = lane % LPR;
    const int item = blockIdx.x * (HD_NT / 32) + (threadIdx.x >> 5);
    const int t = (unsigned)item / (unsigned)a.chunks;
    if (t >= a.tokens) return;
    int c = item - t * a.chunks;
    const int kind = c < a.chunks_q ? 0 : c < a.chunks_q + a.chunks_k ? 1 : 2;  // queries, keys, values
    c -= kind == 0 ? 0 : kind == 1 ? a.chunks_q : a.chunks_q + a.chunks_k;
    const int rows = kind == 0 ? a.hq : kind == 1 ? a.hk : a.hv;
    const long long hs = kind == 0 ? a.q_hs : kind == 1 ? a.k_hs : a.v_hs;
    const int row0 = c * (PASSES * RPW) + lane / LPR;

    // This lane's two groups of channels, at ca and cb.  In halves: partners while the lane's share of
    // the rotated part lasts, then channels that are not rotated; in pairs: neighbours.
    const bool turned = li < (a.rd >> 3);
    int ca = li * 8, cb = ca + 4;
    if (!IL && turned) {
        ca = li * 4;
        cb = ca + (a.rd >> 1);
    }

    const uint16_t *src = (kind == 0 ? a.q + t * a.q_ts : kind == 1 ? a.k + t * a.k_ts : a.v + t * a.v_ts) + row0 * hs;
    uint2 xa[PASSES], xb[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        xa[p] = xb[p] = make_uint2(0u, 0u);
        if (row0 + p * RPW < rows) {
            // many rows pass once: not worth a place in the cache (a 32K prompt's append 57 -> 47 us)
            xa[p] = PASSES > 1 ? __ldcs(reinterpret_cast<const uint2 *>(src + ca)) : *reinterpret_cast<const uint2 *>(src + ca);
            xb[p] = PASSES > 1 ? __ldcs(reinterpret_cast<const uint2 *>(src + cb)) : *reinterpret_cast<const uint2 *>(src + cb);
        }
        src += RPW * hs;
    }

    // Where the rows go.
    uint16_t *dst;
    long long ds;
    if (kind == 0) {
        dst = a.q_out + t * a.qo_ts;
        ds = a.qo_hs;
    } else if (!a.pages) {
        dst = a.k_out + t * a.ko_ts;
        ds = a.ko_hs;
    } else {
        const int s = a.seq[t];
        if (s == -1) return;
        const int i = a.index[t], pg = i >> a.page_shift;
        int page = -1;
        if (s >= 0 && s < a.table_rows && i >= 0 && pg < a.table_stride)
            page = a.table[(long long)s * a.table_stride + pg];
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) raise_error(a.err, ERR_PAGE);
            return;
        }
        dst = a.pages + (((long long)page * a.hk << a.page_shift) + (i & ((1 << a.page_shift) - 1))) * (2 * D) + (kind == 2 ? D : 0);
        ds = (long long)(2 * D) << a.page_shift;
    }
    dst += row0 * ds;

    const uint16_t *w = kind == 0 ? a.wq : a.wk;
    const bool norm = kind != 2 && w;
    if (norm || (kind != 2 && a.rd > 0)) {
        // Coefficients of x and y in the two results.
        f32x2 xc[2], ys[2], yc[2], xs[2], wx[2], wy[2];
        wx[0] = wx[1] = wy[0] = wy[1] = pair(1.0f, 1.0f);
        if (norm) unpack<T, IL>(*reinterpret_cast<const uint2 *>(w + ca), *reinterpret_cast<const uint2 *>(w + cb), wx, wy);
        float sn[4] = {0.0f, 0.0f, 0.0f, 0.0f}, cs[4] = {1.0f, 1.0f, 1.0f, 1.0f};
        if (turned) {  // pairs li * 4 .. + 3 in either order
            const int32_t pos = a.positions[t];
            const ulonglong2 *tp = reinterpret_cast<const ulonglong2 *>(a.turns + li * 4);
            const ulonglong2 t0 = tp[0], t1 = tp[1];
            turn_sincos(pos, t0.x, sn[0], cs[0]);
            turn_sincos(pos, t0.y, sn[1], cs[1]);
            turn_sincos(pos, t1.x, sn[2], cs[2]);
            turn_sincos(pos, t1.y, sn[3], cs[3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const f32x2 co = pair(cs[2 * i], cs[2 * i + 1]), si = pair(sn[2 * i], sn[2 * i + 1]);
            xc[i] = mul2(wx[i], co);
            yc[i] = mul2(wy[i], co);
            xs[i] = mul2(wx[i], si);
            ys[i] = mul2(wy[i], pair(-sn[2 * i], -sn[2 * i + 1]));
        }
        const bool whole = a.rd == D;
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            f32x2 x[2], y[2], u[2], v[2];
            unpack<T, IL>(xa[p], xb[p], x, y);
            f32x2 inv = pair(1.0f, 1.0f);
            if (norm) {
                const float2 ss = split(fma2(x[0], x[0], fma2(x[1], x[1], fma2(y[0], y[0], mul2(y[1], y[1])))));
                float sum = ss.x + ss.y;
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                const float r = rsqrtf(sum * (1.0f / D) + a.eps);
                inv = pair(r, r);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                u[i] = mul2(x[i], xc[i]);
                v[i] = mul2(y[i], yc[i]);
                // a channel that is not rotated stays apart from the other, which may be no number
                if (whole || turned) {
                    u[i] = fma2(y[i], ys[i], u[i]);
                    v[i] = fma2(x[i], xs[i], v[i]);
                }
                u[i] = mul2(u[i], inv);
                v[i] = mul2(v[i], inv);
            }
            repack<T, IL>(u, v, xa[p], xb[p]);
        }
    }
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        if (row0 + p * RPW < rows) {
            if (PASSES > 1) {
                __stcs(reinterpret_cast<uint2 *>(dst + ca), xa[p]);
                __stcs(reinterpret_cast<uint2 *>(dst + cb), xb[p]);
            } else {
                *reinterpret_cast<uint2 *>(dst + ca) = xa[p];
                *reinterpret_cast<uint2 *>(dst + cb) = xb[p];
            }
        }
        dst += RPW * ds;
    }
}

}  // namespace

cudaError_t launch_heads(const HeadsArgs &args, int dtype, int d, cudaStream_t s) {
    HeadsArgs a = args;
    const int rpw = 256 / d;
    // One round a warp while that fills no more than half the warps the GPU holds (below about 250 tokens
    // of 40 heads; 64 tokens 2.2 against 2.6 us, 1024 tokens 7.2 against 5.3), else four.
    int passes = 4;
    if ((long long)a.tokens * (a.hq + a.hk + a.hv) < 152LL * 32 * rpw) passes = 1;
    const auto chunks = [&](int rows) { return (rows + passes * rpw - 1) / (passes * rpw); };
    a.chunks_q = chunks(a.hq);
    a.chunks_k = chunks(a.hk);
    a.chunks = a.chunks_q + a.chunks_k + chunks(a.hv);
    const long long items = (long long)a.tokens * a.chunks, blocks = (items + HD_NT / 32 - 1) / (HD_NT / 32);
    if (items + HD_NT / 32 > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    const bool il = a.interleaved && a.rd > 0;
#define VERKV_HEADS(TT, DT, DD, PP)                                                                                        \
    if (dtype == DT && d == DD && passes == PP) {                                                                          \
        if (il) return launch_pdl(k_heads<TT, DD, PP, true>, dim3((unsigned)blocks), dim3(HD_NT), 0, s, a);                \
        return launch_pdl(k_heads<TT, DD, PP, false>, dim3((unsigned)blocks), dim3(HD_NT), 0, s, a);                       \
    }
    VERKV_HEADS(Bf16, VERKV_BF16, 128, 1) VERKV_HEADS(Bf16, VERKV_BF16, 128, 4)
    VERKV_HEADS(Bf16, VERKV_BF16, 64, 1) VERKV_HEADS(Bf16, VERKV_BF16, 64, 4)
    VERKV_HEADS(F16, VERKV_F16, 128, 1) VERKV_HEADS(F16, VERKV_F16, 128, 4)
    VERKV_HEADS(F16, VERKV_F16, 64, 1) VERKV_HEADS(F16, VERKV_F16, 64, 4)
#undef VERKV_HEADS
    return cudaErrorInvalidValue;
}

}  // namespace verkv
