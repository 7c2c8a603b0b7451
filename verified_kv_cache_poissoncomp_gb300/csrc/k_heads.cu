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
// takes d / 8 lanes of 16 bytes, so a warp holds 2 (d = 128) or 4 rows at once; the square sums
// and the partner channel of a rotation (rotary_dim / 2 channels away: whole lanes) move by
// shuffles, and nothing goes through shared memory.  A warp takes PASSES times that many rows of
// one token, loads them all before it computes, and makes the token's sines once for them.
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

template <typename T>
__device__ __forceinline__ void unpack(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = T::up(w[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
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

template <typename T, int D, int PASSES>
__global__ void __launch_bounds__(HD_NT) k_heads(const HeadsArgs a) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;  // lanes a row, rows a warp holds at once
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, li = lane % LPR, ch = li * 8;
    const long long item = (long long)blockIdx.x * (HD_NT / 32) + (threadIdx.x >> 5);
    const int t = (int)(item / a.chunks);
    if (t >= a.tokens) return;
    const int row0 = (int)(item - (long long)t * a.chunks) * (PASSES * RPW) + lane / LPR;
    const int rows = a.hq + a.hk + a.hv;

    uint4 x[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int r = row0 + p * RPW;
        x[p] = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) {
            const uint16_t *src =
                r < a.hq ? a.q + t * a.q_ts + r * a.q_hs
                : r < a.hq + a.hk ? a.k + t * a.k_ts + (r - a.hq) * a.k_hs
                                  : a.v + t * a.v_ts + (r - a.hq - a.hk) * a.v_hs;
            x[p] = *reinterpret_cast<const uint4 *>(src + ch);
        }
    }

    // The rotation of this lane's channels.  Half style: pair of channel c is c mod (rd / 2), and
    // its partner sits rd / 16 lanes away; interleaved: pairs lie within the lane.
    const int half = a.rd >> 1;
    const bool turned = ch < a.rd;
    const bool second = !a.interleaved && ch >= half;
    float sn[8], cs[8];
    if (a.rd > 0) {
        const int32_t pos = a.positions[t];
        const int n = a.interleaved ? 4 : 8;
        const int j0 = a.interleaved ? ch >> 1 : second ? ch - half : ch;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sn[i] = 0.0f;
            cs[i] = 1.0f;
            if (i < n && turned) turn_sincos(pos, a.turns[j0 + i], sn[i], cs[i]);
        }
    }
    uint4 wq = make_uint4(0u, 0u, 0u, 0u), wk = wq;
    if (a.wq) wq = *reinterpret_cast<const uint4 *>(a.wq + ch);
    if (a.wk) wk = *reinterpret_cast<const uint4 *>(a.wk + ch);

    // Where this token's keys and values go in the pages: element of its slot for head 0, or -1.
    long long place = -1;
    if (a.pages && row0 + (PASSES - 1) * RPW >= a.hq) {
        const int s = a.seq[t];
        if (s != -1) {
            const int i = a.index[t], pg = i >> a.page_shift;
            int page = -1;
            if (s >= 0 && s < a.table_rows && i >= 0 && pg < a.table_stride)
                page = a.table[(long long)s * a.table_stride + pg];
            if (page >= 0 && page < a.num_pages)
                place = (((long long)page * a.hk << a.page_shift) + (i & ((1 << a.page_shift) - 1))) * (2 * D);
            else if (lane == 0)
                raise_error(a.err, ERR_PAGE);
        }
    }

#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int r = row0 + p * RPW;
        const bool is_q = r < a.hq, is_v = r >= a.hq + a.hk;
        uint4 y = x[p];
        float f[8];
        unpack<T>(x[p], f);
        if (a.wq || a.wk) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
            const uint4 w = is_q ? wq : wk;
            if (is_q ? a.wq != nullptr : a.wk != nullptr) {
                const float inv = rsqrtf(ss * (1.0f / D) + a.eps);
                float g[8];
                unpack<T>(w, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] *= inv * g[i];
            }
        }
        if (a.rd > 0) {
            if (a.interleaved) {
                if (turned) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float u = f[2 * i], v = f[2 * i + 1];
                        f[2 * i] = u * cs[i] - v * sn[i];
                        f[2 * i + 1] = v * cs[i] + u * sn[i];
                    }
                }
            } else {
                const int partner = !turned ? lane : second ? lane - half / 8 : lane + half / 8;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float o = __shfl_sync(0xFFFFFFFFu, f[i], partner);
                    if (turned) f[i] = second ? f[i] * cs[i] + o * sn[i] : f[i] * cs[i] - o * sn[i];
                }
            }
        }
        if (!is_v) y = make_uint4(T::down(f[0], f[1]), T::down(f[2], f[3]), T::down(f[4], f[5]), T::down(f[6], f[7]));
        if (r >= rows) continue;  // no shuffle below
        uint16_t *dst = nullptr;
        if (is_q)
            dst = a.q_out + t * a.qo_ts + r * a.qo_hs;
        else if (!a.pages)
            dst = a.k_out + t * a.ko_ts + (r - a.hq) * a.ko_hs;
        else if (place >= 0)
            dst = a.pages + place + ((long long)(is_v ? r - a.hq - a.hk : r - a.hq) << a.page_shift) * (2 * D) +
                  (is_v ? D : 0);
        if (dst) *reinterpret_cast<uint4 *>(dst + ch) = y;
    }
}

}  // namespace

cudaError_t launch_heads(const HeadsArgs &args, int dtype, int d, cudaStream_t s) {
    HeadsArgs a = args;
    const int rows = a.hq + a.hk + a.hv, rpw = 256 / d;
    int passes = 4;
    if ((long long)a.tokens * rows < 152LL * 64 * rpw) passes = 1;
    a.chunks = (rows + passes * rpw - 1) / (passes * rpw);
    const long long blocks = ((long long)a.tokens * a.chunks + HD_NT / 32 - 1) / (HD_NT / 32);
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
#define VERKV_HEADS(TT, DT, DD, PP) \
    if (dtype == DT && d == DD && passes == PP) return launch_pdl(k_heads<TT, DD, PP>, dim3((unsigned)blocks), dim3(HD_NT), 0, s, a);
    VERKV_HEADS(Bf16, VERKV_BF16, 128, 1) VERKV_HEADS(Bf16, VERKV_BF16, 128, 4)
    VERKV_HEADS(Bf16, VERKV_BF16, 64, 1) VERKV_HEADS(Bf16, VERKV_BF16, 64, 4)
    VERKV_HEADS(F16, VERKV_F16, 128, 1) VERKV_HEADS(F16, VERKV_F16, 128, 4)
    VERKV_HEADS(F16, VERKV_F16, 64, 1) VERKV_HEADS(F16, VERKV_F16, 64, 4)
#undef VERKV_HEADS
    return cudaErrorInvalidValue;
}

}  // namespace verkv
