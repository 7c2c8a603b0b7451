// q4.cuh -- pages of 4-bit codes, and products with them.
//
// The layout.  A page holds, for each KV head, blocks of 16 tokens: the keys' codes [16][d / 2], the
// keys' floors and steps binary16 [16][d / 32][2], then the same of the values.  A block is one piece of
// 20 d bytes, so that one bulk copy brings it.  A code's value is floor + code * step; nibble i of a
// token's 32-bit word w is channel i * d / 8 + w: the words of a token, one nibble of each, are
// d / 8 channels of one group of 32.
//
// Products.  A code n, alone in the lower bits of 16, is the binary16 subnormal n 2^-24, and four bits further
// up 16 n 2^-24: exact operands of a matrix product as they lie, for one instruction a pair.  So products are
// of binary16: queries are scaled to it, row by row, by a power of two that puts their largest channel
// in [2^14, 2^15) (a channel 2^-28 of that loses bits, which count 2^-38 of the row's size), and by 1 / 16 more
// where the codes' are 16 n.  The group's steps come after the product, in float32, and the floors' part,
//     sum_c q_c (floor + n_c step) = step sum_c q_c n_c + floor sum_c q_c,
// is one product of its own of floors (exact in tf32) and the groups' sums (in two tf32 parts, 2^-22).  So
// the cached values are not rounded on their way, and no sum is larger than the values make it.  What sums lose:
// the tensor cores cut each addend of a product off at 2^-25 of the largest one's nominal size, in which a
// subnormal operand counts as 2^-14 (measured: a product, and the sum before it, for codes of 1 to 15).  Over codes n
// that is up to 2^-15 an addend of the largest other operand, over 16 n 2^-19: logits are off by some 2^-15 of a group's
// largest query channel times its step.  (16 n everywhere is a shift more for each pair: 32 sequences of up to 16384
// tokens 84.8 us for 82.3, their weights 62.7 for 61.7, with errors against 64 bits as before.  With 16 + n
// in place of n, which either 16-bit type holds, sums over codes are five times as large, as are their
// float32 errors, and a code takes two instructions more: 32 sequences of up to 16384 tokens 128 us.)
//
// Tokens are the rows (m16) of mma.m16n8k16 and queries its columns (n8): eight queries of a KV head
// fill a product, and a token's codes go from shared memory or global memory to the A operand without
// a shuffle.  Which channels a k-step takes, and in which order, is the words' own: of d = 128, k-step i
// is nibble i of the 16 words, and lane (g, t) of the fragment holds words 4 t .. 4 t + 3 of tokens g and
// g + 8; of d = 64, k-step j is nibbles 2 j and 2 j + 1 of the 8 words, and the lane holds words 2 t and
// 2 t + 1.  Either way k-steps 2 j and 2 j + 1 are group j.
#pragma once

#include "paged.cuh"

namespace verkv {

template <int D>
struct Q4 {
    static constexpr int WORDS = D / 8;              // 32-bit words of a token's codes
    static constexpr int GROUPS = D / 32;
    static constexpr int KS = D / 16;                // k-steps of a product over the channels
    static constexpr int CODE = D / 2, PAR = D / 8;  // bytes of a token's codes, and of its floors and steps
    static constexpr int PARS = 16 * CODE;           // where the floors and steps of a side begin
    static constexpr int SIDE = 16 * (CODE + PAR);   // keys or values of a block
    static constexpr int BLOCK = 2 * SIDE;
};

// Byte k of two words, each in the lower byte of a half: a pair of codes in its lower and one in its upper four bits.
__device__ __forceinline__ uint32_t byte_pair(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}
constexpr uint32_t BYTE0 = 0x4400u, BYTE0_TURNED = 0x0044u, NEXT_BYTE = 0x1111u;  // selectors; turned: b's first
constexpr uint32_t LOW4 = 0x000F000Fu, HIGH4 = 0x00F000F0u;
constexpr float CODE_UNIT = 16777216.0f;  // 2^24 codes a unit

// Products without a sum before them.
__device__ __forceinline__ void mma_tf32_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%4,%5}, {%6,%7}, {%8,%8,%8,%8};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t tf32(float x) {
    uint32_t y;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(y) : "f"(x));
    return y;
}
// Halves of a token's word of floor (lower) and step (upper).
__device__ __forceinline__ float floor_of(uint32_t fs) { return __half2float(__ushort_as_half((unsigned short)fs)); }
__device__ __forceinline__ float step_of(uint32_t fs) { return __half2float(__ushort_as_half((unsigned short)(fs >> 16))); }

template <int D>
struct Q4Vec;
template <>
struct Q4Vec<128> {
    typedef uint4 Key;    // a lane's words of a token's keys; also a token's floors and steps
    typedef uint2 Value;  // a lane's words of a token's values
};
template <>
struct Q4Vec<64> {
    typedef uint2 Key;
    typedef uint32_t Value;
};
__device__ __forceinline__ uint32_t word_of(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ uint32_t word_of(const uint2 &v, int i) { return i == 0 ? v.x : v.y; }
__device__ __forceinline__ uint32_t word_of(const uint32_t &v, int) { return v; }

// The keys of 16 tokens, as a lane holds them.
template <int D>
struct KeyCodes {
    uint32_t x[2][D / 64][4];  // [token g, g + 8][pair of words][byte]
    float step[2][D / 32];
    uint32_t floor[2];  // of group t (of t mod 2, d = 64), as tf32
    __device__ __forceinline__ void codes(int i, const typename Q4Vec<D>::Key &w) {
#pragma unroll
        for (int p = 0; p < D / 64; ++p)
#pragma unroll
            for (int k = 0; k < 4; ++k) x[i][p][k] = byte_pair(word_of(w, 2 * p), word_of(w, 2 * p + 1), BYTE0 + k * NEXT_BYTE);
    }
    __device__ __forceinline__ void scales(int i, const typename Q4Vec<D>::Key &par, uint32_t mine) {
#pragma unroll
        for (int j = 0; j < D / 32; ++j) step[i][j] = step_of(word_of(par, j));
        floor[i] = __float_as_uint(floor_of(mine));
    }
    // The A operand of k-step k.
    __device__ __forceinline__ void frag(uint32_t (&a)[4], int k) const {
        if (D == 128) {
            const uint32_t mask = k & 1 ? HIGH4 : LOW4;
            a[0] = x[0][0][k >> 1] & mask;
            a[1] = x[1][0][k >> 1] & mask;
            a[2] = x[0][D / 64 - 1][k >> 1] & mask;
            a[3] = x[1][D / 64 - 1][k >> 1] & mask;
        } else {
            a[0] = x[0][0][k & 3] & LOW4;
            a[1] = x[1][0][k & 3] & LOW4;
            a[2] = x[0][0][k & 3] & HIGH4;
            a[3] = x[1][0][k & 3] & HIGH4;
        }
    }
};

// Eight queries as the B operand, in the channels' order of the k-steps, scaled; and the sums of their groups.
template <typename T, int D>
struct Queries8 {
    uint32_t b[D / 16][2];
    uint32_t sum[2];  // of query g's group t, 2^-24 of it, in two tf32 parts (d = 64: 0 from group 2 on)
    float unit;       // of query g: 2^24 / its scale
    // row: the channels of query g, or null: zeros.  sign: 0x80008000 turns them round.
    __device__ __forceinline__ void load(const uint16_t *row, uint32_t sign) {
        const int t = threadIdx.x & 3;
        float most = 0.0f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            uint2 v = make_uint2(0u, 0u);
            if (row && D == 128) v = *reinterpret_cast<const uint2 *>(row + 16 * k + 4 * t);
            if (row && D == 64) {
                v.x = *reinterpret_cast<const uint32_t *>(row + 16 * k + 2 * t);
                v.y = *reinterpret_cast<const uint32_t *>(row + 16 * k + 8 + 2 * t);
            }
            b[k][0] = v.x ^ sign;
            b[k][1] = v.y ^ sign;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 f = T::unpack(b[k][i]);
                most = fmaxf(most, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
        }
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
        const int e = min(max(14 + 127 - (int)(__float_as_uint(most) >> 23), -100), 100);  // (a row of zeros: 100)
        const float scale = __uint_as_float((uint32_t)(127 + e) << 23);
        unit = __uint_as_float((uint32_t)(127 + 24 - e) << 23);
        float z[D / 32];
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // codes that are 16 n: those of odd nibbles
                const float by = (D == 128 ? k & 1 : i) ? scale * 0.0625f : scale, back = (D == 128 ? k & 1 : i) ? 16.0f : 1.0f;
                const float2 f = T::unpack(b[k][i]);
                b[k][i] = PgF16::pack(f.x * by, f.y * by);
                const float2 h = PgF16::unpack(b[k][i]);
                const float both = (h.x + h.y) * back;
                z[k >> 1] = (k & 1) == 0 && i == 0 ? both : z[k >> 1] + both;
            }
        sum[0] = sum[1] = 0u;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            z[j] += __shfl_xor_sync(0xFFFFFFFFu, z[j], 1);
            z[j] += __shfl_xor_sync(0xFFFFFFFFu, z[j], 2);
            if (t == j) split(z[j]);
        }
    }
    __device__ __forceinline__ void split(float z) {
        z *= 1.0f / CODE_UNIT;
        sum[0] = tf32(z);
        sum[1] = tf32(z - __uint_as_float(sum[0]));
    }
    // The B operands of k-steps 2 j and 2 j + 1.
    __device__ __forceinline__ uint4 at(int j) const { return make_uint4(b[2 * j][0], b[2 * j][1], b[2 * j + 1][0], b[2 * j + 1][1]); }
    // The factor of logits of queries 2 t and 2 t + 1.
    __device__ __forceinline__ float units(float c, int e) const { return __shfl_sync(0xFFFFFFFFu, units_of(c), 8 * (threadIdx.x & 3) + 4 * e); }
    // That of query g: neither 0 nor infinity, so that a masked logit stays -infinity and one of 0 stays 0.
    __device__ __forceinline__ float units_of(float c) const { return fminf(fmaxf(c * unit, 1e-37f), 3e38f); }
};

// Products of 16 tokens' keys with eight queries: s[e] is token g + 8 (e >> 1), query 2 t + (e & 1), in the
// query's units.  at(j): the B operands of k-steps 2 j and 2 j + 1.
template <int D, typename F>
__device__ __forceinline__ void q4_logits(float (&s)[4], const KeyCodes<D> &k, uint32_t sum0, uint32_t sum1, F at) {
    mma_tf32_first(s, k.floor[0], k.floor[1], sum0, sum1);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
        const uint4 q = at(j);
        uint32_t a[2][4];
        k.frag(a[0], 2 * j);
        k.frag(a[1], 2 * j + 1);
        float c[4];
        mma_f16_first(c, a[0], q.x, q.y);
        mma_f16(c, a[1], q.z, q.w);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = fmaf(k.step[e >> 1][j], c[e], s[e]);
    }
}

}  // namespace verkv
