// int4.h -- rows of the INT4 tier: 4-bit codes with a scale and a minimum per 32 dims.
//
// A row of d dims (64 or 128) of one head in groups of 32 consecutive dims:
//     m = min x,  s = bf16((max x - min x) / 15),  u = rint((x - m) / s) in 0 .. 15,  x ~ m + u s,
// differences, quotients and roundings in fp32, ties to even; s = 0 (all values equal, or a range
// too small for a scale) gives u = 0, and a group that holds an infinity or NaN, or whose range
// passes fp32's, reads back as NaN (s = NaN).  m is one of the row's bf16 values, so it is exact;
// s off by 2^-8 leaves the largest quotient below 15.06, so |x - (m + u s)| <= s / 2.
// That is for s >= 2^-126: a subnormal s, or one that underflows, is off by more, and x by the group's range at most.
//
// 5 d / 8 bytes: d / 2 of codes, then for each group the bf16 pair (s, m).  A row depends on no
// other row, so a cache may be trimmed, wrapped, paged and copied at any row.  The codes lie
// as the decode's matrix operands take them (d/32 = G groups):
//  K: word c G + g (c = 0..3) holds dims 32 g + 8 c + j, j = 0..7, in nibble j;
//  V: half-word r G + g (r = 0..7) holds dims 32 g + 4 r + i, i = 0..3, in nibble i.
// The threads that write or read a row take 16 dims each, as two chunks of 8: thread e of d / 16 chunks
// c = e mod 2 and c + 2 of group e / 2.  The two threads of a group are neighbouring lanes of one warp.
#pragma once

#include "kvc_internal.h"

namespace kvc {
namespace int4 {

constexpr int kGroup = 32;                 // dims that share a scale and a minimum
__host__ __device__ constexpr int row_size(int d) { return d / 8 * 5; }

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {       // of two bf16 pairs; NaN where either is
    uint32_t y;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}

// Any scale, any values: the quotients divided out.
static __device__ __noinline__ uint2 quantise_slowly(uint4 x, uint4 y, float lo, float d, uint32_t& scale) {
    const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(d, 15.f));
    const float s = __bfloat162float(sb);
    const bool number = fabsf(s) < INFINITY;
    scale = number ? __bfloat16_as_ushort(sb) : 0x7fffu;
    const uint32_t a[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    uint32_t w[2] = {0, 0};
    if (number && s > 0.f)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v0 = __uint_as_float(a[i] << 16), v1 = __uint_as_float(a[i] & 0xffff0000u);
            w[i / 4] |= (uint32_t)fminf(rintf(__fdiv_rn(v0 - lo, s)), 15.f) << 8 * (i % 4);
            w[i / 4] |= (uint32_t)fminf(rintf(__fdiv_rn(v1 - lo, s)), 15.f) << (8 * (i % 4) + 4);
        }
    return make_uint2(w[0], w[1]);
}

// Codes of a chunk of 8 values y / s, dim j in nibble j: minus = (-m, -m), r = (1 / s, 1 / s), s = (-s, -s).
// With 1 / s to an ulp or two, t = y r is as close to y / s; the fused residual y - t s is exact, and
// t + (y - t s) r is off by some 2^-45 before its last rounding, so a quotient half-way between two codes
// (y and s are numbers of few bits: others are further away) stays there.  Adding 1.5 2^23 rounds to an
// integer, ties to even, in a float's last bits.
__device__ __forceinline__ uint32_t codes_of(const uint4& x, float2 minus, float2 r, float2 s) {
    const uint32_t a[4] = {x.x, x.y, x.z, x.w};
    constexpr float kMagic = 12582912.f;                   // 0x4B400000
    uint32_t f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 y = __fadd2_rn(make_float2(__uint_as_float(a[i] << 16), __uint_as_float(a[i] & 0xffff0000u)), minus);
        const float2 t = __fmul2_rn(y, r);
        const float2 q = __fadd2_rn(__ffma2_rn(__ffma2_rn(t, s, y), r, t), make_float2(kMagic, kMagic));
        f[2 * i] = __float_as_uint(q.x);
        f[2 * i + 1] = __float_as_uint(q.y);
    }
    const uint32_t even = __byte_perm(__byte_perm(f[0], f[2], 0x0040), __byte_perm(f[4], f[6], 0x0040), 0x5410);
    const uint32_t odd = __byte_perm(__byte_perm(f[1], f[3], 0x0040), __byte_perm(f[5], f[7], 0x0040), 0x5410);
    return even + odd * 16u;
}

// The thread's two chunks (bf16 values) of a group: their codes, and the group's (s, m).  Every lane of the warp calls it.
// The scale is divided as the quotients are, with 1 / 15 (Markstein, "Computation of elementary functions on
// the IBM RISC System/6000", 1990).
__device__ __forceinline__ uint2 quantise(const uint4& x, const uint4& y, uint32_t& params) {
    const uint32_t lo2 = min2(min2(min2(x.x, x.y), min2(x.z, x.w)), min2(min2(y.x, y.y), min2(y.z, y.w)));
    const uint32_t hi2 = max2(max2(max2(x.x, x.y), max2(x.z, x.w)), max2(max2(y.x, y.y), max2(y.z, y.w))) ^ 0x80008000u;
    uint32_t r2 = min2(__byte_perm(lo2, hi2, 0x5410), __byte_perm(lo2, hi2, 0x7632));      // (min x, -max x)
    r2 = min2(r2, __shfl_xor_sync(0xffffffffu, r2, 1));
    const float lo = __uint_as_float(r2 << 16), d = -(__uint_as_float(r2 & 0xffff0000u) + lo);
    params = r2 << 16;
    if (!(d >= 0x1p-96f && d <= 0x1p100f)) {               // (equal values, and what is not a number, too)
        uint32_t scale;
        const uint2 w = quantise_slowly(x, y, lo, d, scale);
        params |= scale;
        return w;
    }
    constexpr float k15 = 1.f / 15.f;
    const float d15 = d * k15;
    const __nv_bfloat16 sb = __float2bfloat16_rn(__fmaf_rn(__fmaf_rn(-15.f, d15, d), k15, d15));
    const float s = __bfloat162float(sb);
    params |= __bfloat16_as_ushort(sb);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    const float2 minus = make_float2(-lo, -lo), s_ = make_float2(-s, -s), r_ = make_float2(r, r);
    return make_uint2(codes_of(x, minus, r_, s_), codes_of(y, minus, r_, s_));
}

// Where thread e's words of codes go.  K's words hold a chunk each, c + 2 two steps of G words behind c.  Of a
// chunk's two half-words in V (r = 2 c and 2 c + 1) the threads of groups 2 k and 2 k + 1, two lanes apart,
// swap one, so that each writes a word; chunk c + 2's lies four rows of half-words behind.
template <int D>
__device__ __forceinline__ int k_word(int e) { return (e & 1) * (D / kGroup) + (e >> 1); }
template <int D>
__device__ __forceinline__ int v_word(int e) { return (2 * (e & 1) + (e >> 1 & 1)) * (D / 64) + (e >> 2); }
template <int D> constexpr int kSecondK = 2 * (D / kGroup);
template <int D> constexpr int kSecondV = 4 * (D / 64);

// From a chunk's codes to the word that the thread writes in V; its own inverse.
__device__ __forceinline__ uint32_t v_codes(uint32_t w, int e) {
    const bool odd = e >> 1 & 1;                       // of an odd group: takes r = 2 c + 1
    const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? w & 0xffffu : w >> 16, 2);
    return odd ? (other & 0xffffu) | (w & 0xffff0000u) : (w & 0xffffu) | other << 16;
}

// 8 values m + u s, rounded once to bf16.  Codes become the bf16 numbers 128 + u, then u; the fused multiply-add
// of bf16 pairs rounds once.
__device__ __forceinline__ uint4 values_bf16(uint32_t w, uint32_t params) {
    const uint32_t even = w & 0x0f0f0f0fu, odd = w >> 4 & 0x0f0f0f0fu;
    const uint32_t s2 = __byte_perm(params, 0, 0x1010), m2 = __byte_perm(params, 0, 0x3232);
    constexpr uint32_t kBias = 0x43004300u, kMinusBias = 0xc300c300u, kOne = 0x3f803f80u;
    uint32_t a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t u, x;
        asm("prmt.b32 %0, %1, %2, %3;" : "=r"(u) : "r"(even), "r"(odd), "r"(0xc480u + 0x1111u * i));   // (8 + k: the top bit of byte k, 0)
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(x) : "r"(u | kBias), "r"(kOne), "r"(kMinusBias));
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(a[i]) : "r"(x), "r"(s2), "r"(m2));
    }
    return make_uint4(a[0], a[1], a[2], a[3]);
}

// What thread e has of a K and a V row.
struct Unit {
    uint2 k, v;                                        // words
    uint32_t kp, vp;                                   // parameters of its group
};

__device__ __forceinline__ Unit quantise(const uint4 (&k)[2], const uint4 (&v)[2], int e) {
    Unit u;
    u.k = quantise(k[0], k[1], u.kp);
    u.v = quantise(v[0], v[1], u.vp);
    u.v = make_uint2(v_codes(u.v.x, e), v_codes(u.v.y, e));
    return u;
}

template <int D>
__device__ __forceinline__ void store(char* k, char* v, int e, const Unit& u) {
    uint32_t* kw = reinterpret_cast<uint32_t*>(k) + k_word<D>(e);
    uint32_t* vw = reinterpret_cast<uint32_t*>(v) + v_word<D>(e);
    kw[0] = u.k.x;
    kw[kSecondK<D>] = u.k.y;
    vw[0] = u.v.x;
    vw[kSecondV<D>] = u.v.y;
    if ((e & 1) == 0) {
        reinterpret_cast<uint32_t*>(k + D / 2)[e >> 1] = u.kp;
        reinterpret_cast<uint32_t*>(v + D / 2)[e >> 1] = u.vp;
    }
}

template <int D>
__device__ __forceinline__ Unit load(const char* k, const char* v, int e) {
    const uint32_t* kw = reinterpret_cast<const uint32_t*>(k) + k_word<D>(e);
    const uint32_t* vw = reinterpret_cast<const uint32_t*>(v) + v_word<D>(e);
    Unit u;
    u.k = make_uint2(kw[0], kw[kSecondK<D>]);
    u.v = make_uint2(vw[0], vw[kSecondV<D>]);
    u.kp = reinterpret_cast<const uint32_t*>(k + D / 2)[e >> 1];
    u.vp = reinterpret_cast<const uint32_t*>(v + D / 2)[e >> 1];
    return u;
}

// The 16-byte unit of a bf16 row that is thread e's first chunk; the second lies two units behind.
__device__ __forceinline__ int chunk_of(int e) { return 4 * (e >> 1) + (e & 1); }

}  // namespace int4
}  // namespace kvc
