// int4.h -- rows of the INT4 tier: 4-bit codes with a scale and a minimum per 32 dims.
//
// A row of d dims (64 or 128) of one head in groups of 32 consecutive dims:
//     m = min x,  s = bf16((max x - min x) / 15),  u = rint((x - m) / s) in 0 .. 15,  x ~ m + u s,
// differences, quotients and roundings in fp32, ties to even; s = 0 (all values equal, or a range
// too small for a scale) gives u = 0, and a group that holds an infinity or NaN, or whose range
// passes fp32's, reads back as NaN (s = NaN).  m is one of the row's bf16 values, so it is exact;
// s off by 2^-8 leaves the largest quotient below 15.06, so |x - (m + u s)| <= s / 2.
//
// 5 d / 8 bytes: d / 2 of codes, then for each group the bf16 pair (s, m).  A row depends on no
// other row, so a cache may be trimmed, wrapped, paged and copied at any row.  The codes lie
// as the decode's matrix operands take them (d/32 = G groups):
//  K: word c G + g (c = 0..3) holds dims 32 g + 8 c + j, j = 0..7, in nibble j;
//  V: half-word r G + g (r = 0..7) holds dims 32 g + 4 r + i, i = 0..3, in nibble i.
// The threads that write or read a row take 8 dims each: thread e of d / 8 those of group e / 4,
// from 8 (e mod 4) on.  The four threads of a group are neighbouring lanes of one warp.
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

// Any scale, any values: the quotients divided out.
static __device__ __noinline__ uint32_t quantise_slowly(uint4 v, float lo, float d, uint32_t& scale) {
    __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(d, 15.f));
    const float s = __bfloat162float(sb);
    const bool number = fabsf(s) < INFINITY;
    scale = number ? __bfloat16_as_ushort(sb) : 0x7fffu;
    uint32_t w = 0;
    if (number && s > 0.f)
        for (int j = 7; j >= 0; --j) {
            const uint32_t pair = j / 2 == 0 ? v.x : j / 2 == 1 ? v.y : j / 2 == 2 ? v.z : v.w;
            const float x = __uint_as_float(j & 1 ? pair & 0xffff0000u : pair << 16);
            w = (w << 4) + (uint32_t)fminf(rintf(__fdiv_rn(x - lo, s)), 15.f);
        }
    return w;
}

// The thread's 8 dims (bf16 values) of a group that lanes 4 k .. 4 k + 3 hold: their codes, dim j in
// nibble j, and the group's (s, m).  Every lane of the warp calls it.
// Quotients: with r = 1 / s to an ulp or two, t = y r is as close to y / s; the fused residual
// y - t s is exact, and t + (y - t s) r is off by some 2^-45 before its last rounding, so a quotient half-way
// between two codes (y and s are numbers of few bits: others are further away) stays there.  The scale the same
// way, with 1 / 15 (Markstein, "Computation of elementary functions on the IBM RISC System/6000", 1990).
// Adding 1.5 2^23 rounds to an integer, ties to even, in a float's last bits.
// About 60 instructions for 8 values, half of them on pairs (min2 on the bf16 values, fp32 pairs behind): with
// two values' instructions apart, divisions and an exact reciprocal, 140, a bf16 cache of 66,000 rows of 8 heads of 128 was handed
// over in 89 us.
__device__ __forceinline__ uint32_t quantise(const uint4& v, uint32_t& params) {
    const uint32_t a[4] = {v.x, v.y, v.z, v.w};
    constexpr uint32_t kSigns = 0x80008000u;
    const uint32_t lo2 = min2(min2(a[0], a[1]), min2(a[2], a[3]));
    const uint32_t hi2 = min2(min2(a[0] ^ kSigns, a[1] ^ kSigns), min2(a[2] ^ kSigns, a[3] ^ kSigns));    // of -x
    uint32_t r2 = min2(__byte_perm(lo2, hi2, 0x5410), __byte_perm(lo2, hi2, 0x7632));                      // (min x, min -x)
    r2 = min2(r2, __shfl_xor_sync(0xffffffffu, r2, 1));
    r2 = min2(r2, __shfl_xor_sync(0xffffffffu, r2, 2));
    const float lo = __uint_as_float(r2 << 16), d = -(__uint_as_float(r2 & 0xffff0000u) + lo);
    params = r2 << 16;
    if (!(d >= 0x1p-96f && d <= 0x1p100f)) {               // (equal values, and what is not a number, too)
        uint32_t scale;
        const uint32_t w = quantise_slowly(v, lo, d, scale);
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
    const float2 lo_ = make_float2(-lo, -lo), s_ = make_float2(-s, -s), r_ = make_float2(r, r);
    constexpr float kMagic = 12582912.f;                   // 0x4B400000
    uint32_t f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 y = __fadd2_rn(make_float2(__uint_as_float(a[i] << 16), __uint_as_float(a[i] & 0xffff0000u)), lo_);
        const float2 t = __fmul2_rn(y, r_);
        const float2 q = __fadd2_rn(__ffma2_rn(__ffma2_rn(t, s_, y), r_, t), make_float2(kMagic, kMagic));
        f[2 * i] = __float_as_uint(q.x);
        f[2 * i + 1] = __float_as_uint(q.y);
    }
    const uint32_t even = __byte_perm(__byte_perm(f[0], f[2], 0x0040), __byte_perm(f[4], f[6], 0x0040), 0x5410);
    const uint32_t odd = __byte_perm(__byte_perm(f[1], f[3], 0x0040), __byte_perm(f[5], f[7], 0x0040), 0x5410);
    return even + odd * 16u;
}

// Where thread e's word of codes goes: K's word holds its 8 dims; of V's two half-words (r = 2 c and
// 2 c + 1) the threads of groups 2 k and 2 k + 1, four lanes apart, swap one, so that each writes a word.
template <int D>
__device__ __forceinline__ int k_word(int e) { return (e & 3) * (D / kGroup) + (e >> 2); }
template <int D>
__device__ __forceinline__ int v_word(int e) {         // the word that thread e writes
    return (2 * (e & 3) + (e >> 2 & 1)) * (D / 64) + (e >> 3);
}
__device__ __forceinline__ uint32_t v_codes(uint32_t w, int e) {
    const bool odd = e >> 2 & 1;                       // of an odd group: takes r = 2 c + 1
    const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? w & 0xffffu : w >> 16, 4);
    return odd ? (other & 0xffffu) | (w & 0xffff0000u) : (w & 0xffffu) | other << 16;
}

// Swapping is its own inverse: from the words at v_word it gives each thread its 8 codes again.

// The inverse: 8 values m + u s, rounded once to bf16.
__device__ __forceinline__ uint4 values_bf16(uint32_t w, uint32_t params) {
    const float s = __uint_as_float(params << 16), m = __uint_as_float(params & 0xffff0000u);
    uint32_t a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(__fmaf_rn((float)(w >> 8 * i & 15u), s, m),
                                                       __fmaf_rn((float)(w >> (8 * i + 4) & 15u), s, m));
        a[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    return make_uint4(a[0], a[1], a[2], a[3]);
}

// Thread e's words and, from one thread a group, its parameters into a K and a V row.
template <int D>
__device__ __forceinline__ void store_unit(char* k, char* v, int e, uint32_t kw, uint32_t kp, uint32_t vw, uint32_t vp) {
    reinterpret_cast<uint32_t*>(k)[k_word<D>(e)] = kw;
    reinterpret_cast<uint32_t*>(v)[v_word<D>(e)] = vw;
    if ((e & 3) == 0) {
        reinterpret_cast<uint32_t*>(k + D / 2)[e >> 2] = kp;
        reinterpret_cast<uint32_t*>(v + D / 2)[e >> 2] = vp;
    }
}

// Thread e's 16 bytes of a K and a V row, quantised and stored (all lanes of the warp calling).
template <int D>
__device__ __forceinline__ void store_row(char* k, char* v, int e, const uint4& kx, const uint4& vx, bool there) {
    uint32_t kp, vp;
    const uint32_t kw = quantise(kx, kp), vw = v_codes(quantise(vx, vp), e);
    if (there) store_unit<D>(k, v, e, kw, kp, vw, vp);
}

}  // namespace int4
}  // namespace kvc
