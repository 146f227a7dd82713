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

// Minimum and maximum that a NaN operand makes NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// The thread's 8 dims (bf16 values) of a group that lanes 4 k .. 4 k + 3 hold: their codes, dim j in
// nibble j, and the group's (s, m).  Every lane of the warp calls it.
// The quotients: t = y r with r = 1 / s correctly rounded is within an ulp or so of y / s; the fused
// residual y - t s is exact, and t + (y - t s) r rounds correctly (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000", 1990), where neither over- nor underflows: scales
// out of [2^-100, 2^100] divide instead.  Adding 1.5 2^23 rounds to an integer, ties to even.
__device__ __forceinline__ uint32_t quantise(const float (&x)[8], uint32_t& params) {
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) { lo = min_nan(lo, x[j]); hi = max_nan(hi, x[j]); }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(hi - lo, 15.f));
    float s = __bfloat162float(sb);
    if (!(fabsf(s) < INFINITY)) {
        sb = __ushort_as_bfloat16(0x7fff);
        s = 0.f;                                       // codes 0
    }
    params = (uint32_t)__bfloat16_as_ushort(sb) | (__float_as_uint(lo) & 0xffff0000u);
    constexpr float kMagic = 12582912.f;               // 0x4B400000
    uint32_t w = 0;
    if (s >= 0x1p-100f && s <= 0x1p100f) {
        const float r = __frcp_rn(s);
#pragma unroll
        for (int j = 7; j >= 0; --j) {
            const float y = x[j] - lo, t = y * r;
            const float q = __fmaf_rn(__fmaf_rn(-t, s, y), r, t);
            w = (w << 4) + (__float_as_uint(q + kMagic) & 15u);
        }
    } else if (s > 0.f) {
#pragma unroll 1
        for (int j = 7; j >= 0; --j) {
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) v = i == j ? x[i] : v;
            w = (w << 4) + (uint32_t)fminf(rintf(__fdiv_rn(v - lo, s)), 15.f);
        }
    }
    return w;
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

// The same for 8 bf16 values, and the inverse: m + u s, rounded once to bf16.
__device__ __forceinline__ uint32_t quantise_bf16(const uint4& u, uint32_t& params) {
    const uint32_t a[4] = {u.x, u.y, u.z, u.w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) { x[2 * i] = __uint_as_float(a[i] << 16); x[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u); }
    return quantise(x, params);
}
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
    const uint32_t kw = quantise_bf16(kx, kp), vw = v_codes(quantise_bf16(vx, vp), e);
    if (there) store_unit<D>(k, v, e, kw, kp, vw, vp);
}

}  // namespace int4
}  // namespace kvc
