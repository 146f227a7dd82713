// rope.cu -- rotary positions with several axes: every pair of a head's dims turns by the
// position on one axis (time, height, width of an image or video token; one axis is plain
// RoPE) times the pair's frequency.  A cache with rope_base 0 stores keys as given, so
// queries and keys rotated here go through every other call unchanged.
//
// The angle of a far position has to be exact to a fraction of a turn, which fp32 cannot
// hold and fp64 is slow at.  The host gives each pair's frequency in turns per position
// as a 64-bit fixed-point fraction F (theta / 2 pi mod 1, scaled by 2^64); position * F
// mod 2^64 is the angle in turns with wrap-around for free (one 64-bit multiply).  Its top
// 32 bits, read as a signed number, are the angle in half turns on [-1, 1) times 2^31:
// sincospif of that is off by less than 2^-24 pi from the rounding to fp32, plus its own
// error.  F is the double-precision frequency, so a position p adds p theta 2^-53.
//
// Bound by HBM: x read once, y written once.  The sines of a row are shared by all heads,
// so a CTA computes them once for a few rows into shared memory, and its threads then
// stream the rows in 16-byte units.
#include <cmath>
#include <cstring>

#include "kvc_internal.h"

namespace kvc {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;            // head_dim <= 256
constexpr int kMaxAxes = 8;

struct RopeArgs {
    const void* x;
    void* y;
    const int32_t* pos;                   // [axes][rows]
    long long rows, xs, ys;               // row strides in elements
    int heads, d, pairs, rows_per_cta, halves, in_place;
    uint64_t turn[kMaxPairs];             // frequency, turns per position * 2^64
    uint8_t axis[kMaxPairs];
};

__device__ __forceinline__ float2 cos_sin(uint64_t turn, int32_t p) {
    const uint64_t t = turn * (uint64_t)(int64_t)p;
    float s, c;
    sincospif((float)(int32_t)(uint32_t)(t >> 32) * 0x1p-31f, &s, &c);
    return make_float2(c, s);
}

template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f(float x) { return x; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }

// VEC elements are 16 bytes.  grid (row groups, head groups): a CTA's sines serve its
// rows' heads [h0, h1).  Work item: one head's unit of a row; with halves, a unit of the
// first half and its partner in the second.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
    extern __shared__ float2 cs[];                        // [rows_per_cta][pairs]
    const long long r0 = (long long)blockIdx.x * a.rows_per_cta;
    const int nr = (int)min((long long)a.rows_per_cta, a.rows - r0);
    for (int i = threadIdx.x; i < nr * a.pairs; i += kThreads) {
        const int r = i / a.pairs, p = i % a.pairs;
        cs[i] = cos_sin(a.turn[p], a.pos[a.axis[p] * a.rows + r0 + r]);
    }
    __syncthreads();
    const int hper = (a.heads + gridDim.y - 1) / gridDim.y, h0 = blockIdx.y * hper;
    const int nh = min(a.heads - h0, hper);
    if (nh <= 0) return;
    const T* X = static_cast<const T*>(a.x);
    T* Y = static_cast<T*>(a.y);
    union Pack { uint4 u; T e[VEC]; };
    const int rot = 2 * a.pairs;
    // units of a head: rotated ones (pairs of units with halves), then those that pass through
    const int nrot = a.halves ? a.pairs / VEC : rot / VEC, units = nrot + (a.in_place ? 0 : (a.d - rot) / VEC);
    const int total = nr * nh * units;
    for (int i = threadIdx.x; i < total; i += kThreads) {
        const int u = i % units, rh = i / units, r = rh / nh, h = h0 + rh % nh;
        const T* x = X + (r0 + r) * a.xs + (long long)h * a.d;
        T* y = Y + (r0 + r) * a.ys + (long long)h * a.d;
        const float2* c = cs + r * a.pairs;
        if (u >= nrot) {
            const int o = rot + (u - nrot) * VEC;
            *reinterpret_cast<uint4*>(y + o) = *reinterpret_cast<const uint4*>(x + o);
        } else if (a.halves) {
            const int o = u * VEC;
            Pack p, q;
            p.u = *reinterpret_cast<const uint4*>(x + o);
            q.u = *reinterpret_cast<const uint4*>(x + a.pairs + o);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float y0, y1;
                rope_pair(to_f(p.e[e]), to_f(q.e[e]), c[o + e], y0, y1);
                p.e[e] = from_f<T>(y0);
                q.e[e] = from_f<T>(y1);
            }
            *reinterpret_cast<uint4*>(y + o) = p.u;
            *reinterpret_cast<uint4*>(y + a.pairs + o) = q.u;
        } else {
            const int o = u * VEC;
            Pack p;
            p.u = *reinterpret_cast<const uint4*>(x + o);
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
                float y0, y1;
                rope_pair(to_f(p.e[e]), to_f(p.e[e + 1]), c[(o + e) / 2], y0, y1);
                p.e[e] = from_f<T>(y0);
                p.e[e + 1] = from_f<T>(y1);
            }
            *reinterpret_cast<uint4*>(y + o) = p.u;
        }
    }
}

// Any head size, section split and alignment of elements: a pair or a dim per item.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_pairs_kernel(const __grid_constant__ RopeArgs a) {
    extern __shared__ float2 cs[];
    const long long r0 = (long long)blockIdx.x * a.rows_per_cta;
    const int nr = (int)min((long long)a.rows_per_cta, a.rows - r0);
    for (int i = threadIdx.x; i < nr * a.pairs; i += kThreads) {
        const int r = i / a.pairs, p = i % a.pairs;
        cs[i] = cos_sin(a.turn[p], a.pos[a.axis[p] * a.rows + r0 + r]);
    }
    __syncthreads();
    const int hper = (a.heads + gridDim.y - 1) / gridDim.y, h0 = blockIdx.y * hper;
    const int nh = min(a.heads - h0, hper);
    if (nh <= 0) return;
    const int rot = 2 * a.pairs, items = a.pairs + (a.in_place ? 0 : a.d - rot);
    for (int i = threadIdx.x; i < nr * nh * items; i += kThreads) {
        const int k = i % items, rh = i / items, r = rh / nh, h = h0 + rh % nh;
        const T* x = static_cast<const T*>(a.x) + (r0 + r) * a.xs + (long long)h * a.d;
        T* y = static_cast<T*>(a.y) + (r0 + r) * a.ys + (long long)h * a.d;
        if (k >= a.pairs) {
            y[rot + k - a.pairs] = x[rot + k - a.pairs];
        } else {
            const int i0 = a.halves ? k : 2 * k, i1 = a.halves ? a.pairs + k : 2 * k + 1;
            float y0, y1;
            rope_pair(to_f(x[i0]), to_f(x[i1]), cs[r * a.pairs + k], y0, y1);
            y[i0] = from_f<T>(y0);
            y[i1] = from_f<T>(y1);
        }
    }
}

}  // namespace
}  // namespace kvc

using namespace kvc;

extern "C" int kvc_rope_axes(const void* d_x, int64_t x_stride, void* d_y, int64_t y_stride, int32_t dtype, int64_t rows,
                             int32_t heads, int32_t head_dim, const int32_t* d_pos, int32_t n_axes,
                             const int32_t* h_sections, double base, int32_t flags, kvc_stream_t stream) {
    if ((dtype != KVC_F32 && dtype != KVC_BF16) || rows < 0 || heads < 1 || head_dim < 2 || head_dim > 256 || head_dim % 2 ||
        n_axes < 1 || n_axes > kMaxAxes || !h_sections || (flags & ~(KVC_ROPE_HALVES | KVC_ROPE_PER_AXIS)) ||
        !(base > 0.0) || std::isinf(base))
        return KVC_ERR_ARG;
    RopeArgs a{};
    int pairs = 0;
    for (int i = 0; i < n_axes; ++i) {
        if (h_sections[i] < 1 || h_sections[i] > head_dim / 2 - pairs) return KVC_ERR_ARG;
        pairs += h_sections[i];
    }
    const long long width = (long long)heads * head_dim;
    a.xs = x_stride ? x_stride : width;
    a.ys = y_stride ? y_stride : width;
    if (a.xs < width || a.ys < width || width > (1 << 24)) return KVC_ERR_ARG;
    if (rows == 0) return KVC_OK;
    if (rows > (1LL << 31) || a.xs > (1LL << 31) || a.ys > (1LL << 31)) return KVC_ERR_ARG;
    if (!d_x || !d_y || !d_pos) return KVC_ERR_ARG;
    const int elem = dtype == KVC_BF16 ? 2 : 4;
    // a row may be rotated where it lies, never across another one
    const char *x0 = static_cast<const char*>(d_x), *y0 = static_cast<const char*>(d_y);
    const char *x1 = x0 + ((rows - 1) * a.xs + width) * elem, *y1 = y0 + ((rows - 1) * a.ys + width) * elem;
    if ((reinterpret_cast<uintptr_t>(d_x) | reinterpret_cast<uintptr_t>(d_y)) % elem || reinterpret_cast<uintptr_t>(d_pos) % 4)
        return KVC_ERR_ARG;
    if (x0 == y0 ? (a.xs != a.ys && rows > 1) : (x0 < y1 && y0 < x1)) return KVC_ERR_ARG;
    int p = 0;
    for (int i = 0; i < n_axes; ++i)
        for (int j = 0; j < h_sections[i]; ++j, ++p) {
            const double e = (flags & KVC_ROPE_PER_AXIS) ? (double)j / h_sections[i] : (double)p / pairs;
            const double t = std::pow(base, -e) * 0.15915494309189533577;   // turns per position: theta / 2 pi
            const double f = t - std::floor(t);
            const double scaled = std::ldexp(f, 64);
            a.turn[p] = scaled >= 18446744073709551615.0 ? 0 : (uint64_t)scaled;
            a.axis[p] = (uint8_t)i;
        }
    a.x = d_x; a.y = d_y; a.pos = d_pos; a.rows = rows;
    a.heads = heads; a.d = head_dim; a.pairs = pairs;
    a.halves = flags & KVC_ROPE_HALVES ? 1 : 0;
    a.in_place = d_x == d_y;
    a.rows_per_cta = 4;
    const long long groups = (rows + a.rows_per_cta - 1) / a.rows_per_cta;
    if (groups > 0x7fffffffLL) return KVC_ERR_ARG;
    const size_t smem = (size_t)a.rows_per_cta * pairs * sizeof(float2);
    const int vec = 16 / elem;
    // 16-byte units: every unit aligned and whole within the rotated dims (a half of them)
    const bool wide = aligned16(d_x) && aligned16(d_y) && head_dim % vec == 0 && a.xs % vec == 0 && a.ys % vec == 0 &&
                      (a.halves ? pairs % vec == 0 : 2 * pairs % vec == 0);
    const dim3 grid((unsigned)groups, 1);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == KVC_BF16) {
        if (wide) rope_kernel<__nv_bfloat16, 8><<<grid, kThreads, smem, st>>>(a);
        else rope_pairs_kernel<__nv_bfloat16><<<grid, kThreads, smem, st>>>(a);
    } else {
        if (wide) rope_kernel<float, 4><<<grid, kThreads, smem, st>>>(a);
        else rope_pairs_kernel<float><<<grid, kThreads, smem, st>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? KVC_OK : KVC_ERR_CUDA;
}
