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
// error.  F is the double-precision frequency (pow and a product: relative error below 2^-51), so
// a position p adds p theta 2^-51 at most.
//
// Bound by HBM: x read once, y written once.  A thread keeps one 16-byte unit's place in a
// row (with halves, the unit and its partner), works out that unit's sines once and takes
// the row's heads eight at a time, every load issued before the first product: 64 us for 32760
// tokens of 24 bf16 heads of 128 (6.3 TB/s; a thread per unit, its sines worked out again for
// every head, took 74).
#include <algorithm>
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
    int units, heads_per_cta;             // units of a row that a CTA's threads take (rotated first); heads per grid y
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

constexpr int kHeads = 8;                 // heads that a CTA takes where rows are few

// VEC elements are 16 bytes.  grid (row groups, head groups); thread = (row, unit).
// kFlight heads in flight: eight units a thread either way.
template <typename T, int VEC, bool HALVES>
__global__ void __launch_bounds__(kThreads, 3) rope_kernel(const __grid_constant__ RopeArgs a) {
    dep_wait();                                          // launched dependent: see launch_dep
    dep_release();
    const int u = threadIdx.x % a.units;
    const long long r = (long long)blockIdx.x * a.rows_per_cta + threadIdx.x / a.units;
    if (threadIdx.x / a.units >= a.rows_per_cta || r >= a.rows) return;
    const int h1 = min(a.heads, ((int)blockIdx.y + 1) * a.heads_per_cta);
    union Pack { uint4 u; T e[VEC]; };
    const int nrot = HALVES ? a.pairs / VEC : 2 * a.pairs / VEC;
    const bool pass = u >= nrot;                         // a unit behind the rotated dims
    const int o = pass ? 2 * a.pairs + (u - nrot) * VEC : u * VEC, partner = a.pairs;
    const T* x = static_cast<const T*>(a.x) + r * a.xs + o;
    T* y = static_cast<T*>(a.y) + r * a.ys + o;
    constexpr int kPairs = HALVES ? VEC : VEC / 2, kFlight = HALVES ? 4 : 8;
    Pack p[kFlight], q[HALVES ? kFlight : 1];
    auto load = [&](int h0) {
#pragma unroll
        for (int e = 0; e < kFlight; ++e)
            if (h0 + e < h1) {
                p[e].u = *reinterpret_cast<const uint4*>(x + (h0 + e) * a.d);
                if (HALVES && !pass) q[HALVES ? e : 0].u = *reinterpret_cast<const uint4*>(x + (h0 + e) * a.d + partner);
            }
    };
    int h0 = blockIdx.y * a.heads_per_cta;
    load(h0);
    float2 cs[kPairs];
    if (!pass) {
        const int p0 = HALVES ? o : o / 2;
#pragma unroll
        for (int e = 0; e < kPairs; ++e) cs[e] = cos_sin(a.turn[p0 + e], a.pos[a.axis[p0 + e] * a.rows + r]);
    }
    for (;;) {
#pragma unroll
        for (int e = 0; e < kFlight; ++e)
            if (h0 + e < h1) {
                if (!pass) {
#pragma unroll
                    for (int k = 0; k < kPairs; ++k) {
                        T& e0 = p[e].e[HALVES ? k : 2 * k];
                        T& e1 = HALVES ? q[HALVES ? e : 0].e[k] : p[e].e[HALVES ? k : 2 * k + 1];
                        float y0, y1;
                        rope_pair(to_f(e0), to_f(e1), cs[k], y0, y1);
                        e0 = from_f<T>(y0);
                        e1 = from_f<T>(y1);
                    }
                    if (HALVES) *reinterpret_cast<uint4*>(y + (h0 + e) * a.d + partner) = q[HALVES ? e : 0].u;
                }
                *reinterpret_cast<uint4*>(y + (h0 + e) * a.d) = p[e].u;
            }
        h0 += kFlight;
        if (h0 >= h1) break;
        load(h0);
    }
}

// Any head size, section split and alignment of elements: a pair or a dim per item.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_pairs_kernel(const __grid_constant__ RopeArgs a) {
    extern __shared__ float2 cs[];
    dep_wait();
    dep_release();
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
            if (!std::isfinite(t)) return KVC_ERR_ARG;       // a base near 0
            a.turn[p] = (uint64_t)std::ldexp(t - std::floor(t), 64);   // (below 2^64: a double below 1 times 2^64)
            a.axis[p] = (uint8_t)i;
        }
    a.x = d_x; a.y = d_y; a.pos = d_pos; a.rows = rows;
    a.heads = heads; a.d = head_dim; a.pairs = pairs;
    a.halves = flags & KVC_ROPE_HALVES ? 1 : 0;
    a.in_place = d_x == d_y;
    const int vec = 16 / elem;
    // 16-byte units: every unit aligned and whole within the rotated dims (a half of them)
    const bool wide = aligned16(d_x) && aligned16(d_y) && head_dim % vec == 0 && a.xs % vec == 0 && a.ys % vec == 0 &&
                      (a.halves ? pairs % vec == 0 : 2 * pairs % vec == 0);
    a.units = (a.halves ? pairs : 2 * pairs) / vec + (a.in_place ? 0 : (head_dim - 2 * pairs) / vec);
    a.rows_per_cta = wide ? kThreads / a.units : 4;
    const long long groups = (rows + a.rows_per_cta - 1) / a.rows_per_cta;
    if (groups > 0x7fffffffLL) return KVC_ERR_ARG;
    // many rows: a CTA takes every head of its rows; few (a decode step): eight each, to fill the GPU,
    // or more where a grid would not hold the groups
    a.heads_per_cta = wide && groups < 608 ? std::max(kHeads, (heads + 65534) / 65535) : heads;
    const unsigned hgroups = (unsigned)((heads + a.heads_per_cta - 1) / a.heads_per_cta);
    const dim3 grid((unsigned)groups, hgroups);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t smem = (size_t)a.rows_per_cta * pairs * sizeof(float2);
    cudaError_t e = cudaSuccess;
    auto launch = [&](void (*kernel)(RopeArgs), size_t bytes) { e = launch_dep(kernel, grid, dim3(kThreads), bytes, st, a); };
    if (dtype == KVC_BF16) {
        if (!wide) launch(rope_pairs_kernel<__nv_bfloat16>, smem);
        else if (a.halves) launch(rope_kernel<__nv_bfloat16, 8, true>, 0);
        else launch(rope_kernel<__nv_bfloat16, 8, false>, 0);
    } else {
        if (!wide) launch(rope_pairs_kernel<float>, smem);
        else if (a.halves) launch(rope_kernel<float, 4, true>, 0);
        else launch(rope_kernel<float, 4, false>, 0);
    }
    return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA;
}
