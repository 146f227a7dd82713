// prompt.cu -- packed prompts: the rows of every request, each request with a count of its
// own, appended to the cache and attended causally in one call.
//
// [PREFIX] "哪些東西必須一起裁剪" for a batch whose requests have cuts and suffix lengths of
// their own: request b brings n_b rows (possibly none), packed behind those of request
// b - 1; its row i sits at position p = c_b + i, c_b its next_position, and attends to
// positions [max(0, p - W + 1), p] ([LEAN] §2.1), those below c_b from the cache.
// Keys and queries are rotated in fp32 and rounded to the cache's type, the query as its
// key is: both products then take the cache's own type.
//
// Rows of one (request, KV head) are (token, query head of the group) pairs, token-major:
// a tile of query rows holds a few tokens' whole groups, so a group's heads share every
// key and value read, and short prompts still fill a tile.
//
// On a ring of W slots, appending first would evict rows that early queries need
// ([LEAN] §3.4): the rotated rows are staged beside the resident rows from the cut
// rounded down to 16, attended, and appended afterwards, as the chunk call does.
#include <algorithm>
#include <cmath>
#include <vector>

#include "prompt.h"

namespace kvc {
namespace {

constexpr int kThreads = 256;
struct RowArgs {
    const void* k; const void* v;         // packed rows, stride kv_stride, keys not rotated
    long long stride;
    void* kc; void* vc;                   // cache rows
    __nv_bfloat16* wk; __nv_bfloat16* wv; // ring staging [B][Hkv][ws_rows][d]
    const int32_t* table;
    int32_t* pos;
    const int32_t* next_pos;              // the cut: advanced after every kernel of the call
    const float2* rope;
    uint32_t* hdr;
    int Hkv, d, S, P, ring, bf16, ws_rows;
    int stage;                            // 1: into the staging rows, with the resident rows they follow
    const void* q;                        // packed queries to rotate into `out` for the tensor-core kernel (else nullptr):
    __nv_bfloat16* out;                   // head h of packed row t at (t Hq + h) out_head elements
    long long q_stride;
    int Hq, out_head;
};

// Whether request b's row at p may be written: the host checked what it knows, but a captured
// call replayed too often passes the capacity, or the pages mapped when it was captured.
__device__ __forceinline__ bool position_ok(const RowArgs& a, int b, long long p) {
    if (!(p >= 0 && p <= 0x7ffffffeLL && (a.ring || p < a.S) && (!a.rope || p < a.P))) return false;
    return !a.table || __ldg(a.table + (size_t)b * (a.S / kPage) + (int)(p % a.S) / kPage) >= 0;
}

// Four pairs of a bf16 row, rotated in fp32, each product and sum rounded once.
__device__ __forceinline__ uint4 turned(const uint4 u, const float2* cs) {
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float y0, y1;
        rope_pair(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u), cs[e], y0, y1);
        const __nv_bfloat162 o2 = __floats2bfloat162_rn(y0, y1);
        w[e] = *reinterpret_cast<const uint32_t*>(&o2);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kRowsPerCta = 8;

// Rows of any head size and type, a pair per item.  grid (row groups of the longest request,
// requests).  RoPE in fp32, each product and sum rounded once, one rounding to the cache's
// type: the arithmetic of the other appends.
__global__ void __launch_bounds__(kThreads) prompt_pairs_kernel(const RowArgs a, const __grid_constant__ Packed g) {
    dep_wait();                                        // launched dependent (see launch_dep).  No early release: the
                                                       // attention, placed while rows are still written, took 6 us longer
    const int bi = blockIdx.y, b = g.b0 + bi;
    const int n = g.off[bi + 1] - g.off[bi];
    const int cut = a.next_pos[b], d = a.d;
    const int lead = a.stage ? cut & 15 : 0;                    // resident rows staged before the first new one
    const int r0 = blockIdx.x * kRowsPerCta - lead;
    if (n == 0 || r0 >= n) return;
    const int rows = min(n - r0, kRowsPerCta);
    const int per = d / 2, total = rows * a.Hkv * per;
    for (int i = threadIdx.x; i < total; i += kThreads) {
        const int c = i % per, h = (i / per) % a.Hkv, r = r0 + i / (per * a.Hkv);
        const long long p = (long long)cut + r;
        if (!a.stage && a.ring && r < n - a.S) continue;        // overwritten later in this call
        if (!position_ok(a, b, p)) { atomicOr(a.hdr, kErrPosition); continue; }
        const int slot = a.ring ? (int)(p % a.S) : (int)p;
        const size_t crow = kv_row(a.table, b, h, slot, a.Hkv, a.S) * d;
        const size_t dst = a.stage ? stage_row(b, h, (int)p, cut, a.Hkv, a.ws_rows) * d : crow;
        void* kd = a.stage ? a.wk : a.kc;
        void* vd = a.stage ? a.wv : a.vc;
        const size_t src = (size_t)(g.row0 + g.off[bi] + r) * a.stride + (size_t)h * d;   // (used for r >= 0)
        float k0, k1, v0, v1;
        if (r < 0) {
            k0 = ld_elem(a.kc, crow + 2 * c, a.bf16); k1 = ld_elem(a.kc, crow + 2 * c + 1, a.bf16);
            v0 = ld_elem(a.vc, crow + 2 * c, a.bf16); v1 = ld_elem(a.vc, crow + 2 * c + 1, a.bf16);
        } else {
            k0 = ld_elem(a.k, src + 2 * c, a.bf16); k1 = ld_elem(a.k, src + 2 * c + 1, a.bf16);
            v0 = ld_elem(a.v, src + 2 * c, a.bf16); v1 = ld_elem(a.v, src + 2 * c + 1, a.bf16);
            if (a.rope) {
                const float x0 = k0, x1 = k1;
                rope_pair(x0, x1, a.rope[(size_t)p * (d / 2) + c], k0, k1);
            }
        }
        if (a.bf16) {
            reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(kd) + dst)[c] = __floats2bfloat162_rn(k0, k1);
            reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(vd) + dst)[c] = __floats2bfloat162_rn(v0, v1);
        } else {
            reinterpret_cast<float2*>(static_cast<float*>(kd) + dst)[c] = make_float2(k0, k1);
            reinterpret_cast<float2*>(static_cast<float*>(vd) + dst)[c] = make_float2(v0, v1);
        }
        if (!a.stage && h == 0 && c == 0) a.pos[(size_t)b * a.S + slot] = (int)p;
    }
}

// bf16 rows with d a multiple of 8, in 16-byte units: the same arithmetic.  Bound by HBM: 11,000
// rows of 32 + 2 x 8 heads of 128 in 40 us, 6.5 TB/s.  A
// thread holds one unit of a row's {cos, sin} and takes kHeads heads of that row, every load
// issued first.  grid (row groups of the longest request, requests, head groups: those of the
// rotated queries (where the tensor-core attention takes them), then those of keys and
// values); a CTA covers 256 / (d / 8) rows.
constexpr int kHeads = 8;

__global__ void __launch_bounds__(kThreads) prompt_rows_kernel(const RowArgs a, const __grid_constant__ Packed g) {
    dep_wait();                                        // (no early release, as above: 7 us for 12,000 ragged rows)
    const int bi = blockIdx.y, b = g.b0 + bi;
    const int n = g.off[bi + 1] - g.off[bi];
    const int cut = a.next_pos[b], d = a.d, per = d / 8;
    const int lead = a.stage ? cut & 15 : 0;                    // resident rows staged before the first new one
    const int c = threadIdx.x % per, r = blockIdx.x * (kThreads / per) + threadIdx.x / per - lead;
    if (threadIdx.x / per >= kThreads / per || r >= n) return;
    const long long p = (long long)cut + r;
    if (!position_ok(a, b, p)) { atomicOr(a.hdr, kErrPosition); return; }
    float2 cs[4] = {};
    if (a.rope && r >= 0) {
        const float4* rp = reinterpret_cast<const float4*>(a.rope + (size_t)p * (d / 2) + 4 * c);
        const float4 c0 = __ldg(rp), c1 = __ldg(rp + 1);
        cs[0] = make_float2(c0.x, c0.y); cs[1] = make_float2(c0.z, c0.w);
        cs[2] = make_float2(c1.x, c1.y); cs[3] = make_float2(c1.z, c1.w);
    }
    const long long t = g.row0 + g.off[bi] + r;                 // (packed row, for r >= 0)
    const int qgroups = a.q ? (a.Hq + kHeads - 1) / kHeads : 0;
    uint4 u[kHeads];
    if ((int)blockIdx.z < qgroups) {
        if (r < 0) return;
        const int h0 = blockIdx.z * kHeads, nh = min(kHeads, a.Hq - h0);
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + t * a.q_stride + (size_t)h0 * d + 8 * c);
        __nv_bfloat16* dst = a.out + (t * a.Hq + h0) * a.out_head + 8 * c;
#pragma unroll
        for (int h = 0; h < kHeads; ++h)
            if (h < nh) u[h] = __ldg(src + h * per);
#pragma unroll
        for (int h = 0; h < kHeads; ++h)
            if (h < nh) *reinterpret_cast<uint4*>(dst + (size_t)h * a.out_head) = turned(u[h], cs);
        return;
    }
    if (!a.stage && a.ring && r < n - a.S) return;              // overwritten later in this call
    const int h0 = ((int)blockIdx.z - qgroups) * (kHeads / 2), nh = min(kHeads / 2, a.Hkv - h0);
    const int slot = a.ring ? (int)(p % a.S) : (int)p;
    // heads of a row lie S rows apart (16 in a page), of the staging area ws_rows
    const size_t crow = kv_row(a.table, b, h0, slot, a.Hkv, a.S), cstep = a.table ? kPage : a.S;
    const size_t drow = a.stage ? stage_row(b, h0, (int)p, cut, a.Hkv, a.ws_rows) : crow, dstep = a.stage ? (size_t)a.ws_rows : cstep;
    const __nv_bfloat16* ks = r < 0 ? static_cast<const __nv_bfloat16*>(a.kc) + crow * d : static_cast<const __nv_bfloat16*>(a.k) + t * a.stride + (size_t)h0 * d;
    const __nv_bfloat16* vs = r < 0 ? static_cast<const __nv_bfloat16*>(a.vc) + crow * d : static_cast<const __nv_bfloat16*>(a.v) + t * a.stride + (size_t)h0 * d;
    const size_t sstep = r < 0 ? cstep * d : d;
#pragma unroll
    for (int h = 0; h < kHeads / 2; ++h)
        if (h < nh) {
            u[2 * h] = *reinterpret_cast<const uint4*>(ks + h * sstep + 8 * c);
            u[2 * h + 1] = *reinterpret_cast<const uint4*>(vs + h * sstep + 8 * c);
        }
    __nv_bfloat16* kd = (a.stage ? a.wk : static_cast<__nv_bfloat16*>(a.kc)) + drow * d + 8 * c;
    __nv_bfloat16* vd = (a.stage ? a.wv : static_cast<__nv_bfloat16*>(a.vc)) + drow * d + 8 * c;
#pragma unroll
    for (int h = 0; h < kHeads / 2; ++h)
        if (h < nh) {
            *reinterpret_cast<uint4*>(kd + h * dstep * d) = a.rope && r >= 0 ? turned(u[2 * h], cs) : u[2 * h];
            *reinterpret_cast<uint4*>(vd + h * dstep * d) = u[2 * h + 1];
        }
    if (!a.stage && h0 == 0 && c == 0) a.pos[(size_t)b * a.S + slot] = (int)p;
}

__global__ void prompt_advance_kernel(int32_t* next_pos, const __grid_constant__ Packed g) {
    dep_wait();
    dep_release();
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < g.nb) next_pos[g.b0 + i] += g.off[i + 1] - g.off[i];
}

// Joins the parts of split keys: a warp per (row, head); lanes over the dims.
__global__ void __launch_bounds__(256) prompt_join_kernel(const AttnArgs a, long long row0, long long rows) {
    dep_wait();
    dep_release();
    const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5), at = row0 + i;
    const int lane = threadIdx.x & 31;
    if (i >= rows) return;
    const float2* ml = a.part_ml + at * a.parts;
    float m = -INFINITY;
    for (int q = 0; q < a.parts; ++q) m = fmaxf(m, ml[q].x);
    float l = 0.f, o[8] = {};
    for (int q = 0; q < a.parts; ++q) {
        const float2 x = ml[q];
        if (x.y == 0.f) continue;                     // the part holds no key that the row sees
        const float f = x.x == -INFINITY ? 1.f : exp2f(x.x - m);    // (no finite score: its sum is not a number)
        l += f * x.y;
        const float* acc = a.part_acc + (at * a.parts + q) * a.d;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (32 * e + lane < a.d) o[e] += f * acc[32 * e + lane];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int x = 32 * e + lane;
        if (x >= a.d) continue;
        const float v = o[e] / l;
        if (a.out_bf16) static_cast<__nv_bfloat16*>(a.out)[at * a.d + x] = __float2bfloat16_rn(v);
        else static_cast<float*>(a.out)[at * a.d + x] = v;
    }
}

// ---- attention on the CUDA cores: fp32 caches and other head sizes ------------------
// CTA = 8 R query rows (token, head) of one (request, KV head); 8 warps of R rows.  Tiles of 64
// keys in shared memory as fp32; a lane scores two keys, then holds a run of the output's
// dims; the running maximum and sum of a row live in its warp.  Everything in fp32.
// Bound by what shared memory returns to registers, 4 cycles a 16-byte load of a warp: with
// R = 8, 10 loads feed 64 products of each lane in the scores and 12 feed 128 in P.V (products:
// 16 and 32 cycles); with R = 4 6 feed 32 and 8 feed 64.  So R = 8 wherever CTAs of
// 64 rows fill the SMs.  Half warps of 8 x 4 and 8 x 8 products a lane load less, but with half
// the warps they took longer: 1090 against 950 us (4 requests of 2000 rows, 8 fp32 heads of
// 128: 35 TFLOP/s), where one CTA after the other and no loads ahead took 2050.
// The next tile's keys are copied while the values of this one are used, its values while the
// next scores are.  CTAs start in the order of the keys that they see, most first (1130 -> 950).
constexpr int kBN = 64;

__host__ __device__ constexpr int round4(int d) { return (d + 3) & ~3; }
// keys: rows of an odd number of 16-byte units, so that 8 lanes read 8 rows without conflicts
__host__ __device__ constexpr int key_step(int d) { return round4(d) / 4 % 2 ? round4(d) : round4(d) + 4; }
__host__ __device__ constexpr size_t simt_smem(int d, int R) {
    return ((size_t)(8 * R + kBN) * round4(d) + (size_t)kBN * key_step(d) + 8 * R * kBN) * 4;
}

__device__ __forceinline__ void copy16(float* dst, const float* src, bool there) {
    const int n = there ? 16 : 0;                     // 0: zeros, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(n) : "memory");
}

enum { kLoadPairs, kLoadAsync, kLoadWide };           // rows of pairs; fp32 rows of 16-byte units; bf16 ones

// DIMS: 64 (head_dim up to it), 128 or 256.  SINKS: the first tiles hold those of the first positions
// that lie before the window of the CTA's first row; sinks in that window's tiles stay in sight there.
template <int DIMS, int R, int LOAD, bool SINKS>
__global__ void __launch_bounds__(kThreads, DIMS <= 128 ? 2 : 1) prompt_simt_kernel(const AttnArgs a, const __grid_constant__ Packed g) {
    constexpr int kBM = 8 * R, VW = DIMS == 64 ? 2 : 4, NV = DIMS == 256 ? 2 : 1;      // a lane's dims: NV runs of VW
    extern __shared__ float4 smem4[];
    dep_wait();
    dep_release();
    const int bi = blockIdx.x / a.Hkv, b = g.b0 + bi, h = blockIdx.x % a.Hkv;
    const int n = g.off[bi + 1] - g.off[bi];
    // the rows that see most keys first (of all requests); their keys in parts
    const int part = (int)blockIdx.y % a.parts;
    const long long at_tile = (long long)blockIdx.z * (gridDim.y / a.parts) + blockIdx.y / a.parts;
    const long long all = (long long)n * a.g, row0 = ((all + kBM - 1) / kBM - 1 - at_tile) * kBM;
    if (row0 < 0) return;
    const int d = a.d, d4 = round4(d), kp = key_step(d);
    float* sQ = reinterpret_cast<float*>(smem4);
    float* sK = sQ + kBM * d4;
    float* sV = sK + kBN * kp;
    float* sP = sV + kBN * d4;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cut = a.next_pos[b];
    const int nrow = (int)min((long long)kBM, all - row0);
    const int p_first = cut + (int)(row0 / a.g), p_last = cut + (int)((row0 + nrow - 1) / a.g);
    const int kmin = a.W > 0 ? max(0, p_first - a.W + 1) : 0;
    const int cal = cut & ~15;
    const int sunk = SINKS ? min(a.sinks, kmin) : 0, nsunk = (sunk + kBN - 1) / kBN;
    const int tiles = p_last >= kmin ? nsunk + (p_last - kmin) / kBN + 1 : 0;
    auto first_of = [&](int j) { return SINKS && j < nsunk ? kBN * j - kmin : kBN * (j - nsunk); };   // of a tile, from kmin
    const int j0 = (int)((long long)tiles * part / a.parts), ntiles = (int)((long long)tiles * (part + 1) / a.parts);

    // rows of tile j into shared memory (what: 0 keys, 1 values), eight lanes a row
    auto fill = [&](int j, int what) {
        // (positions past the capacity, flagged before, have no rows to read)
        const int kb = kmin + first_of(j), left = (a.ring ? p_last : min(p_last, a.S - 1)) - kb;
        float* dst = what ? sV : sK;
        const int step = what ? d4 : kp;
#pragma unroll
        for (int half = 0; half < kBN / 32; ++half) {
            const int r = 32 * half + tid / 8, c0 = tid % 8, key = kb + r;
            const bool there = r <= left, staged = there && a.ring && key >= cal;
            const size_t row = !there ? 0 : (staged ? stage_row(b, h, key, cut, a.Hkv, a.ws_rows)
                                                    : kv_row(a.table, b, h, a.ring ? key % a.S : key, a.Hkv, a.S)) * d;
            const void* src = staged ? (what ? static_cast<const void*>(a.wv) : a.wk) : (what ? a.vc : a.kc);
            if constexpr (LOAD == kLoadAsync) {
                const float* x = static_cast<const float*>(src) + row;
#pragma unroll 8
                for (int c = c0; c < d / 4; c += 8) copy16(dst + r * step + 4 * c, x + 4 * c, there);
            } else if constexpr (LOAD == kLoadWide) {
                const uint4* x = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(src) + row);
#pragma unroll 4
                for (int c = c0; c < d / 8; c += 8) {
                    const uint4 u = there ? x[c] : make_uint4(0, 0, 0, 0);
                    float4* y = reinterpret_cast<float4*>(dst + r * step + 8 * c);
                    y[0] = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
                    y[1] = make_float4(__uint_as_float(u.z << 16), __uint_as_float(u.z & 0xffff0000u),
                                       __uint_as_float(u.w << 16), __uint_as_float(u.w & 0xffff0000u));
                }
            } else {
#pragma unroll 4
                for (int c = c0; c < d4 / 2; c += 8) {
                    const bool in = there && 2 * c < d;
                    *reinterpret_cast<float2*>(dst + r * step + 2 * c) =
                        in ? make_float2(ld_elem(src, row + 2 * c, a.bf16), ld_elem(src, row + 2 * c + 1, a.bf16)) : make_float2(0.f, 0.f);
                }
            }
        }
    };
    auto landed = [&]() {
        if constexpr (LOAD == kLoadAsync) asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
    };

    if (j0 < ntiles) fill(j0, 0);
    // queries, rotated and rounded to the cache's type
#pragma unroll 4
    for (int i = tid; i < kBM * (d4 / 2); i += kThreads) {
        const int r = i / (d4 / 2), c = i % (d4 / 2);
        float y0 = 0.f, y1 = 0.f;
        if (r < nrow && 2 * c < d) {
            const int t = (int)((row0 + r) / a.g), hq = h * a.g + (int)((row0 + r) % a.g);
            const size_t src = (size_t)(g.row0 + g.off[bi] + t) * a.q_stride + (size_t)hq * d + 2 * c;
            const float x0 = ld_elem(a.q, src, a.bf16), x1 = ld_elem(a.q, src + 1, a.bf16);
            y0 = x0; y1 = x1;
            const long long p = (long long)cut + t;
            if (a.rope && p < a.P) rope_pair(x0, x1, a.rope[(size_t)p * (d / 2) + c], y0, y1);
            if (a.bf16) { y0 = __bfloat162float(__float2bfloat16_rn(y0)); y1 = __bfloat162float(__float2bfloat16_rn(y1)); }
        }
        *reinterpret_cast<float2*>(sQ + r * d4 + 2 * c) = make_float2(y0, y1);
    }
    // the warp's rows: positions relative to kmin (-1: no row) and first visible keys
    int p[R], lo[R];
    float m[R], l[R];
    float2 acc[R][NV * VW / 2];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int rr = R * warp + r, at = cut + (int)((row0 + rr) / a.g);
        p[r] = rr < nrow ? at - kmin : -1;
        lo[r] = a.W > 0 ? max(0, at - a.W + 1) - kmin : 0;
        m[r] = -INFINITY; l[r] = 0.f;
#pragma unroll
        for (int e = 0; e < NV * VW / 2; ++e) acc[r][e] = make_float2(0.f, 0.f);
    }
    float* myP = sP + R * warp * kBN;
    for (int j = j0; j < ntiles; ++j) {
        landed();                         // keys of this tile; the values before are used
        fill(j, 1);
        float2 s2[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r) s2[r][0] = s2[r][1] = make_float2(0.f, 0.f);
#pragma unroll 2
        for (int c = 0; c < d4; c += 4) {
            const float4 k0 = *reinterpret_cast<const float4*>(sK + lane * kp + c);
            const float4 k1 = *reinterpret_cast<const float4*>(sK + (lane + 32) * kp + c);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float4 q = *reinterpret_cast<const float4*>(sQ + (R * warp + r) * d4 + c);
                s2[r][0] = __ffma2_rn(make_float2(q.x, q.y), make_float2(k0.x, k0.y), s2[r][0]);
                s2[r][1] = __ffma2_rn(make_float2(q.x, q.y), make_float2(k1.x, k1.y), s2[r][1]);
                s2[r][0] = __ffma2_rn(make_float2(q.z, q.w), make_float2(k0.z, k0.w), s2[r][0]);
                s2[r][1] = __ffma2_rn(make_float2(q.z, q.w), make_float2(k1.z, k1.w), s2[r][1]);
            }
        }
        const int kb = first_of(j);       // (relative to kmin)
        // keys c of the tile that a row sees by the sinks: those below this
        const int cs = !SINKS ? 0 : j < nsunk ? sunk - kmin - kb : a.sinks - kmin - kb;
        bool whole = true;                // every key of the tile visible to every row of the warp
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c0 = SINKS && j < nsunk ? kBN : lo[r] - kb, c1 = p[r] - kb;      // visible: keys c0 .. c1 of the tile
            const bool in0 = (lane >= c0 || (SINKS && lane < cs)) && lane <= c1;
            const bool in1 = (lane + 32 >= c0 || (SINKS && lane + 32 < cs)) && lane + 32 <= c1;
            whole = whole && c0 <= 0 && c1 >= kBN - 1;
            const float x0 = in0 ? (s2[r][0].x + s2[r][0].y) * a.scale_log2 : -INFINITY;
            const float x1 = in1 ? (s2[r][1].x + s2[r][1].y) * a.scale_log2 : -INFINITY;
            float mx = fmaxf(x0, x1);
            for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            mx = fmaxf(mx, m[r]);
            const float base = mx == -INFINITY ? 0.f : mx;        // nothing visible so far: every weight 0
            const float alpha = exp2f(m[r] - base), w0 = exp2f(x0 - base), w1 = exp2f(x1 - base);
            m[r] = mx;
            l[r] = l[r] * alpha + (w0 + w1);                      // the lane's keys; joined at the end
#pragma unroll
            for (int e = 0; e < NV * VW / 2; ++e) acc[r][e] = make_float2(acc[r][e].x * alpha, acc[r][e].y * alpha);
            myP[r * kBN + lane] = w0;
            myP[r * kBN + lane + 32] = w1;
        }
        landed();                         // values of this tile; its keys are used
        if (j + 1 < ntiles) fill(j + 1, 0);
        auto weigh = [&](int c, bool all_seen) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int x = VW * (32 * v + lane);
                if (x >= d4) continue;
                float2 w4[4][VW / 2];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if constexpr (VW == 2) {
                        w4[e][0] = *reinterpret_cast<const float2*>(sV + (c + e) * d4 + x);
                    } else {
                        const float4 y = *reinterpret_cast<const float4*>(sV + (c + e) * d4 + x);
                        w4[e][0] = make_float2(y.x, y.y); w4[e][VW / 2 - 1] = make_float2(y.z, y.w);
                    }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float4 w = *reinterpret_cast<const float4*>(myP + r * kBN + c);
                    const float we[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // a masked key adds nothing, whatever its value row holds
                        if (!all_seen && (((SINKS && j < nsunk) || kb + c + e < lo[r]) && !(SINKS && c + e < cs))) continue;
                        if (!all_seen && kb + c + e > p[r]) continue;
#pragma unroll
                        for (int q = 0; q < VW / 2; ++q)
                            acc[r][v * VW / 2 + q] = __ffma2_rn(make_float2(we[e], we[e]), w4[e][q], acc[r][v * VW / 2 + q]);
                    }
                }
            }
        };
        if (whole) {
#pragma unroll 2
            for (int c = 0; c < kBN; c += 4) weigh(c, true);
        } else {
#pragma unroll 1
            for (int c = 0; c < kBN; c += 4) weigh(c, false);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float sum = l[r];
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (p[r] < 0) continue;
        const int rr = R * warp + r, t = (int)((row0 + rr) / a.g), hq = h * a.g + (int)((row0 + rr) % a.g);
        const size_t row = (size_t)(g.row0 + g.off[bi] + t) * a.Hq + hq, at = row * d;
        if (a.parts > 1 && lane == 0) a.part_ml[row * a.parts + part] = make_float2(m[r], sum);
#pragma unroll
        for (int e = 0; e < NV * VW; ++e) {
            const int x = VW * (32 * (e / VW) + lane) + e % VW;
            if (x >= d) continue;
            const float y = e % 2 ? acc[r][e / 2].y : acc[r][e / 2].x, o = y / sum;
            if (a.parts > 1) a.part_acc[(row * a.parts + part) * d + x] = y;        // unnormalised, to be joined
            else if (a.out_bf16) static_cast<__nv_bfloat16*>(a.out)[at + x] = __float2bfloat16_rn(o);
            else static_cast<float*>(a.out)[at + x] = o;
        }
    }
}

template <int DIMS, int R, int LOAD>
cudaError_t launch_rows(const AttnArgs& a, const Packed& g, int most, cudaStream_t st) {
    auto kernel = a.sinks ? prompt_simt_kernel<DIMS, R, LOAD, true> : prompt_simt_kernel<DIMS, R, LOAD, false>;
    if (cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), simt_smem(DIMS, R))) return e;
    const long long tiles = ((long long)most * a.g + 8 * R - 1) / (8 * R), per = std::min<long long>(tiles, 65535 / a.parts);
    const dim3 grid((unsigned)(a.Hkv * g.nb), (unsigned)(per * a.parts), (unsigned)((tiles + per - 1) / per));
    return launch_dep(kernel, grid, dim3(kThreads), simt_smem(a.d, R), st, a, g);
}

template <int DIMS>
cudaError_t launch_simt(const AttnArgs& a, const Packed& g, int most, bool tall, cudaStream_t st) {
    const int load = a.bf16 ? (a.d % 8 == 0 ? kLoadWide : kLoadPairs) : (a.d % 4 == 0 ? kLoadAsync : kLoadPairs);
    switch (load) {
        case kLoadAsync: return tall ? launch_rows<DIMS, 8, kLoadAsync>(a, g, most, st) : launch_rows<DIMS, 4, kLoadAsync>(a, g, most, st);
        case kLoadWide: return tall ? launch_rows<DIMS, 8, kLoadWide>(a, g, most, st) : launch_rows<DIMS, 4, kLoadWide>(a, g, most, st);
        default: return launch_rows<DIMS, 4, kLoadPairs>(a, g, most, st);
    }
}

cudaError_t launch_attention(const kvc_handle* h, const AttnArgs& args, const Packed& g, int most, cudaStream_t st) {
    AttnArgs a = args;
    // CTAs of 64 rows where they fill the SMs, else of 32 (two requests of 1000 rows, 8 heads of
    // 256: 347 against 410 us).  Few CTAs split their keys, two tiles each at least (a row behind
    // 2000 keys: 161 -> 31 us), as far as the workspace of the decode's split reaches.  The
    // host's lengths choose the shape and the split only.
    long long ctas[2] = {0, 0}, seen = 0;
    for (int i = 0; i < g.nb; ++i) {
        const long long n = g.off[i + 1] - g.off[i];
        for (int t = 0; t < 2; ++t) ctas[t] += (n * a.g + 32 * t + 31) / (32 * t + 32) * a.Hkv;
        if (n > 0) seen = std::max(seen, h->np[g.b0 + i] + n);
    }
    const bool tall = ctas[1] >= h->num_sms;
    const long long longest = (a.W > 0 ? std::min(seen, (long long)a.W + a.sinks + 64) : seen) / kBN + 1;
    const long long room = (long long)h->sh.B * h->sh.max_splits / g.off[g.nb];
    a.parts = (int)std::max(1ll, std::min({2 * h->num_sms / ctas[tall], longest / 2, room, (long long)kMaxKeyParts}));
    if (a.parts > 1) split_workspace(h, g, a.parts, &a);
    const cudaError_t e = a.d <= 64    ? launch_simt<64>(a, g, most, tall, st)
                          : a.d <= 128 ? launch_simt<128>(a, g, most, tall, st)
                                       : launch_simt<256>(a, g, most, tall, st);
    return e == cudaSuccess && a.parts > 1 ? launch_join(a, g, st) : e;
}

}  // namespace

void split_workspace(const kvc_handle* h, const Packed& g, int parts, AttnArgs* a) {
    a->parts = parts;
    const long long first = g.row0 * a->Hq * parts;
    a->part_ml = reinterpret_cast<float2*>(h->state + h->L.part_ml) - first;
    a->part_acc = reinterpret_cast<float*>(h->state + h->L.part_acc) - first * a->d;
}

cudaError_t launch_join(const AttnArgs& a, const Packed& g, cudaStream_t st) {
    const long long rows = (long long)g.off[g.nb] * a.Hq;
    return launch_dep(prompt_join_kernel, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, st, a, g.row0 * a.Hq, rows);
}

bool prompt_supported(const Shape& s) {
    return !s.int8 && !s.int4 && s.Hq <= kMaxGridHeads && (!s.ring || (s.bf16 && s.S % kPage == 0));
}

cudaError_t launch_prompt(kvc_handle* h, const PromptArgs& p, const int32_t* counts, cudaStream_t st) {
    const Shape& s = h->sh;
    auto at = [&](size_t off) { return h->state + off; };
    RowArgs r{};
    r.k = p.k; r.v = p.v; r.stride = p.kv_stride;
    r.kc = at(h->L.k); r.vc = at(h->L.v);
    if (s.ring) {
        r.ws_rows = chunk_ws_rows(s);
        r.wk = reinterpret_cast<__nv_bfloat16*>(at(h->L.cws));
        r.wv = r.wk + (size_t)s.B * s.Hkv * r.ws_rows * s.d;
    }
    r.table = s.pages ? reinterpret_cast<const int32_t*>(at(h->L.table)) : nullptr;
    r.pos = reinterpret_cast<int32_t*>(at(h->L.pos));
    int32_t* next_pos = reinterpret_cast<int32_t*>(at(h->L.next_pos));
    r.next_pos = next_pos;
    r.rope = s.rope ? reinterpret_cast<const float2*>(at(h->L.rope)) : nullptr;
    r.hdr = reinterpret_cast<uint32_t*>(at(h->L.hdr));
    r.Hkv = s.Hkv; r.d = s.d; r.S = s.S; r.P = s.P; r.ring = s.ring; r.bf16 = s.bf16;
    AttnArgs a{};
    a.q = p.q; a.out = p.out; a.q_stride = p.q_stride;
    a.kc = r.kc; a.vc = r.vc; a.wk = r.wk; a.wv = r.wv; a.table = r.table; a.next_pos = next_pos; a.rope = r.rope;
    a.hdr = r.hdr;
    a.Hq = s.Hq; a.Hkv = s.Hkv; a.g = s.g; a.d = s.d; a.S = s.S; a.W = s.W; a.P = s.P; a.ring = s.ring; a.bf16 = s.bf16;
    a.out_bf16 = s.out_bf16; a.ws_rows = r.ws_rows;
    a.parts = 1;
    a.sinks = s.sinks;
    a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)s.d));
    // the entry point checked alignment and strides
    const bool vec = s.bf16 && s.d % 8 == 0;
    const bool tensor = prompt_tc_supported(s);
    if (tensor && s.rope) {
        r.q = p.q; r.q_stride = p.q_stride; r.Hq = s.Hq;
        r.out = static_cast<__nv_bfloat16*>(p.out);
        r.out_head = s.out_bf16 ? s.d : 2 * s.d;
    }
    long long row0 = 0;
    for (int b0 = 0; b0 < s.B; b0 += kPromptGroup) {
        static thread_local Packed g;
        g.b0 = b0;
        g.nb = std::min(s.B - b0, kPromptGroup);
        g.row0 = row0;
        int most = 0;
        g.off[0] = 0;
        for (int i = 0; i < g.nb; ++i) {
            g.off[i + 1] = g.off[i] + counts[b0 + i];
            most = std::max(most, counts[b0 + i]);
        }
        row0 += g.off[g.nb];
        if (most == 0) continue;
        cudaError_t e = cudaSuccess;
        auto rows = [&](int stage) {
            r.stage = stage;
            const int longest = most + (stage ? 15 : 0), per_cta = vec ? kThreads / (s.d / 8) : kRowsPerCta;
            const int groups = (r.q ? (s.Hq + kHeads - 1) / kHeads : 0) + (s.Hkv + kHeads / 2 - 1) / (kHeads / 2);
            const dim3 grid((longest + per_cta - 1) / per_cta, g.nb, vec ? groups : 1);
            return launch_dep(vec ? prompt_rows_kernel : prompt_pairs_kernel, grid, dim3(kThreads), 0, st, r, g);
        };
        if ((e = rows(s.ring ? 1 : 0)) != cudaSuccess) return e;
        e = tensor ? launch_prompt_tc(h, a, g, st) : launch_attention(h, a, g, most, st);
        if (e != cudaSuccess) return e;
        if (s.ring) {
            r.q = nullptr;                                // d_out holds the output by now
            if ((e = rows(0)) != cudaSuccess) return e;
            r.q = tensor && s.rope ? p.q : nullptr;
        }
        if ((e = launch_dep(prompt_advance_kernel, dim3((g.nb + 255) / 256), dim3(256), 0, st, next_pos, g)) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace kvc
