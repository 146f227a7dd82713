// int4.cu -- the INT4 tier: rows quantised as they are appended, and decode attention over them.
//
// Rows (int4.h): per head and token 5 d / 8 bytes of K and as many of V, 4-bit codes u with a
// bf16 scale s and minimum m per 32 dims g.  With x = m + u s the products split into sums over
// codes, which are small integers, and terms per group (t a key, h a head):
//     score_t   = sum_g s_tg (q_g . u_tg) + m_tg sum(q_g),
//     out_x     = sum_t p_t s_tg u_tx + sum_t p_t m_tg          (x in group g).
#include <algorithm>
#include <cmath>

#include "async_copy.h"
#include "int4.h"

namespace kvc {
namespace {

constexpr int kThreads = 256;

// ---- appends ---------------------------------------------------------------------------------
__device__ __forceinline__ void flag(uint32_t* hdr, uint32_t bit) { atomicOr(hdr, bit); }

__device__ __forceinline__ bool position_ok(const AppendArgs& a, long long p) {
    return p >= 0 && p <= 0x7fffffffLL && (a.ring || p < a.S) && (!a.rope || p < a.P);
}

// Page of `slot` of request b, < 0 if none is mapped (a captured call replayed past its pages).
__device__ __forceinline__ int slot_page(const AppendArgs& a, int b, int slot) {
    return a.table ? a.table[(size_t)b * (a.S / kPage) + slot / kPage] : 0;
}

__device__ __forceinline__ size_t slot_row(const AppendArgs& a, int b, int h, int slot, int page) {
    return a.table ? ((size_t)page * a.Hkv + h) * kPage + slot % kPage : ((size_t)b * a.Hkv + h) * a.S + slot;
}

// Chunk c (8 dims) of a key rotated at position p, rounded to bf16 as in the bf16 cache.
__device__ __forceinline__ uint4 turned(const AppendArgs& a, const uint4 u, int p, int c) {
    const float4* rp = reinterpret_cast<const float4*>(a.rope + (size_t)p * (a.d / 2) + 4 * c);
    const float4 c0 = __ldg(rp), c1 = __ldg(rp + 1);
    const float2 cs[4] = {make_float2(c0.x, c0.y), make_float2(c0.z, c0.w), make_float2(c1.x, c1.y), make_float2(c1.z, c1.w)};
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float y0, y1;
        rope_pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u), cs[i], y0, y1);
        const __nv_bfloat162 o2 = __floats2bfloat162_rn(y0, y1);
        w[i] = *reinterpret_cast<const uint32_t*>(&o2);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One token per request: a CTA per request, a thread per 16 dims of a head.
template <int D>
__global__ void __launch_bounds__(kThreads) int4_token_kernel(const AppendArgs a) {
    dep_wait();                                        // launched dependent: see launch_dep
    dep_release();
    const int b = blockIdx.x, p = a.next_pos[b];
    const int slot = a.ring ? p % a.S : p;
    const bool ok = position_ok(a, p);
    const int page = ok ? slot_page(a, b, slot) : -1;
    if (page < 0) {                                    // (the whole CTA)
        if (threadIdx.x == 0) flag(a.hdr, kErrPosition);
        return;
    }
    constexpr int kVec = D / 16;
    const int n = a.Hkv * kVec;
    const uint4* K = static_cast<const uint4*>(a.k) + (size_t)b * 2 * n;
    const uint4* V = static_cast<const uint4*>(a.v) + (size_t)b * 2 * n;
    for (int base = 0; base < n; base += kThreads) {   // (a warp's lanes stay together)
        const int i = base + threadIdx.x, h = i < n ? i / kVec : 0, e = i % kVec, c = int4::chunk_of(e);
        uint4 k[2] = {}, v[2] = {};
        if (i < n) {
            const size_t at = (size_t)h * (D / 8) + c;
            k[0] = __ldg(K + at); k[1] = __ldg(K + at + 2);
            v[0] = __ldg(V + at); v[1] = __ldg(V + at + 2);
            if (a.rope) { k[0] = turned(a, k[0], p, c); k[1] = turned(a, k[1], p, c + 2); }
        }
        const int4::Unit u = int4::quantise(k, v, e);
        const size_t o = slot_row(a, b, h, slot, page) * int4::row_size(D);
        if (i < n) int4::store<D>(static_cast<char*>(a.kc) + o, static_cast<char*>(a.vc) + o, e, u);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        a.pos[(size_t)b * a.S + slot] = p;
        a.next_pos[b] = p + 1;
    }
}

// Bound by the instructions of the quantiser and HBM alike: 64000 rows of 8 heads of 128 in 59 us (5.8 TB/s).
// Many rows: grid (groups of kRowsUnroll x 256 / (D / 16) rows, KV heads, requests), a thread per 16 dims of every
// 256 / (D / 16)-th row of its group, their loads all issued first.  next_position is advanced by the launch that follows.
constexpr int kRowsUnroll = 2;

template <int D>
__global__ void __launch_bounds__(kThreads) int4_rows_kernel(const AppendArgs a, const __grid_constant__ RowCounts g) {
    dep_wait();                                        // (no early release, as the bf16 appends)
    constexpr int kVec = D / 16, kStep = kThreads / kVec;
    const int bi = blockIdx.z, b = g.b0 + bi, h = blockIdx.y, cnt = g.val[bi];
    const int r0 = blockIdx.x * (kRowsUnroll * kStep);
    if (r0 >= cnt) return;
    const int e = threadIdx.x % kVec, c = int4::chunk_of(e), np = a.next_pos[b];
    // rows [skip, fit): those before are overwritten later in this call (a ring), those behind have no place (replays)
    const int skip = a.ring ? cnt - a.S : 0;
    const int fit = (int)min((long long)cnt, min(a.ring ? 1ll << 31 : (long long)a.S, a.rope ? (long long)a.P : 1ll << 31) - np);
    uint4 k[kRowsUnroll][2], v[kRowsUnroll][2];
    int to[kRowsUnroll];                               // the row's slot, -1: no row, or none that stays
#pragma unroll
    for (int j = 0; j < kRowsUnroll; ++j) {
        const int r = r0 + j * kStep + threadIdx.x / kVec;
        k[j][0] = k[j][1] = v[j][0] = v[j][1] = make_uint4(0, 0, 0, 0);
        to[j] = -1;
        if (r >= fit && r < cnt) flag(a.hdr, kErrPosition);
        if (r >= fit || r < skip) continue;
        to[j] = a.ring ? (np + r) % a.S : np + r;
        const size_t src = (size_t)b * a.sb + (size_t)h * a.sh + (size_t)r * a.sr + 8 * (size_t)c;
        const uint4* K = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.k) + src);
        const uint4* V = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.v) + src);
        k[j][0] = __ldg(K); k[j][1] = __ldg(K + 2);
        v[j][0] = __ldg(V); v[j][1] = __ldg(V + 2);
    }
    int page[kRowsUnroll];
#pragma unroll
    for (int j = 0; j < kRowsUnroll; ++j) page[j] = to[j] < 0 ? -1 : slot_page(a, b, to[j]);
#pragma unroll
    for (int j = 0; j < kRowsUnroll; ++j) {
        const int p = np + r0 + j * kStep + threadIdx.x / kVec;
        if (a.rope && to[j] >= 0) { k[j][0] = turned(a, k[j][0], p, c); k[j][1] = turned(a, k[j][1], p, c + 2); }
        if (to[j] >= 0 && page[j] < 0) flag(a.hdr, kErrPosition);
        const int4::Unit u = int4::quantise(k[j], v[j], e);
        if (page[j] < 0) continue;
        const size_t o = slot_row(a, b, h, to[j], page[j]) * int4::row_size(D);
        int4::store<D>(static_cast<char*>(a.kc) + o, static_cast<char*>(a.vc) + o, e, u);
        if (h == 0 && e == 0) a.pos[(size_t)b * a.S + to[j]] = p;
    }
}

// ---- decode ------------------------------------------------------------------------------------
// Bound by the matrix instructions and the ALU pipe, close to the memory's rate: 8 requests of 131072 keys, 8 KV
// heads of 128, 32 query heads in 256 us (5.2 TB/s; copies alone 198).  An SM takes some 270 cycles for a tile of 32 keys,
// 32 matrix instructions of 8 and 360 ALU instructions of 2 on each of its quarters for four of them.
// CTA = 4 warps = a split of the keys of one request and KV head, for up to 8 of its query heads; a warp
// streams tiles of 32 keys through its stages of shared memory by bulk copies (a page, or 16 rows, is
// contiguous).  Both products on the tensor cores (mma m16n8k16, fp16 operands, fp32
// accumulation), operands unpacked in registers from the words that a lane loads.  A nibble
// masked out of its 16-bit half is the fp16 number u 2^-24, one four bits higher u 2^-20, both exact
// (subnormal) and without a bias, so a word's 8 codes take four ANDs and a shift; the factor 16 of
// every other one is taken back in the query, or in the output.
//  * scores, transposed: S^T[16 keys][cols] = U[16][32 dims of g] . Q^T, the query times log2(e)/sqrt(d) and
//    a power of two that puts its largest value below 2^15.  It enters in two fp16 parts, 21 significant
//    bits: up to 4 heads as columns (head, hi) and (head, lo), up to 8 as columns of two instructions (one part
//    of 11 bits: rings of 32768, 64 query heads, 49 us, with both parts of query and weights 57).  The groups' sums are weighed by
//    s_tg and joined by the lane that holds head and keys;
//  * P.V, transposed: O^T[16 dims of g][heads] += U^T . P_g^T, P_g = p s_tg times a power of two of the head's
//    group (norm) in two fp16 parts as the query's, brought from score order to operand order by movmatrix.
//    The norm starts high and falls when a weight would pass 2^15, to put the largest at 2^9:
//    weights down to 2^-23 of the largest stay normal.  It rises as earlier weights fall behind a
//    softmax reference that moves.  The terms p m_tg are summed in fp32.
// Row r of a fragment of 16 keys stands for key tok(r): rows are 80 bytes apart (d = 128), and with this
// order the lanes' 16-byte loads of K (rows r, r + 1 together) and 8-byte loads of V (rows 0, 2, 4, 6
// together) fall into different banks.
// Lane L: g = L / 4 (fragment row), qd = L % 4 (its head, or its heads 2 qd and 2 qd + 1).
constexpr int kWarps = 4;
constexpr int kTile = 32;
constexpr float kLazyMax = 4.f;                          // log2-domain headroom of the reference maximum
// The highest norm: a weight, 2^kLazyMax at most, stays within fp32 with it, and the least normal scale (2^-126) leaves weights down
// to 2^-8 normal in fp16.
constexpr int kNormMost = 120;

__device__ __forceinline__ int tok(int r) { return r & 1 ? 8 + ((r + 3) & 7) : r; }      // rows 0..7; row r + 8: tok(r) + 1

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float fmax3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// D (16x8, fp32) = A (16x16, fp16, row) . B (16x8, fp16, col) + C
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// 8 x 8 matrix of 16-bit elements, transposed across the warp.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// The four pairs of codes of a word: pair i is nibble i of its low and of its high half.
struct Pairs {
    uint32_t x[4];                                       // times 2^-24, 2^-20, 2^-24, 2^-20
};
__device__ __forceinline__ Pairs pairs_of(uint32_t w) {
    const uint32_t v = w >> 8;
    return Pairs{{w & 0x000f000fu, w & 0x00f000f0u, v & 0x000f000fu, v & 0x00f000f0u}};
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    const __half2 t = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&t);
}

// The leading 11 bits of a pair, exact in fp16 from 2^-14 on, and what they leave.
__device__ __forceinline__ float2 first_part(float2 x) {
    return make_float2(__uint_as_float(__float_as_uint(x.x) & 0xffffe000u), __uint_as_float(__float_as_uint(x.y) & 0xffffe000u));
}
__device__ __forceinline__ float2 rest_of(float2 x, float2 first) { return __ffma2_rn(first, make_float2(-1.f, -1.f), x); }

__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((127 + e) << 23); }      // -126 .. 127

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// HL: heads per lane (1: up to 4 heads of the CTA, 2: up to 8).
template <int D, int HL>
struct I4 {
    static constexpr int G = D / int4::kGroup;           // groups of a row
    static constexpr int ROW = int4::row_size(D);
    static constexpr int HALF = kTile * ROW;             // K (or V) rows of a stage
    static constexpr int STAGEB = 2 * HALF;
    static constexpr int STAGES = 2;
    static constexpr int WARPB = STAGES * STAGEB;
    static constexpr int HEADS = 4 * HL;
    static constexpr int PARTF = HEADS * (D + 2);        // a warp's partial (m, l, acc), in its stages at the end
    static_assert(PARTF * 4 <= WARPB, "partial must fit in the warp's stages");
    static constexpr int OFF_Q = kWarps * WARPB;         // query [HEADS][D] fp32
    static constexpr int OFF_SUM = OFF_Q + HEADS * D * 4; // its sums and largest magnitudes over a group [2][HEADS][G]
    static constexpr int OFF_BAR = OFF_SUM + 2 * HEADS * G * 4;
    static constexpr size_t SMEM = OFF_BAR + kWarps * STAGES * 8;
    static_assert(HALF % 16 == 0 && kPage * ROW % 16 == 0, "bulk copies");
};

template <int D, int HL, bool PAGED>
__global__ void __launch_bounds__(kWarps * 32, HL == 1 || D == 64 ? 4 : 3) int4_decode_kernel(const DecodeArgs a, const int chunks) {
    using C = I4<D, HL>;
    constexpr int G = C::G;
    extern __shared__ __align__(128) unsigned char smem[];
    float* sQ = reinterpret_cast<float*>(smem + C::OFF_Q);
    float* sSum = reinterpret_cast<float*>(smem + C::OFF_SUM);
    float* sTop = sSum + C::HEADS * G;
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.z, kvh = blockIdx.y / chunks, chunk = blockIdx.y % chunks;
    // the CTA's query heads: [h0, h0 + nh) of the KV head's g
    const int h0 = a.g * chunk / chunks, nh = a.g * (chunk + 1) / chunks - h0;
    dep_wait();                                          // launched dependent: see launch_dep
    dep_release();
    const int len = a.next_pos[b];
    const Int4Span sp = int4_span(len, a.S, a.W, a.ring, a.sinks);
    const int per = a.split / kInt4Step, nsplit = (sp.steps + per - 1) / per;
    if ((int)blockIdx.x >= nsplit) return;
    int s_first = blockIdx.x * per, tiles = min(per, sp.steps - s_first);        // the split's steps: a tile each for this warp

    unsigned char* myS = smem + warp * C::WARPB;
    uint64_t* myBar = bar + warp * C::STAGES;
    const char* Kg = static_cast<const char*>(a.k);
    const char* Vg = static_cast<const char*>(a.v);
    // this warp's tile of a step: its first key, the end of the keys of its part, and the first (rows of others may be anything)
    struct Tile {
        int k0, end, lo;
    };
    auto tile_at = [&](int s) {
        return s < sp.nwin ? Tile{sp.lo_t + s * kInt4Step + warp * kTile, sp.hi, sp.lo}
                           : Tile{(s - sp.nwin) * kInt4Step + warp * kTile, sp.sunk, 0};
    };
    auto next = [&](Tile& t, int s) {                    // to step s, the one behind
        t.k0 += kInt4Step;
        if (s == sp.nwin) t = Tile{warp * kTile, sp.sunk, 0};
    };
    const int32_t* pages = PAGED ? a.table + (size_t)b * (a.S / kPage) : nullptr;
    const size_t head_row0 = ((size_t)b * a.Hkv + kvh) * a.S;
    // paged: lane i holds the pages of both blocks of the warp's tile i of the split, all loaded in one round trip (looked up
    // tile by tile, before each copy, 16 requests of 8192 keys and 64 query heads took 65 us, 60 us so)
    int2 page = make_int2(0, 0);
    auto look_up = [&]() {
        if (!PAGED || lane >= tiles) return;
        const Tile t = tile_at(s_first + lane);
        // (unmapped: only behind a replay's flagged append)
        if (t.k0 < t.end) page.x = max(pages[t.k0 / kPage], 0);
        if (t.k0 + kPage < t.end) page.y = max(pages[t.k0 / kPage + 1], 0);
    };
    // tile i of the split into stage i mod 2: blocks of 16 rows that hold a visible key (whole: the cache's rows are a
    // multiple of 16); called by the whole warp
    auto issue = [&](const Tile& t, int i) {
        const int sg = i & 1;
        int2 at = make_int2(0, 0);
        if (PAGED) at = make_int2(__shfl_sync(0xffffffffu, page.x, i), __shfl_sync(0xffffffffu, page.y, i));
        if (lane == 0 && t.k0 < t.end) {
            const int k0 = t.k0, nb = (min(kTile, t.end - k0) + kPage - 1) / kPage;
            unsigned char* st = myS + sg * C::STAGEB;
            mbar_arrive_expect_tx(&myBar[sg], (uint32_t)(2 * nb * kPage * C::ROW));
            if (!PAGED) {
                const size_t o = (head_row0 + k0) * C::ROW;
                bulk_copy_g2s(st, Kg + o, nb * kPage * C::ROW, &myBar[sg]);
                bulk_copy_g2s(st + C::HALF, Vg + o, nb * kPage * C::ROW, &myBar[sg]);
            } else {
                for (int j = 0; j < nb; ++j) {
                    const size_t o = ((size_t)(j ? at.y : at.x) * a.Hkv + kvh) * kPage * C::ROW;
                    bulk_copy_g2s(st + j * kPage * C::ROW, Kg + o, kPage * C::ROW, &myBar[sg]);
                    bulk_copy_g2s(st + C::HALF + j * kPage * C::ROW, Vg + o, kPage * C::ROW, &myBar[sg]);
                }
            }
        }
    };
    if (lane == 0) {
#pragma unroll
        for (int sg = 0; sg < C::STAGES; ++sg) mbar_init(&myBar[sg], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    static_assert(C::STAGES == 2, "stages are filled by name");
    Tile cur = tile_at(s_first), ahead = cur;            // of the tile in use and of the last one issued
    look_up();
    issue(ahead, 0);
    if (tiles > 1) {
        next(ahead, s_first + 1);
        issue(ahead, 1);
    }

    // the queries, rotated at t = len - 1, times log2(e)/sqrt(d); heads past nh: 0.  16 lanes hold a group.
#pragma unroll
    for (int idx = threadIdx.x; idx < C::HEADS * D / 2; idx += kWarps * 32) {
        const int h = idx / (D / 2), i = idx % (D / 2);
        float y0 = 0.f, y1 = 0.f;
        if (h < nh) {
            const size_t off = ((size_t)b * a.Hq + (size_t)kvh * a.g + h0 + h) * D + 2 * i;
            const float x0 = ld_elem(a.q, off, 1), x1 = ld_elem(a.q, off + 1, 1);
            y0 = x0; y1 = x1;
            if (a.rope) rope_pair(x0, x1, a.rope[(size_t)(len - 1) * (D / 2) + i], y0, y1);
        }
        y0 *= a.scale_log2;
        y1 *= a.scale_log2;
        *reinterpret_cast<float2*>(sQ + h * D + 2 * i) = make_float2(y0, y1);
        float sum = (y0 + y1) * 0x1p-5f, top = fmaxf(fabsf(y0), fabsf(y1));     // (32 dims of any size stay within fp32)
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        }
        if ((lane & 15) == 0) {
            sSum[idx / 16] = sum;
            sTop[idx / 16] = top;
        }
    }
    __syncthreads();

    const int g = lane >> 2, qd = lane & 3;
    // B operand of the scores: column g is (head g / 2, hi | lo) or head g; k-step s of group j takes dims
    // 32 j + 8 qd + {2 s, 2 s + 4} and, with codes 16 times as large, {2 s + 1, 2 s + 5}.  Each column's
    // head times 2^e: its largest value in [2^14, 2^15).
    auto exponent = [&](int h) {
        float m = sTop[h * G];
#pragma unroll
        for (int j = 1; j < G; ++j) m = fmaxf(m, sTop[h * G + j]);
        return min(120, 15 + 126 - (int)(__float_as_uint(m) >> 23));         // -114 for infinities and NaN
    };
    uint32_t qb[G][2][2], ql[HL == 1 ? 1 : G][2][2];       // (up to 4 heads: both parts in qb's columns)
    {
        const int hcol = HL == 1 ? g / 2 : g;
        const float up = power_of_two(exponent(hcol));
#pragma unroll
        for (int j = 0; j < G; ++j) {
            const float* q = sQ + hcol * D + 32 * j + 8 * qd;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float f = k == 0 ? up : up * 0.0625f, x = q[2 * s + k] * f, y = q[2 * s + k + 4] * f;
                    const __half xh = __float2half_rn(x), yh = __float2half_rn(y);
                    const uint32_t rest = pack_half(x - __half2float(xh), y - __half2float(yh));
                    qb[j][s][k] = HL == 1 && (g & 1) ? rest : pack_half(x, y);
                    if constexpr (HL == 2) ql[j][s][k] = rest;
                }
        }
    }
    // the lane's heads: sums of the query over a group in the accumulators' unit, and that unit
    float qsum[HL][G], unit[HL];
    bool vast = false;                                   // a unit past 2^126 (queries from 2^119 on): its rest goes into the scores
#pragma unroll
    for (int n = 0; n < HL; ++n) {
        const int h = HL * qd + n, e = exponent(h);
        unit[n] = power_of_two(min(24 - e, 126));
        vast |= 24 - e > 126;
#pragma unroll
        for (int j = 0; j < G; ++j) qsum[n][j] = ldexpf(sSum[h * G + j], e - 24 + 5);
    }
    vast = __any_sync(0xffffffffu, vast);

    const int tr = tok(g), ta = tok(2 * qd), tb = tok(2 * qd + 1);     // keys of rows g, 2 qd, 2 qd + 1 (and + 8: the next)

    uint32_t parity = 0;                                 // of each stage's barrier (bit)
    for (int split = blockIdx.x;; split += gridDim.x) {
        float base[HL], l_w[HL], norm[HL][G], acc[G][2][4];
        float2 gacc[G];                                      // sums of the minima's terms
#pragma unroll
        for (int n = 0; n < HL; ++n) {
            base[n] = -INFINITY;
            l_w[n] = 0.f;
#pragma unroll
            for (int j = 0; j < G; ++j) norm[n][j] = power_of_two(kNormMost);
        }
#pragma unroll
        for (int j = 0; j < G; ++j) {
            gacc[j] = both(0.f);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][0][e] = acc[j][1][e] = 0.f;
        }
        for (int i = 0; i < tiles; ++i, next(cur, s_first + i)) {
            const int nk = cur.end - cur.k0, kmin = cur.lo - cur.k0, sg = i & 1;     // keys of the tile; those before the window
            auto refill = [&]() {
                if (i + 2 >= tiles) return;
                next(ahead, s_first + i + 2);
                issue(ahead, i + 2);
            };
            if (nk <= 0) {                                   // (of the window's or the sinks' last step)
                refill();
                continue;
            }
            if (!mbar_wait(&myBar[sg], parity >> sg & 1)) {
                // give up: flag it, and let this stage's copy and the other's (if issued) land before the stages are
                // reused for the partial
                if (lane == 0) atomicOr(a.hdr, kErrWait);
                mbar_wait(&myBar[sg], parity >> sg & 1);
                parity ^= 1u << sg;
                if (i + 1 < tiles && ahead.k0 < ahead.end) {
                    mbar_wait(&myBar[sg ^ 1], parity >> (sg ^ 1) & 1);
                    parity ^= 2u >> sg;
                }
                break;
            }
            parity ^= 1u << sg;
            const unsigned char* tK = myS + sg * C::STAGEB;
            const unsigned char* tV = tK + C::HALF;
            const bool whole = nk >= kTile && kmin <= 0;

            // ---- scores of keys tr, tr + 1 of both blocks
            float sc[2][2][HL];
#pragma unroll
            for (int blk = 0; blk < 2; ++blk) {
                const unsigned char* r0 = tK + (16 * blk + tr) * C::ROW;
                uint32_t w0[G], w1[G], p0[G], p1[G];
                if constexpr (G == 4) {
                    const uint4 u0 = *reinterpret_cast<const uint4*>(r0 + 16 * qd), u1 = *reinterpret_cast<const uint4*>(r0 + C::ROW + 16 * qd);
                    const uint4 v0 = *reinterpret_cast<const uint4*>(r0 + D / 2), v1 = *reinterpret_cast<const uint4*>(r0 + C::ROW + D / 2);
                    w0[0] = u0.x; w0[1] = u0.y; w0[2] = u0.z; w0[3] = u0.w; w1[0] = u1.x; w1[1] = u1.y; w1[2] = u1.z; w1[3] = u1.w;
                    p0[0] = v0.x; p0[1] = v0.y; p0[2] = v0.z; p0[3] = v0.w; p1[0] = v1.x; p1[1] = v1.y; p1[2] = v1.z; p1[3] = v1.w;
                } else {
                    const uint2 u0 = *reinterpret_cast<const uint2*>(r0 + 8 * qd), u1 = *reinterpret_cast<const uint2*>(r0 + C::ROW + 8 * qd);
                    const uint2 v0 = *reinterpret_cast<const uint2*>(r0 + D / 2), v1 = *reinterpret_cast<const uint2*>(r0 + C::ROW + D / 2);
                    w0[0] = u0.x; w0[1] = u0.y; w1[0] = u1.x; w1[1] = u1.y;
                    p0[0] = v0.x; p0[1] = v0.y; p1[0] = v1.x; p1[1] = v1.y;
                }
                // sums of the keys' rows: by columns (hi and lo, or two heads), and (one head) of the minima's terms by rows
                float2 x0 = both(0.f), x1 = both(0.f), xm = both(0.f);
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    const Pairs u = pairs_of(w0[j]), v = pairs_of(w1[j]);
                    float c[4];
                    mma_first(c, u.x[0], v.x[0], u.x[1], v.x[1], qb[j][0][0], qb[j][0][1]);
                    mma(c, u.x[2], v.x[2], u.x[3], v.x[3], qb[j][1][0], qb[j][1][1]);
                    if constexpr (HL == 2) {
                        mma(c, u.x[0], v.x[0], u.x[1], v.x[1], ql[j][0][0], ql[j][0][1]);
                        mma(c, u.x[2], v.x[2], u.x[3], v.x[3], ql[j][1][0], ql[j][1][1]);
                    }
                    const float m0 = __uint_as_float(p0[j] & 0xffff0000u), m1 = __uint_as_float(p1[j] & 0xffff0000u);
                    x0 = __ffma2_rn(both(__uint_as_float(p0[j] << 16)), make_float2(c[0], c[1]), x0);
                    x1 = __ffma2_rn(both(__uint_as_float(p1[j] << 16)), make_float2(c[2], c[3]), x1);
                    if constexpr (HL == 1) {
                        xm = __ffma2_rn(make_float2(m0, m1), both(qsum[0][j]), xm);
                    } else {
                        const float2 q = make_float2(qsum[0][j], qsum[HL - 1][j]);
                        x0 = __ffma2_rn(both(m0), q, x0);
                        x1 = __ffma2_rn(both(m1), q, x1);
                    }
                }
                if constexpr (HL == 1) {
                    sc[blk][0][0] = x0.x + x0.y + xm.x;
                    sc[blk][1][0] = x1.x + x1.y + xm.y;
                } else {
                    sc[blk][0][0] = x0.x; sc[blk][0][HL - 1] = x0.y;
                    sc[blk][1][0] = x1.x; sc[blk][1][HL - 1] = x1.y;
                }
            }
            if (vast) {
#pragma unroll
                for (int n = 0; n < HL; ++n) {
                    const float rest = power_of_two(max(24 - exponent(HL * qd + n) - 126, 0));
#pragma unroll
                    for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                        for (int e = 0; e < 2; ++e) sc[blk][e][n] *= rest;
                }
            }
            if (!whole) {
#pragma unroll
                for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int key = 16 * blk + tr + e;
#pragma unroll
                        for (int n = 0; n < HL; ++n) sc[blk][e][n] = key < nk && key >= kmin ? sc[blk][e][n] : -INFINITY;
                    }
            }
            // ---- online softmax of the lane's heads over the tile (base: its reference, in log2; scores kLazyMax
            // above move it)
            bool grow = false;
            float bm[HL];
#pragma unroll
            for (int n = 0; n < HL; ++n) {
                bm[n] = fmaxf(fmax3(sc[0][0][n], sc[0][1][n], sc[1][0][n]), sc[1][1][n]);
                bm[n] = fmaxf(bm[n], __shfl_xor_sync(0xffffffffu, bm[n], 4));
                bm[n] = fmaxf(bm[n], __shfl_xor_sync(0xffffffffu, bm[n], 8));
                bm[n] = fmaxf(bm[n], __shfl_xor_sync(0xffffffffu, bm[n], 16));
                grow |= bm[n] * unit[n] > base[n] + kLazyMax;
            }
            if (__any_sync(0xffffffffu, grow)) {
                // the accumulators' columns are heads 2 qd and 2 qd + 1, or the lane's head and nothing.  A reference is a whole
                // number, so it moves by a power of two, which the products take up in their norm: what they hold stays as it is,
                // and weights to come keep their bits however much larger the values were that no longer weigh
                int up[HL];                                  // 2^up: by how much earlier weights fall
                float f[HL];
#pragma unroll
                for (int n = 0; n < HL; ++n) {
                    const float m = bm[n] * unit[n];
                    up[n] = m > base[n] + kLazyMax ? (int)fminf(ceilf(m) - base[n], 400.f) : 0;
                    if (up[n] > 0) base[n] = ceilf(m);
                    f[n] = up[n] > 126 ? 0.f : power_of_two(-up[n]);
                    l_w[n] *= f[n];
                }
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    gacc[j] = __fmul2_rn(gacc[j], make_float2(f[0], f[HL - 1]));
                    float left[HL];                          // 1, but where the norm reaches its highest
#pragma unroll
                    for (int n = 0; n < HL; ++n) {
                        const int e = (int)(__float_as_uint(norm[n][j]) >> 23) - 127 + up[n], to = min(e, kNormMost);
                        norm[n][j] = power_of_two(to);
                        left[n] = e - to > 126 ? 0.f : power_of_two(to - e);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        acc[j][0][e] *= left[HL == 1 ? 0 : e & 1];
                        acc[j][1][e] *= left[HL == 1 ? 0 : e & 1];
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < HL; ++n) {
#pragma unroll
                for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                    for (int e = 0; e < 2; ++e) sc[blk][e][n] = ex2(fmaf(sc[blk][e][n], unit[n], -base[n]));     // masked keys: 0
                l_w[n] += (sc[0][0][n] + sc[0][1][n]) + (sc[1][0][n] + sc[1][1][n]);
            }
            // ---- P.V, a block at a time
#pragma unroll
            for (int blk = 0; blk < 2; ++blk) {
                // scales and minima of keys tr and tr + 1; a masked key adds nothing, whatever its row holds
                uint32_t p0[G], p1[G];
                {
                    const unsigned char* r = tV + (16 * blk + tr) * C::ROW + D / 2;
                    if constexpr (G == 4) {
                        const uint4 u = *reinterpret_cast<const uint4*>(r), v = *reinterpret_cast<const uint4*>(r + C::ROW);
                        p0[0] = u.x; p0[1] = u.y; p0[2] = u.z; p0[3] = u.w; p1[0] = v.x; p1[1] = v.y; p1[2] = v.z; p1[3] = v.w;
                    } else {
                        const uint2 u = *reinterpret_cast<const uint2*>(r), v = *reinterpret_cast<const uint2*>(r + C::ROW);
                        p0[0] = u.x; p0[1] = u.y; p1[0] = v.x; p1[1] = v.y;
                    }
                }
                if (!whole) {
                    const int key = 16 * blk + tr;
#pragma unroll
                    for (int j = 0; j < G; ++j) {
                        if (!(key < nk && key >= kmin)) p0[j] = 0u;
                        if (!(key + 1 < nk && key + 1 >= kmin)) p1[j] = 0u;
                    }
                }
                // weights times scales: of keys tr and tr + 1 (one head), else of two heads, for each key
                float2 pw[G][HL];
                auto weigh = [&]() {
                    float top = 0.f;
#pragma unroll
                    for (int j = 0; j < G; ++j) {
                        const float s0 = __uint_as_float(p0[j] << 16), s1 = __uint_as_float(p1[j] << 16);
                        if constexpr (HL == 1) {
                            pw[j][0] = __fmul2_rn(__fmul2_rn(make_float2(sc[blk][0][0], sc[blk][1][0]), both(norm[0][j])), make_float2(s0, s1));
                            top = fmax3(top, pw[j][0].x, pw[j][0].y);
                        } else {
                            const float2 nn = make_float2(norm[0][j], norm[HL - 1][j]);
                            pw[j][0] = __fmul2_rn(__fmul2_rn(make_float2(sc[blk][0][0], sc[blk][0][HL - 1]), nn), both(s0));
                            pw[j][HL - 1] = __fmul2_rn(__fmul2_rn(make_float2(sc[blk][1][0], sc[blk][1][HL - 1]), nn), both(s1));
                            top = fmax3(fmax3(top, pw[j][0].x, pw[j][0].y), pw[j][HL - 1].x, pw[j][HL - 1].y);
                        }
                    }
                    return top;
                };
                if (__any_sync(0xffffffffu, weigh() > 32768.f)) {
                    // a group of a head whose largest weight passes 2^15 gets a norm that puts it into [2^9, 2^10)
#pragma unroll
                    for (int j = 0; j < G; ++j) {
                        float f[HL];
#pragma unroll
                        for (int n = 0; n < HL; ++n) {
                            float top = fmaxf(sc[blk][0][n] * __uint_as_float(p0[j] << 16), sc[blk][1][n] * __uint_as_float(p1[j] << 16));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                            const int e = (int)(__float_as_uint(top) >> 23) - 127;
                            const float to = top * norm[n][j] > 32768.f ? power_of_two(max(-118, min(kNormMost, 9 - e))) : norm[n][j];
                            f[n] = to / norm[n][j];
                            norm[n][j] = to;
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            acc[j][0][e] *= f[HL == 1 ? 0 : e & 1];
                            acc[j][1][e] *= f[HL == 1 ? 0 : e & 1];
                        }
                    }
                    weigh();
                }
                const unsigned char* xa = tV + (16 * blk + ta) * C::ROW;
                const unsigned char* xb = tV + (16 * blk + tb) * C::ROW;
                uint32_t wa[G / 2], wb[G / 2], wc[G / 2], wd[G / 2];
                if constexpr (G == 4) {
                    const uint2 ya = *reinterpret_cast<const uint2*>(xa + 8 * g), yb = *reinterpret_cast<const uint2*>(xb + 8 * g);
                    const uint2 yc = *reinterpret_cast<const uint2*>(xa + C::ROW + 8 * g), yd = *reinterpret_cast<const uint2*>(xb + C::ROW + 8 * g);
                    wa[0] = ya.x; wa[1] = ya.y; wb[0] = yb.x; wb[1] = yb.y; wc[0] = yc.x; wc[1] = yc.y; wd[0] = yd.x; wd[1] = yd.y;
                } else {
                    wa[0] = *reinterpret_cast<const uint32_t*>(xa + 4 * g); wb[0] = *reinterpret_cast<const uint32_t*>(xb + 4 * g);
                    wc[0] = *reinterpret_cast<const uint32_t*>(xa + C::ROW + 4 * g); wd[0] = *reinterpret_cast<const uint32_t*>(xb + C::ROW + 4 * g);
                }
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    const float m0 = __uint_as_float(p0[j] & 0xffff0000u), m1 = __uint_as_float(p1[j] & 0xffff0000u);
                    // (one head: the terms of keys tr and of keys tr + 1; else of the two heads)
                    if constexpr (HL == 1) {
                        gacc[j] = __ffma2_rn(make_float2(sc[blk][0][0], sc[blk][1][0]), make_float2(m0, m1), gacc[j]);
                    } else {
                        gacc[j] = __ffma2_rn(make_float2(sc[blk][0][0], sc[blk][0][HL - 1]), both(m0), gacc[j]);
                        gacc[j] = __ffma2_rn(make_float2(sc[blk][1][0], sc[blk][1][HL - 1]), both(m1), gacc[j]);
                    }
                    const int sel = j & 1 ? 0x7632 : 0x5410;
                    const Pairs u = pairs_of(__byte_perm(wa[j / 2], wb[j / 2], sel)), v = pairs_of(__byte_perm(wc[j / 2], wd[j / 2], sel));
                    const float2 p = pw[j][0], r = pw[j][HL - 1];
                    const float2 ph = first_part(p), rh = first_part(r), pl = rest_of(p, ph), rl = rest_of(r, rh);
                    const uint32_t b0 = transposed(HL == 1 ? pack_half(ph.x, pl.x) : pack_half(ph.x, ph.y));
                    const uint32_t b1 = transposed(HL == 1 ? pack_half(ph.y, pl.y) : pack_half(rh.x, rh.y));
                    mma(acc[j][0], u.x[0], u.x[1], v.x[0], v.x[1], b0, b1);
                    mma(acc[j][1], u.x[2], u.x[3], v.x[2], v.x[3], b0, b1);
                    if constexpr (HL == 2) {
                        const uint32_t c0 = transposed(pack_half(pl.x, pl.y)), c1 = transposed(pack_half(rl.x, rl.y));
                        mma(acc[j][0], u.x[0], u.x[1], v.x[0], v.x[1], c0, c1);
                        mma(acc[j][1], u.x[2], u.x[3], v.x[2], v.x[3], c0, c1);
                    }
                }
            }
            // the stage is free once every lane is past its reads
            __syncwarp();
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            refill();
        }

        // ---- this warp's partial into its own stages (every issued tile was waited for): l and the
        // groups' terms summed over the 8 lanes of a head; output = products in their unit + the group's term
        __syncwarp();
        float* part_w = reinterpret_cast<float*>(myS);       // [HEADS][2 + D]
#pragma unroll
        for (int n = 0; n < HL; ++n) {
            const int h = HL * qd + n;
            float l = l_w[n];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            if (g == 0) { part_w[h * (D + 2)] = base[n]; part_w[h * (D + 2) + 1] = l; }
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const float unit_w = 1.f / norm[n][j];   // (codes' units first: 2^24 / norm may pass fp32's range)
                float t = HL == 1 ? gacc[j].x + gacc[j].y : n == 0 ? gacc[j].x : gacc[j].y;
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
                float* o = part_w + h * (D + 2) + 2 + 32 * j + 4 * g;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    // (one head: the second column is its weights' second part)
                    const float x = HL == 1 ? acc[j][k][0] + acc[j][k][1] : acc[j][k][n], y = HL == 1 ? acc[j][k][2] + acc[j][k][3] : acc[j][k][2 + n];
                    o[2 * k] = fmaf(x * 0x1p24f, unit_w, t);
                    o[2 * k + 1] = fmaf(y * 0x1p20f, unit_w, t);
                }
            }
        }
        __syncthreads();
        for (int idx = threadIdx.x; idx < nh * D; idx += blockDim.x) {
            const int h = idx / D, x = idx % D;
            float mx = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, reinterpret_cast<const float*>(smem + w * C::WARPB)[h * (D + 2)]);
            float l = 0.f, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float* pw = reinterpret_cast<const float*>(smem + w * C::WARPB) + h * (D + 2);
                const float f = pw[0] == -INFINITY ? 0.f : exp2f(pw[0] - mx);
                l += pw[1] * f;
                sum += pw[2 + x] * f;
            }
            const size_t row = ((size_t)b * a.Hq + (size_t)kvh * a.g + h0 + h) * a.max_splits + split;
            a.part_acc[row * D + x] = sum;
            if (x == 0) a.part_ml[row] = make_float2(mx, l);
        }
        if (split + (int)gridDim.x >= nsplit) return;
        // a launch of fewer CTAs than splits (lengths that the host does not know): the stages are free once read
        s_first = (split + gridDim.x) * per;
        tiles = min(per, sp.steps - s_first);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
        cur = ahead = tile_at(s_first);
        look_up();
        issue(ahead, 0);
        if (tiles > 1) {
            next(ahead, s_first + 1);
            issue(ahead, 1);
        }
    }
}

template <int D, int HL>
cudaError_t launch_t(const DecodeArgs& a, int splits, int chunks, cudaStream_t st) {
    using C = I4<D, HL>;
    auto kernel = a.table ? int4_decode_kernel<D, HL, true> : int4_decode_kernel<D, HL, false>;
    if (cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), C::SMEM)) return e;
    return launch_dep(kernel, dim3(splits, a.Hkv * chunks, a.B), dim3(kWarps * 32), C::SMEM, st, a, chunks);
}

}  // namespace

static_assert(kInt4StepsMost <= 32, "a split's tiles (their pages) fit in a warp's lanes");
static_assert(kInt4Step == kWarps * kTile && kInt4Heads == 8, "split and head shapes");

cudaError_t launch_int4_append_token(const AppendArgs& a, cudaStream_t st) {
    return launch_dep(a.d == 128 ? int4_token_kernel<128> : int4_token_kernel<64>, dim3(a.B), dim3(kThreads), 0, st, a);
}

cudaError_t launch_int4_append_rows(const AppendArgs& a, const RowCounts& g, cudaStream_t st) {
    const int per = kRowsUnroll * (kThreads / (a.d / 16));
    return launch_dep(a.d == 128 ? int4_rows_kernel<128> : int4_rows_kernel<64>, dim3((a.n + per - 1) / per, a.Hkv, g.nb),
                      dim3(kThreads), 0, st, a, g);
}

// Steps per split, by the host's lengths.  Three CTAs or four keep an SM as busy as it gets, so the SM with the longest
// CTAs counts: as many of one length as fill the SMs evenly, or many more than are resident.  The
// estimate: a step takes an SM kStepUs, a CTA kCtaUs of its own, which resident ones hide from each other.  Over 30
// batches and one to 32 steps it picked the fastest, or one within 3 % or 2 us of it (64 query heads over 4 x 32768 keys: 57 us with 19
// steps, 148 with 1, 66 with 32).
int steps_per_split(const kvc_handle* h, int whole, int chunks, int resident) {
    const Shape& s = h->sh;
    constexpr float kStepUs = 0.5f, kCtaUs = 5.f;
    const float rows = (float)s.Hkv * chunks, sms = (float)h->num_sms;
    const int lowest = s.split / kInt4Step;
    // every request counts, wherever it stands in the batch: in classes of alike numbers of steps, by a class's mean
    constexpr int kClasses = 64;
    const int width = (whole + kClasses - 1) / kClasses;
    int count[kClasses] = {}, steps[kClasses], classes = 0;
    long long sum[kClasses] = {};
    for (int b = 0; b < s.B; ++b) {
        const int n = int4_span(h->np[b], s.S, s.W, s.ring, s.sinks).steps;
        ++count[(n - 1) / width];
        sum[(n - 1) / width] += n;
    }
    for (int i = 0; i < kClasses; ++i) {
        if (count[i] == 0) continue;
        count[classes] = count[i];
        steps[classes++] = (int)((sum[i] + count[i] - 1) / count[i]);
    }
    int best = lowest;
    float least = INFINITY;
    for (int per = lowest; per <= std::max(lowest, std::min(kInt4StepsMost, whole)); ++per) {
        float ctas = 0.f;
        for (int i = 0; i < classes; ++i) ctas += (float)count[i] * (float)((steps[i] + per - 1) / per);
        const int longest = std::min(whole, per);
        const float per_sm = ctas * rows / sms, waves = per_sm / resident;
        const float load = waves <= 1.f ? std::ceil(per_sm) : per_sm + 0.5f;
        const float us = load * longest * kStepUs + kCtaUs * (waves <= 1.f ? 1.f : waves + 0.5f);
        if (us < least) { least = us; best = per; }
    }
    return best;
}

cudaError_t launch_int4_decode(const kvc_handle* h, DecodeArgs a, CombineArgs c, cudaStream_t st) {
    const Shape& s = h->sh;
    const int chunks = int4_chunks(s), heads = (s.g + chunks - 1) / chunks;
    // a captured call serves lengths that nobody knows: as many CTAs as the cache may need
    const bool fixed = capturing(st);
    int whole = 1;                                       // steps of the longest request
    for (int b = 0; b < s.B && !fixed; ++b) whole = std::max(whole, int4_span(h->np[b], s.S, s.W, s.ring, s.sinks).steps);
    const int per = fixed ? std::max(s.split / kInt4Step, 4) : steps_per_split(h, whole, chunks, heads <= 4 || s.d == 64 ? 4 : 3);
    a.split = c.split = per * kInt4Step;
    const int splits = fixed ? (s.max_splits * s.split + a.split - 1) / a.split : (whole + per - 1) / per;
    cudaError_t e;
    if (s.d == 128) e = heads <= 4 ? launch_t<128, 1>(a, splits, chunks, st) : launch_t<128, 2>(a, splits, chunks, st);
    else e = heads <= 4 ? launch_t<64, 1>(a, splits, chunks, st) : launch_t<64, 2>(a, splits, chunks, st);
    return e != cudaSuccess ? e : launch_combine(c, splits, st);
}

}  // namespace kvc
