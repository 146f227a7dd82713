// int4.cu -- the INT4 tier: rows quantised as they are appended, and decode attention over them.
//
// Rows (int4.h): per head and token 5 d / 8 bytes of K and as many of V, 4-bit codes u with a
// bf16 scale s and minimum m per 32 dims g.  With x = m + u s the products split into sums over
// codes, which are small integers, and terms per group (t a key, h a head):
//     score_t   = sum_g s_tg (q_g . u_tg) + m_tg sum(q_g),
//     out_x     = sum_t p_t s_tg u_tx + sum_t p_t m_tg          (x in group g).
// Codes enter the tensor cores as the bf16 numbers 16 + u: a shift, an AND and an OR make two of
// them; the 16 is taken back in the group's term, whose factor is m - 16 s instead of m.
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

// Eight dims of a key (from dim 8 e) rotated at position p, rounded to bf16 as in the bf16 cache.
__device__ __forceinline__ uint4 turned(const AppendArgs& a, const uint4 u, int p, int e) {
    const float4* rp = reinterpret_cast<const float4*>(a.rope + (size_t)p * (a.d / 2) + 4 * e);
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

// One token per request: a CTA per request, a thread per 8 dims of a head.
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
    constexpr int kVec = D / 8, kU = 2;
    const int n = a.Hkv * kVec;
    const uint4* K = static_cast<const uint4*>(a.k) + (size_t)b * n;
    const uint4* V = static_cast<const uint4*>(a.v) + (size_t)b * n;
    for (int base = 0; base < n; base += kU * kThreads) {
        uint4 kx[kU] = {}, vx[kU] = {};
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = base + u * kThreads + threadIdx.x;
            if (i < n) { kx[u] = __ldg(K + i); vx[u] = __ldg(V + i); }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = base + u * kThreads + threadIdx.x, h = i / kVec, e = i % kVec;
            if (base + u * kThreads >= n) break;       // (the whole CTA; a warp's lanes stay together)
            const size_t o = slot_row(a, b, i < n ? h : 0, slot, page) * int4::row_size(D);
            int4::store_row<D>(static_cast<char*>(a.kc) + o, static_cast<char*>(a.vc) + o, e,
                               a.rope ? turned(a, kx[u], p, e) : kx[u], vx[u], i < n);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        a.pos[(size_t)b * a.S + slot] = p;
        a.next_pos[b] = p + 1;
    }
}

// Many rows: grid (groups of rows, KV heads, requests), a thread per 8 dims of a row.
// next_position is advanced by the launch that follows.
template <int D>
__global__ void __launch_bounds__(kThreads) int4_rows_kernel(const AppendArgs a, const __grid_constant__ RowCounts g) {
    dep_wait();                                        // (no early release, as the bf16 appends)
    constexpr int kVec = D / 8;
    const int bi = blockIdx.z, b = g.b0 + bi, h = blockIdx.y, cnt = g.val[bi];
    const int r0 = blockIdx.x * (kThreads / kVec);
    if (r0 >= cnt) return;
    const int r = r0 + threadIdx.x / kVec, e = threadIdx.x % kVec;
    const long long p = (long long)a.next_pos[b] + r;
    bool there = r < cnt && !(a.ring && r < cnt - a.S);         // a ring: not overwritten later in this call
    if (there && !position_ok(a, p)) { flag(a.hdr, kErrPosition); there = false; }
    const int slot = there ? (a.ring ? (int)(p % a.S) : (int)p) : 0;
    const int page = there ? slot_page(a, b, slot) : 0;
    uint4 kx = make_uint4(0, 0, 0, 0), vx = kx;
    if (there) {
        const size_t src = (size_t)b * a.sb + (size_t)h * a.sh + (size_t)r * a.sr + 8 * (size_t)e;
        kx = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.k) + src));
        vx = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.v) + src));
        if (a.rope) kx = turned(a, kx, (int)p, e);
        if (page < 0) { flag(a.hdr, kErrPosition); there = false; }
    }
    const size_t o = slot_row(a, b, h, slot, page < 0 ? 0 : page) * int4::row_size(D);
    int4::store_row<D>(static_cast<char*>(a.kc) + o, static_cast<char*>(a.vc) + o, e, kx, vx, there);
    if (there && h == 0 && e == 0) a.pos[(size_t)b * a.S + slot] = (int)p;
}

// ---- decode ------------------------------------------------------------------------------------
// CTA = 4 warps = a split of the keys of one request and KV head, for up to 8 of its query heads; a warp
// streams tiles of 32 keys through its stages of shared memory by bulk copies (a page, or 16 rows, is
// contiguous).  Both products on the tensor cores (mma m16n8k16, bf16 operands, fp32
// accumulation), operands unpacked in registers from the words that a lane loads:
//  * scores, transposed: S^T[16 keys][cols] = U[16][32 dims of g] . Q^T, the columns (head, hi) and
//    (head, lo): the rotated query times log2(e)/sqrt(d) in two bf16 parts (16 significant
//    bits); the groups' sums are weighed by s_tg and joined by the lane that holds head and keys;
//  * P.V, transposed: O^T[16 dims of g][cols] += U^T . P_g^T, P_g = p s_tg as bf16 hi + lo,
//    brought from score order to operand order by movmatrix (the pair (hi, lo) of a key and head
//    is one register of a score fragment).
// Row r of a fragment of 16 keys stands for key tok(r): rows are 80 bytes apart (d = 128), and with this
// order the lanes' 16-byte loads of K (rows r, r + 1 together) and 8-byte loads of V (rows 0, 2, 4, 6
// together) fall into different banks.
// Lane L: g = L / 4 (fragment row), qd = L % 4 (head, and head 4 + qd).
constexpr int kWarps = 4;
constexpr int kTile = 32;
constexpr float kLazyMax = 8.f;                          // log2-domain headroom of the reference maximum

__device__ __forceinline__ int tok(int r) { return r & 1 ? 8 + ((r + 3) & 7) : r; }      // rows 0..7; row r + 8: tok(r) + 1

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// D (16x8, fp32) += A (16x16, bf16, row) . B (16x8, bf16, col)
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 x 8 matrix of 16-bit elements, transposed across the warp.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// (16 + low nibble, 16 + high-half nibble) of nibble i of both halves of w, as bf16: 16 is 0x4180,
// and between 16 and 32 the last 7 bits count eighths.
template <int I>
__device__ __forceinline__ uint32_t pair_of(uint32_t w) {
    const uint32_t x = I == 0 ? w << 3 : w >> (I == 0 ? 0 : 4 * I - 3);
    return (x & 0x00780078u) | 0x41804180u;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&t);
}

// (hi, lo) with hi = bf16(x), lo = bf16(x - hi), hi in the low half
__device__ __forceinline__ uint32_t split_pair(float x) {
    const float hi = __bfloat162float(__float2bfloat16_rn(x));
    return pack_bf16(hi, x - hi);
}

template <int D, int NT>
struct I4 {
    static constexpr int G = D / int4::kGroup;           // groups of a row
    static constexpr int ROW = int4::row_size(D);
    static constexpr int HALF = kTile * ROW;             // K (or V) rows of a stage
    static constexpr int STAGEB = 2 * HALF;
    static constexpr int STAGES = 2;
    static constexpr int WARPB = STAGES * STAGEB;
    static constexpr int HEADS = 4 * NT;
    static constexpr int PARTF = HEADS * (D + 2);        // a warp's partial (m, l, acc), in its stages at the end
    static_assert(PARTF * 4 <= WARPB, "partial must fit in the warp's stages");
    static constexpr int OFF_Q = kWarps * WARPB;         // query [HEADS][D] fp32
    static constexpr int OFF_BAR = OFF_Q + HEADS * D * 4;
    static constexpr size_t SMEM = OFF_BAR + kWarps * STAGES * 8;
    static_assert(HALF % 16 == 0 && kPage * ROW % 16 == 0, "bulk copies");
};

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 4 : 3) int4_decode_kernel(const DecodeArgs a, const int chunks) {
    using C = I4<D, NT>;
    constexpr int G = C::G;
    extern __shared__ __align__(128) unsigned char smem[];
    float* sQ = reinterpret_cast<float*>(smem + C::OFF_Q);
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.z, kvh = blockIdx.y / chunks, chunk = blockIdx.y % chunks, split = blockIdx.x;
    // the CTA's query heads: [h0, h0 + nh) of the KV head's g
    const int h0 = a.g * chunk / chunks, nh = a.g * (chunk + 1) / chunks - h0;
    dep_wait();                                          // launched dependent: see launch_dep
    dep_release();
    const int len = a.next_pos[b];
    int lo, hi;
    key_range(len, a.S, a.W, a.ring, lo, hi);
    const int lo_t = lo & ~(kPage - 1);                  // tiles start at a page
    if (split >= split_count(lo_t, lo, hi, a.split, a.sinks)) return;
    int k_first;                                         // the CTA's keys
    split_keys(split, lo_t, a.split, a.sinks, lo, hi, k_first);
    const int k_end = min(hi, k_first + a.split);

    unsigned char* myS = smem + warp * C::WARPB;
    uint64_t* myBar = bar + warp * C::STAGES;
    const char* Kg = static_cast<const char*>(a.k);
    const char* Vg = static_cast<const char*>(a.v);
    // tiles of the 4 warps interleaved; tile i of this warp
    auto tile_k0 = [&](int i) { return k_first + (i * kWarps + warp) * kTile; };
    auto tile_nk = [&](int i) { return max(0, min(kTile, k_end - tile_k0(i))); };
    const int32_t* pages = a.table ? a.table + (size_t)b * (a.S / kPage) : nullptr;
    const size_t head_row0 = ((size_t)b * a.Hkv + kvh) * a.S;
    // blocks of 16 rows that hold a visible key (whole: the cache's rows are a multiple of 16)
    auto issue = [&](int i) {
        const int nk = tile_nk(i);
        if (lane == 0 && nk > 0) {
            const int sg = i % C::STAGES, k0 = tile_k0(i), nb = (nk + kPage - 1) / kPage;
            unsigned char* st = myS + sg * C::STAGEB;
            mbar_arrive_expect_tx(&myBar[sg], (uint32_t)(2 * nb * kPage * C::ROW));
            if (!pages) {
                const size_t o = (head_row0 + k0) * C::ROW;
                bulk_copy_g2s(st, Kg + o, nb * kPage * C::ROW, &myBar[sg]);
                bulk_copy_g2s(st + C::HALF, Vg + o, nb * kPage * C::ROW, &myBar[sg]);
            } else {
                for (int j = 0; j < nb; ++j) {
                    const int page = max(pages[k0 / kPage + j], 0);    // (unmapped: only behind a replay's flagged append)
                    const size_t o = ((size_t)page * a.Hkv + kvh) * kPage * C::ROW;
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
#pragma unroll
    for (int i = 0; i < C::STAGES; ++i) issue(i);

    // the queries, rotated at t = len - 1, times log2(e)/sqrt(d); heads past nh: 0
    for (int idx = threadIdx.x; idx < C::HEADS * D / 2; idx += blockDim.x) {
        const int h = idx / (D / 2), i = idx % (D / 2);
        float y0 = 0.f, y1 = 0.f;
        if (h < nh) {
            const size_t off = ((size_t)b * a.Hq + (size_t)kvh * a.g + h0 + h) * D + 2 * i;
            const float x0 = ld_elem(a.q, off, 1), x1 = ld_elem(a.q, off + 1, 1);
            y0 = x0; y1 = x1;
            if (a.rope) rope_pair(x0, x1, a.rope[(size_t)(len - 1) * (D / 2) + i], y0, y1);
        }
        sQ[h * D + 2 * i] = y0 * a.scale_log2;
        sQ[h * D + 2 * i + 1] = y1 * a.scale_log2;
    }
    __syncthreads();

    const int g = lane >> 2, qd = lane & 3;
    // B operand of the scores: column n = 8 nt + g is (head 4 nt + g / 2, hi | lo); k-step s of group j takes
    // dims 32 j + 8 qd + {2 s, 2 s + 4} and {2 s + 1, 2 s + 5}.  And the lane's heads' sums over a group.
    uint32_t qb[NT][G][2][2];
    float qsum[NT][G];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < G; ++j) {
            const float* q = sQ + (4 * nt + g / 2) * D + 32 * j + 8 * qd;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t x = split_pair(q[2 * s + k]), y = split_pair(q[2 * s + k + 4]);
                    qb[nt][j][s][k] = g & 1 ? __byte_perm(x, y, 0x7632) : __byte_perm(x, y, 0x5410);
                }
            float sum = 0.f;
            for (int i = 0; i < 32; ++i) sum += sQ[(4 * nt + qd) * D + 32 * j + ((i + lane) & 31)];
            qsum[nt][j] = sum;
        }

    float m_w[NT], l_w[NT], gacc[NT][G], acc[G][2][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m_w[nt] = -INFINITY; l_w[nt] = 0.f;
#pragma unroll
        for (int j = 0; j < G; ++j) {
            gacc[nt][j] = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][0][nt][e] = acc[j][1][nt][e] = 0.f;
        }
    }
    const int tr = tok(g), ta = tok(2 * qd), tb = tok(2 * qd + 1);     // keys of rows g, 2 qd, 2 qd + 1 (and + 8: the next)

    const int tpw = a.split / (kWarps * kTile);
    for (int i = 0; i < tpw; ++i) {
        const int nk = tile_nk(i);
        if (nk == 0) break;                              // later tiles of this warp are empty too
        const int sg = i % C::STAGES;
        if (!mbar_wait(&myBar[sg], (uint32_t)((i / C::STAGES) & 1))) {
            // give up: flag it, and let this stage's copy and the later stages' (if issued) land
            // before the stages are reused for the partial
            if (lane == 0) atomicOr(a.hdr, kErrWait);
            mbar_wait(&myBar[sg], (uint32_t)((i / C::STAGES) & 1));
            for (int j = i + 1; j < i + C::STAGES && j < tpw; ++j)
                if (tile_nk(j) > 0) mbar_wait(&myBar[j % C::STAGES], (uint32_t)((j / C::STAGES) & 1));
            break;
        }
        const unsigned char* tK = myS + sg * C::STAGEB;
        const unsigned char* tV = tK + C::HALF;
        const int kmin = lo - tile_k0(i);                // keys of the tile before the window
        const bool whole = nk == kTile && kmin <= 0;

        // ---- scores of keys tr, tr + 1 of both blocks
        float sc[2][2][NT];
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
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) sc[blk][0][nt] = sc[blk][1][nt] = 0.f;
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const uint32_t x0 = pair_of<0>(w0[j]), x1 = pair_of<0>(w1[j]), x2 = pair_of<1>(w0[j]), x3 = pair_of<1>(w1[j]);
                const uint32_t y0 = pair_of<2>(w0[j]), y1 = pair_of<2>(w1[j]), y2 = pair_of<3>(w0[j]), y3 = pair_of<3>(w1[j]);
                const float s0 = __uint_as_float(p0[j] << 16), s1 = __uint_as_float(p1[j] << 16);
                const float t0 = fmaf(-16.f, s0, __uint_as_float(p0[j] & 0xffff0000u));
                const float t1 = fmaf(-16.f, s1, __uint_as_float(p1[j] & 0xffff0000u));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
                    mma(c, x0, x1, x2, x3, qb[nt][j][0][0], qb[nt][j][0][1]);
                    mma(c, y0, y1, y2, y3, qb[nt][j][1][0], qb[nt][j][1][1]);
                    sc[blk][0][nt] = fmaf(s0, c[0] + c[1], fmaf(t0, qsum[nt][j], sc[blk][0][nt]));
                    sc[blk][1][nt] = fmaf(s1, c[2] + c[3], fmaf(t1, qsum[nt][j], sc[blk][1][nt]));
                }
            }
        }
        if (!whole) {
#pragma unroll
            for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int key = 16 * blk + tr + e;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) sc[blk][e][nt] = key < nk && key >= kmin ? sc[blk][e][nt] : -INFINITY;
                }
        }
        // ---- online softmax of the lane's heads over the tile
        bool rescale = false;
        float alpha[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float bm = fmaxf(fmaxf(sc[0][0][nt], sc[0][1][nt]), fmaxf(sc[1][0][nt], sc[1][1][nt]));
            bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 4));
            bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 8));
            bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 16));
            const float mn = bm > m_w[nt] + kLazyMax ? bm : m_w[nt];
            alpha[nt] = ex2(m_w[nt] - mn);               // 0 while the maximum was -inf
            rescale |= alpha[nt] != 1.f;
            m_w[nt] = mn;
            float sum = 0.f;
#pragma unroll
            for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sc[blk][e][nt] = ex2(sc[blk][e][nt] - mn);        // masked keys: 0
                    sum += sc[blk][e][nt];
                }
            l_w[nt] = fmaf(l_w[nt], alpha[nt], sum);
        }
        if (__any_sync(0xffffffffu, rescale) && i > 0) {  // at i = 0 the accumulators are 0
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    gacc[nt][j] *= alpha[nt];
#pragma unroll
                    for (int e = 0; e < 4; ++e) { acc[j][0][nt][e] *= alpha[nt]; acc[j][1][nt][e] *= alpha[nt]; }
                }
        }
        // ---- P.V of both blocks
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
            const unsigned char* v0 = tV + 16 * blk * C::ROW;
            uint32_t p0[G], p1[G], wa[G / 2], wb[G / 2], wc[G / 2], wd[G / 2];
            {
                const unsigned char* r0 = v0 + tr * C::ROW + D / 2;
                const unsigned char *xa = v0 + ta * C::ROW, *xb = v0 + tb * C::ROW;
                if constexpr (G == 4) {
                    const uint4 u0 = *reinterpret_cast<const uint4*>(r0), u1 = *reinterpret_cast<const uint4*>(r0 + C::ROW);
                    p0[0] = u0.x; p0[1] = u0.y; p0[2] = u0.z; p0[3] = u0.w; p1[0] = u1.x; p1[1] = u1.y; p1[2] = u1.z; p1[3] = u1.w;
                    const uint2 ya = *reinterpret_cast<const uint2*>(xa + 8 * g), yb = *reinterpret_cast<const uint2*>(xb + 8 * g);
                    const uint2 yc = *reinterpret_cast<const uint2*>(xa + C::ROW + 8 * g), yd = *reinterpret_cast<const uint2*>(xb + C::ROW + 8 * g);
                    wa[0] = ya.x; wa[1] = ya.y; wb[0] = yb.x; wb[1] = yb.y; wc[0] = yc.x; wc[1] = yc.y; wd[0] = yd.x; wd[1] = yd.y;
                } else {
                    const uint2 u0 = *reinterpret_cast<const uint2*>(r0), u1 = *reinterpret_cast<const uint2*>(r0 + C::ROW);
                    p0[0] = u0.x; p0[1] = u0.y; p1[0] = u1.x; p1[1] = u1.y;
                    wa[0] = *reinterpret_cast<const uint32_t*>(xa + 4 * g); wb[0] = *reinterpret_cast<const uint32_t*>(xb + 4 * g);
                    wc[0] = *reinterpret_cast<const uint32_t*>(xa + C::ROW + 4 * g); wd[0] = *reinterpret_cast<const uint32_t*>(xb + C::ROW + 4 * g);
                }
            }
            if (!whole) {
                // a masked key adds nothing, whatever its row holds
                const int k0 = 16 * blk + tr;
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    if (!(k0 < nk && k0 >= kmin)) p0[j] = 0u;
                    if (!(k0 + 1 < nk && k0 + 1 >= kmin)) p1[j] = 0u;
                }
            }
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const float s0 = __uint_as_float(p0[j] << 16), s1 = __uint_as_float(p1[j] << 16);
                const float t0 = fmaf(-16.f, s0, __uint_as_float(p0[j] & 0xffff0000u));
                const float t1 = fmaf(-16.f, s1, __uint_as_float(p1[j] & 0xffff0000u));
                const int sel = j & 1 ? 0x7632 : 0x5410;
                const uint32_t x = __byte_perm(wa[j / 2], wb[j / 2], sel), y = __byte_perm(wc[j / 2], wd[j / 2], sel);
                const uint32_t x0 = pair_of<0>(x), x1 = pair_of<1>(x), x2 = pair_of<2>(x), x3 = pair_of<3>(x);
                const uint32_t y0 = pair_of<0>(y), y1 = pair_of<1>(y), y2 = pair_of<2>(y), y3 = pair_of<3>(y);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float e0 = sc[blk][0][nt], e1 = sc[blk][1][nt];
                    gacc[nt][j] = fmaf(e0, t0, fmaf(e1, t1, gacc[nt][j]));
                    const uint32_t b0 = transposed(split_pair(e0 * s0)), b1 = transposed(split_pair(e1 * s1));
                    mma(acc[j][0][nt], x0, x1, y0, y1, b0, b1);
                    mma(acc[j][1][nt], x2, x3, y2, y3, b0, b1);
                }
            }
        }
        // the stage is free once every lane is past its reads
        __syncwarp();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        if (i + C::STAGES < tpw) issue(i + C::STAGES);
    }

    // ---- this warp's partial into its own stages (every issued tile was waited for): l and the
    // groups' terms summed over the 8 lanes of a head; output = hi + lo columns + the group's term
    __syncwarp();
    float* part_w = reinterpret_cast<float*>(myS);       // [HEADS][2 + D]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int h = 4 * nt + qd;
        float l = l_w[nt];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (g == 0) { part_w[h * (D + 2)] = m_w[nt]; part_w[h * (D + 2) + 1] = l; }
#pragma unroll
        for (int j = 0; j < G; ++j) {
            float t = gacc[nt][j];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            float* o = part_w + h * (D + 2) + 2 + 32 * j + 4 * g;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                o[2 * k] = acc[j][k][nt][0] + acc[j][k][nt][1] + t;
                o[2 * k + 1] = acc[j][k][nt][2] + acc[j][k][nt][3] + t;
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
}

template <int D, int NT>
cudaError_t launch_t(const DecodeArgs& a, int chunks, cudaStream_t st) {
    using C = I4<D, NT>;
    if (cudaError_t e = allow_smem(reinterpret_cast<const void*>(int4_decode_kernel<D, NT>), C::SMEM)) return e;
    return launch_dep(int4_decode_kernel<D, NT>, dim3(a.max_splits, a.Hkv * chunks, a.B), dim3(kWarps * 32), C::SMEM, st, a, chunks);
}

}  // namespace

static_assert(kInt4SplitLeast % (kWarps * kTile) == 0 && kInt4Heads == 8, "split and head shapes");

cudaError_t launch_int4_append_token(const AppendArgs& a, cudaStream_t st) {
    return launch_dep(a.d == 128 ? int4_token_kernel<128> : int4_token_kernel<64>, dim3(a.B), dim3(kThreads), 0, st, a);
}

cudaError_t launch_int4_append_rows(const AppendArgs& a, const RowCounts& g, cudaStream_t st) {
    const int per = kThreads / (a.d / 8);
    return launch_dep(a.d == 128 ? int4_rows_kernel<128> : int4_rows_kernel<64>, dim3((a.n + per - 1) / per, a.Hkv, g.nb),
                      dim3(kThreads), 0, st, a, g);
}

cudaError_t launch_int4_splits(const DecodeArgs& a, cudaStream_t st) {
    const int chunks = (a.g + kInt4Heads - 1) / kInt4Heads, heads = (a.g + chunks - 1) / chunks;
    if (a.d == 128) return heads <= 4 ? launch_t<128, 1>(a, chunks, st) : launch_t<128, 2>(a, chunks, st);
    return heads <= 4 ? launch_t<64, 1>(a, chunks, st) : launch_t<64, 2>(a, chunks, st);
}

}  // namespace kvc
