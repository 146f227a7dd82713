// prompt_tc.cu -- attention of packed prompts on tcgen05 (bf16 caches, head_dim 64 or 128).
//
// o = softmax(q K^T / sqrt(d)) V per query row over the keys that it sees, one pass over the
// keys with a running maximum and sum per row (fp32).  A dense contraction: bound by the
// tensor cores, whose pace the softmax between the two products has to keep.
//  * CTA = 256 query rows (token, head of the group) of one (request, KV head), as two
//    slots of 128 rows; both read the same tiles of 128 keys, walked upwards from the first
//    key that any of its rows sees.
//  * Warps 0-3 and 4-7: softmax of slot 0 and 1, thread = row = tensor-memory lane.  Warp 8
//    issues the tensor copies, warps 9 and 10 the matrix instructions of a slot each, warp 11
//    looks over the value rows of boundary tiles.
//  * Tensor memory: S of the slots in columns [0, 128) and [128, 256), fp32; the weights P
//    replace the first 64 columns of S as bf16 pairs (the A operand of P.V); O in [256, 384)
//    and [384, 512).  Q sits in shared memory.
//  * All operands are bf16: q and the keys as the cache's type holds them, the weights
//    rounded once (relative error 2^-8, at most 2^8 in size).  fp16 weights (2^-11) would
//    need the values in fp16 too: a conversion pass over every tile and a narrower range.
//  * Per slot: S(j) -> softmax(j) -> P.V(j) -> S(j+1), which overwrites the columns that P.V(j)
//    reads and so waits for it; the slots alternate on the tensor cores.
//  * A row's reference maximum moves only when a tile exceeds it by more than 2^8 (log2
//    domain); the softmax thread then rescales its O row itself (no P.V of its slot in flight).
//  * Masked scores are replaced, not added to, so a masked key may hold anything.  A masked
//    weight of 0 times a value that is not finite would still spoil a row, so boundary tiles
//    (where some row sees only some of the keys) have such values replaced by 0 in shared
//    memory before P.V, and the epilogue adds them back to the rows that see them.
//  * Key tiles start on multiples of 16.  A contiguous cache is read in 128-row boxes; paged
//    caches and rings in 16-row boxes, a lane each, from the page, the ring slot or the
//    staging rows.  Groups past the last key repeat the last one.
//  * CTAs run longest first (host-sorted items), the KV heads of an item adjacent.
// Every mbarrier wait is bounded; on expiry the kernel flags the device error word, skips
// the remaining work, waits (bounded) for its copies and matrix instructions in flight and
// frees its tensor memory.
#include <algorithm>
#include <vector>

#include "prompt.h"
#include "tcgen05.h"

namespace kvc {
namespace {

using namespace tc;

constexpr int kBM = 128;            // rows per slot
constexpr int kSlots = 2;
constexpr int kRows = kSlots * kBM;
constexpr int kThreads = 12 * 32;
constexpr int kWarpCopy = 8, kWarpMma = 9, kWarpLook = 11;   // (a matrix warp per slot: 9 and 10)
constexpr float kLazyMax = 8.f;     // log2-domain headroom of a row's reference maximum
constexpr int kRegSoftmax = 216, kRegOther = 72, kRegLaunch = 168;
static_assert(8 * kRegSoftmax + 4 * kRegOther == 12 * kRegLaunch, "register split sums to the launch's registers");
constexpr int kItems = 512;         // (request, tile) items per launch
constexpr uint32_t kTmemCols = 512;

struct Items {
    int n;
    int4 e[kItems];                 // (index in the group, tile of 256 rows, packed row of the request, its rows)
};

template <int D>
struct Plan {
    static constexpr int kBN = D == 128 ? 80 : 128;        // keys per tile: S, P and O of both slots fill tensor memory
    static constexpr uint32_t kColS = 0, kColP = 2 * kBN;  // S of slot i at kColS + i kBN (fp32) ...
    static constexpr uint32_t kPStep = D == 128 ? 48 : 64; // ... P at kColP + i kPStep (bf16 pairs)
    static constexpr uint32_t kColO = kTmemCols - 2 * D;   // ... O at kColO + i D (fp32)
    static_assert(kColP + kPStep + kBN / 2 <= kColO, "tensor memory columns");
    static constexpr int kHalves = D / 64;                 // 64-dim halves: 128-byte rows, 128-byte swizzle
    static constexpr int kHalf = kBN * 128;                // of a K or V tile
    static constexpr int kTile = kHalves * kHalf;
    static constexpr int kQHalf = kBM * 128;
    static constexpr int kQTile = kHalves * kQHalf;
    static constexpr int kStages = 4;                      // of K and of V each
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + kSlots * kQTile;
    static constexpr int kV = kK + kStages * kTile;
    static constexpr int kBar = kV + kStages * kTile;
    enum {
        kKFull = 0,                          // [stage] K copied
        kVFull = kKFull + kStages,           // [stage] V copied
        kVClean = kVFull + kStages,          // [stage] V looked over
        kSFull = kVClean + kStages,          // [slot][stage] S complete
        kODone = kSFull + kSlots * kStages,  // [slot][stage] P.V complete
        kSFree = kODone + kSlots * kStages,  // [slot] S read (4 warps)
        kPFull = kSFree + kSlots,            // [slot] P written (4 warps)
        kQReady = kPFull + kSlots,           // Q of both slots in shared memory (8 warps)
        kDone = kQReady + 1,                 // [slot] every product issued so far complete
        kBars = kDone + kSlots
    };
    static constexpr int kMisc = kBar + 8 * kBars;         // tensor memory base, abort flag, spoilt flag
    static constexpr int kBytes = kMisc + 16 + 1024;       // + alignment of the dynamic base
    static_assert(kBytes <= (int)kMaxSmemPerBlock, "shared memory per block");
    static_assert(kTile % (16 * 8 * 32) == 0, "looked over in rounds of eight chunks a lane");
};

// Bits 15 and 31 tell whether the low and the high bf16 of a pair are not finite.
__device__ __forceinline__ uint32_t odd_bits(uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; }

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ CUtensorMap tmWK, const __grid_constant__ CUtensorMap tmWV,
                       const __grid_constant__ AttnArgs a, const int b0, const __grid_constant__ Items items) {
    using L = Plan<D>;
    constexpr int kBN = L::kBN;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char* sQ = smem + L::kQ;
    unsigned char* sK = smem + L::kK;
    unsigned char* sV = smem + L::kV;
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
    volatile int* spoilt = reinterpret_cast<volatile int*>(smem + L::kMisc + 8);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int kvh = blockIdx.x % a.Hkv;
    const int4 item = items.e[blockIdx.x / a.Hkv];
    const int b = b0 + item.x, n = item.w;
    const int cut = a.next_pos[b];
    const long long all = (long long)n * a.g, row0 = (long long)item.y * kRows;
    const int nrow = (int)min((long long)kRows, all - row0);
    const int t0 = (int)(row0 / a.g);                       // first token of the CTA
    const int j0 = (int)(row0 - (long long)t0 * a.g);       // ... and its head in the group
    auto token = [&](int r) { return t0 + (j0 + r) / a.g; };
    // keys: the CTA's and each slot's first and last, in tiles from k0
    const int p_first = cut + t0, p_last = cut + token(nrow - 1);
    auto first_key = [&](int p) { return a.W > 0 ? max(0, p - a.W + 1) : 0; };
    const int k0 = first_key(p_first) & ~15;
    const int ntiles = (p_last - k0) / kBN + 1;
    // slot i multiplies tiles [0, slot_hi(i)); the last slot with rows goes through all of them
    auto slot_hi = [&](int i) { return kBM * i < nrow ? (cut + token(min(nrow, kBM * (i + 1)) - 1) - k0) / kBN + 1 : 0; };
    // tiles [w0, w1): every row of the CTA sees every key; the others are boundary tiles
    const int w0 = (first_key(p_last) - k0 + kBN - 1) / kBN, w1 = max(w0, (p_first - k0 + 1) / kBN);
    // slot i's barrier for tile j (`which`: kSFull or kODone) and its phase: one per stage, so
    // that the copies, kStages tiles ahead of the products at most, can wait on them too
    auto stage_bar = [&](int which, int i, int j) { return &bar[which + i * L::kStages + j % L::kStages]; };
    auto phase = [](int j) { return (uint32_t)((j / L::kStages) & 1); };

    if (tid == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(&bar[L::kKFull + s], 1);
            mbar_init(&bar[L::kVFull + s], 1);
            mbar_init(&bar[L::kVClean + s], 1);
        }
        for (int i = 0; i < kSlots; ++i) {
            for (int s = 0; s < L::kStages; ++s) {
                mbar_init(&bar[L::kSFull + i * L::kStages + s], 1);
                mbar_init(&bar[L::kODone + i * L::kStages + s], 1);
            }
            mbar_init(&bar[L::kSFree + i], 4);
            mbar_init(&bar[L::kPFull + i], 4);
            mbar_init(&bar[L::kDone + i], 1);
        }
        mbar_init(&bar[L::kQReady], 8);
        *abort_flag = 0;
        *spoilt = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kWarpMma) tmem_alloc(tmem_slot, kTmemCols);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    // every warpgroup changes its register share together
    if (warp < 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegSoftmax));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegOther));

    if (warp < 8) {
        // ================= softmax: warp w serves slot w / 4, rows 32 (w % 4) .. + 31
        const int slot = warp >> 2, lg = warp & 3;
        const int row = 32 * lg + lane, r = kBM * slot + row;
        const uint32_t lane_off = (uint32_t)(32 * lg) << 16;
        const uint32_t tS = tmem + L::kColS + kBN * slot + lane_off;
        const uint32_t tP = tmem + L::kColP + L::kPStep * slot + lane_off;
        const uint32_t tO = tmem + L::kColO + D * slot + lane_off;
        const bool valid = r < nrow;
        const int p = cut + token(r);
        const int key_lo = first_key(p);
        const int hi = slot_hi(slot);
        // all rows of the slot see all keys of a tile from sl to sh
        const int sl = first_key(cut + token(min(nrow, kBM * (slot + 1)) - 1)), sh = cut + token(kBM * slot);
        bool fail = false;
        // the warp's 32 queries, rotated at their positions in fp32 and rounded to bf16, into the
        // slot's Q tile (16-byte chunk c of row r at c ^ (r mod 8)): D / 8 lanes a row, all
        // rounds of loads in flight
        constexpr int kPer = D / 8, kTogether = 32 / kPer, kRounds = 32 / kTogether;
        const int dt = kTogether / a.g, dj = kTogether % a.g;
        auto next_row = [&](int& tt, int& jj) {
            tt += dt;
            jj += dj;
            if (jj >= a.g) { jj -= a.g; ++tt; }
        };
        uint4 qv[kRounds];
        int q_tok[kRounds / 8], q_head[kRounds / 8];                           // token and head of every eighth round's row
        {
            const int r0 = kBM * slot + 32 * lg + lane / kPer;
            int tt = t0 + (j0 + r0) / a.g, jj = (j0 + r0) % a.g;
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (size_t)item.z * a.q_stride +
                                     (size_t)kvh * a.g * D + 8 * (lane % kPer);
#pragma unroll
            for (int e = 0; e < kRounds; ++e) {
                if (e % 8 == 0) { q_tok[e / 8] = tt; q_head[e / 8] = jj; }
                qv[e] = make_uint4(0u, 0u, 0u, 0u);
                if (r0 + e * kTogether < nrow) qv[e] = __ldg(reinterpret_cast<const uint4*>(q + tt * a.q_stride + jj * D));
                next_row(tt, jj);
            }
        }
        {
            unsigned char* qt = sQ + slot * L::kQTile;
            const int c = lane % kPer, r0 = 32 * lg + lane / kPer;             // chunk, first row
#pragma unroll
            for (int e0 = 0; e0 < kRounds; e0 += 8) {
                float4 ra[8], rb[8];
                int tt = q_tok[e0 / 8], jj = q_head[e0 / 8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ra[e] = rb[e] = make_float4(1.f, 0.f, 1.f, 0.f);
                    if (a.rope && kBM * slot + r0 + (e0 + e) * kTogether < nrow && cut + tt < a.P) {
                        const float4* rp = reinterpret_cast<const float4*>(a.rope + (size_t)(cut + tt) * (D / 2) + 4 * c);
                        ra[e] = __ldg(rp);
                        rb[e] = __ldg(rp + 1);
                    }
                    next_row(tt, jj);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int rr = r0 + (e0 + e) * kTogether;
                    uint32_t w[4] = {qv[e0 + e].x, qv[e0 + e].y, qv[e0 + e].z, qv[e0 + e].w};
                    if (a.rope) {
                        const float2 cs[4] = {make_float2(ra[e].x, ra[e].y), make_float2(ra[e].z, ra[e].w),
                                              make_float2(rb[e].x, rb[e].y), make_float2(rb[e].z, rb[e].w)};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float y0, y1;
                            rope_pair(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u), cs[k], y0, y1);
                            const __nv_bfloat162 o2 = __floats2bfloat162_rn(y0, y1);
                            w[k] = *reinterpret_cast<const uint32_t*>(&o2);
                        }
                    }
                    *reinterpret_cast<uint4*>(qt + (c >> 3) * L::kQHalf + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[L::kQReady]);
        }
        // o[0, 32) += the values that are not finite and were left out of boundary tiles, of the
        // keys that a row sees
        auto add_spoilt = [&](float* o, int x0, int lo, int hi_key) {
            for (int key = lo; key <= hi_key; ++key) {
                if ((key - k0) / kBN >= w0 && (key - k0) / kBN < w1) { key = k0 + w1 * kBN - 1; continue; }
                const bool staged = a.ring && key >= (cut & ~15);
                const size_t at = staged ? stage_row(b, kvh, key, cut, a.Hkv, a.ws_rows)
                                         : kv_row(a.table, b, kvh, a.ring ? key % a.S : key, a.Hkv, a.S);
                const uint4* v = reinterpret_cast<const uint4*>((staged ? a.wv : static_cast<const __nv_bfloat16*>(a.vc)) + at * D + x0);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint4 u = v[e];
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float v0 = __uint_as_float(w[k] << 16), v1 = __uint_as_float(w[k] & 0xffff0000u);
                        if (!isfinite(v0)) o[8 * e + 2 * k] += v0;
                        if (!isfinite(v1)) o[8 * e + 2 * k + 1] += v1;
                    }
                }
            }
        };
        float m_ref = -INFINITY, l = 0.f;                       // m_ref: of the scores, before scaling
        const float sc = a.scale_log2, lazy = kLazyMax / sc;
        for (int j = 0; j < hi; ++j) {
            const bool w = wait(stage_bar(L::kSFull, slot, j), phase(j), abort_flag);
            if (!__all_sync(0xffffffffu, w)) { fail = true; break; }
            fence_after();
            float s[kBN];
#pragma unroll
            for (int c = 0; c + 32 <= kBN; c += 32) tmem_ld32(tS + c, s + c);
            if constexpr (kBN % 32 == 16) tmem_ld16(tS + kBN - 16, s + kBN - 16);
            tmem_wait_ld();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[L::kSFree + slot]);          // S(j + 1) may overwrite it
            const int kb = k0 + kBN * j;
            if (!(kb >= sl && kb + kBN - 1 <= sh) || nrow < kBM * (slot + 1)) {
                const int c0 = key_lo - kb, width = valid ? p - key_lo : -1;      // visible: c0 .. c0 + width
#pragma unroll
                for (int c = 0; c < kBN; ++c) s[c] = width >= 0 && (uint32_t)(c - c0) <= (uint32_t)width ? s[c] : -INFINITY;
            }
            // row maximum: eight independent chains of three-input maxima, then a tree
            float m8[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) m8[e] = fmaxf(s[e], s[8 + e]);
#pragma unroll
            for (int c = 16; c < kBN; c += 16)
#pragma unroll
                for (int e = 0; e < 8; ++e) m8[e] = fmax3(m8[e], s[c + e], s[c + 8 + e]);
            const float mx = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
            bool grow = false;
            float alpha = 1.f;
            if (mx > m_ref + lazy) {
                grow = m_ref != -INFINITY;
                alpha = grow ? ex2((m_ref - mx) * sc) : 1.f;
                m_ref = mx;
            }
            const bool any = __any_sync(0xffffffffu, grow);
            // P.V(j - 1) reads P and adds to O: usually done long before the weights are
            auto done = [&]() -> bool {
                return j == 0 || __all_sync(0xffffffffu, wait(stage_bar(L::kODone, slot, j - 1), phase(j - 1), abort_flag));
            };
            if (any) {
                if (!done()) { fail = true; break; }
                fence_after();
                const float f = grow ? alpha : 1.f;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    tmem_ld32(tO + c, o);
                    tmem_wait_ld();
                    uint32_t u[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(o[e] * f);
                    tmem_st32(tO + c, u);
                }
                tmem_wait_st();
            }
            const float base = m_ref == -INFINITY ? 0.f : m_ref * sc;      // nothing visible so far: weights 0
            uint32_t pk[kBN / 2];
            float2 rs[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const float2 nb2 = make_float2(-base, -base), sc2 = make_float2(sc, sc);
#pragma unroll
            for (int e = 0; e < kBN / 2; ++e) {
                const float2 x = __ffma2_rn(make_float2(s[2 * e], s[2 * e + 1]), sc2, nb2);
                const float p0 = ex2(x.x), p1 = ex2(x.y);                   // masked keys: 0
                rs[e & 3] = __fadd2_rn(rs[e & 3], make_float2(p0, p1));
                const __nv_bfloat162 t2 = __floats2bfloat162_rn(p0, p1);
                pk[e] = *reinterpret_cast<const uint32_t*>(&t2);
            }
            const float2 r4 = __fadd2_rn(__fadd2_rn(rs[0], rs[1]), __fadd2_rn(rs[2], rs[3]));
            l = l * alpha + (r4.x + r4.y);
            if (!any && !done()) { fail = true; break; }
            fence_after();
#pragma unroll
            for (int c = 0; c + 32 <= kBN / 2; c += 32) tmem_st32(tP + c, pk + c);
            if constexpr (kBN / 2 % 32 == 8) tmem_st8(tP + kBN / 2 - 8, pk + kBN / 2 - 8);
            tmem_wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[L::kPFull + slot]);
        }
        if (!fail && hi > 0) {
            const bool w = wait(stage_bar(L::kODone, slot, hi - 1), phase(hi - 1), abort_flag);
            fail = !__all_sync(0xffffffffu, w);
        }
        if (fail) {
            if (lane == 0) atomicOr(a.hdr, kErrWait);
            *abort_flag = 1;
        } else if (hi > 0 && !*abort_flag) {
            fence_after();
            const float inv = 1.f / l;
            const bool fix = *spoilt != 0;
            // through the warp's own rows of the Q tile (its scores are all done), so that a store
            // covers whole 128-byte lines: 32 dims at a time as fp32, 64 as bf16
            unsigned char* stage = sQ + slot * L::kQTile + 32 * lg * 128;
            const int c = lane & 7, r1 = kBM * slot + 32 * lg + (lane >> 3);   // store: chunk, first row (then every fourth)
            const int tok = t0 + (j0 + r1) / a.g, head = (j0 + r1) % a.g, dt4 = 4 / a.g, dj4 = 4 % a.g;
            const size_t orow = ((size_t)item.z * a.Hq + kvh * a.g) * D;
#pragma unroll 1
            for (int x0 = 0; x0 < D; x0 += 32) {
                float o[32];
                tmem_ld32(tO + x0, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= inv;
                if (fix && valid) add_spoilt(o, x0, key_lo, p);
                if (a.out_bf16) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t u[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const __nv_bfloat162 t2 = __floats2bfloat162_rn(o[8 * e + 2 * k], o[8 * e + 2 * k + 1]);
                            u[k] = *reinterpret_cast<const uint32_t*>(&t2);
                        }
                        *reinterpret_cast<uint4*>(stage + lane * 128 + (((x0 / 32 % 2 * 4 + e) ^ (lane & 7)) << 4)) =
                            make_uint4(u[0], u[1], u[2], u[3]);
                    }
                    if (x0 % 64 == 0) continue;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<float4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                            make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
                __syncwarp();
                int tt = tok, jj = head;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int rr = (lane >> 3) + 4 * e;
                    if (r1 + 4 * e < nrow) {
                        const uint4 u = *reinterpret_cast<const uint4*>(stage + rr * 128 + ((c ^ (rr & 7)) << 4));
                        const size_t at = orow + ((size_t)tt * a.Hq + jj) * D;
                        if (a.out_bf16) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at + x0 / 64 * 64 + 8 * c) = u;
                        else *reinterpret_cast<uint4*>(static_cast<float*>(a.out) + at + x0 + 4 * c) = u;
                    }
                    tt += dt4;
                    jj += dj4;
                    if (jj >= a.g) { jj -= a.g; ++tt; }
                }
                __syncwarp();
            }
        }
    } else if (warp == kWarpCopy) {
        // ================= tensor copies of K and V tiles
        // one box of kBN rows a half on a contiguous cache; else a box per 16 rows, both halves,
        // whose number a lane looks up and the elected lane issues
        const bool boxes = a.table || a.ring, lead = elect_one();
        const int head_row0 = (b * a.Hkv + kvh) * a.S, cal = cut & ~15;
        const int ws_row0 = (b * a.Hkv + kvh) * a.ws_rows;
        // first row of the lane's group in tile j; a staged row as -1 - row
        auto row_of = [&](int j) {
            const int kb = k0 + kBN * j;
            if (!boxes) return head_row0 + kb;
            if (lane >= kBN / 16 || j >= ntiles) return 0;
            const int pos = min(kb + 16 * lane, p_last & ~15);
            if (a.ring && pos >= cal) return -1 - (ws_row0 + (pos - cal));
            const int slot = a.ring ? pos % a.S : pos;
            return a.table ? (max(a.table[(size_t)b * (a.S / kPage) + slot / kPage], 0) * a.Hkv + kvh) * kPage : head_row0 + slot;
        };
        auto load_tile = [&](const CUtensorMap* tm, const CUtensorMap* tmw, unsigned char* dst, uint64_t* full, int row) {
            if (lead) mbar_arrive_expect_tx(full, L::kTile);
            if (!boxes) {
                if (lead) {
#pragma unroll
                    for (int half = 0; half < L::kHalves; ++half) tma_load_2d(dst + half * L::kHalf, tm, 64 * half, row, full);
                }
            } else {
#pragma unroll
                for (int gi = 0; gi < kBN / 16; ++gi) {
                    const int r = __shfl_sync(0xffffffffu, row, gi);
                    if (lead) tma_load_4d(dst + gi * L::kHalves * 2048, r < 0 ? tmw : tm, 0, 0, 0, (r < 0 ? -1 - r : r) / 8, full);
                }
            }
            __syncwarp();
        };
        // a stage is free when the slots that multiply its tile are done with it
        const int hi0 = slot_hi(0), hi1 = slot_hi(1);
        auto free_again = [&](int which, int j) -> bool {
            return __all_sync(0xffffffffu, (j >= hi0 || wait(stage_bar(which, 0, j), phase(j), abort_flag)) &&
                                               (j >= hi1 || wait(stage_bar(which, 1, j), phase(j), abort_flag)));
        };
        auto looked = [&](int j) -> bool {
            return __all_sync(0xffffffffu, wait(&bar[L::kVClean + j % L::kStages], phase(j), abort_flag));
        };
        bool ok = true;
        int k_issued = 0, v_issued = 0;
        int row = row_of(0);
        for (int j = 0; j < ntiles; ++j) {
            const int st = j % L::kStages;
            const int ahead = row_of(j + 1);                    // its page number is read while this tile waits
            if (j >= L::kStages && !(ok = free_again(L::kSFull, j - L::kStages))) break;
            load_tile(&tmK, &tmWK, sK + st * L::kTile, &bar[L::kKFull + st], row);
            k_issued = j + 1;
            if (j >= L::kStages && !(ok = free_again(L::kODone, j - L::kStages) && looked(j - L::kStages))) break;
            load_tile(&tmV, &tmWV, sV + st * L::kTile, &bar[L::kVFull + st], row);
            v_issued = j + 1;
            row = ahead;
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0) atomicOr(a.hdr, kErrWait);
            // the last copy issued into each stage lands before the CTA can exit
            for (int j = max(0, k_issued - L::kStages); j < k_issued; ++j)
                drain(&bar[L::kKFull + j % L::kStages], (uint32_t)((j / L::kStages) & 1));
            for (int j = max(0, v_issued - L::kStages); j < v_issued; ++j)
                drain(&bar[L::kVFull + j % L::kStages], (uint32_t)((j / L::kStages) & 1));
        }
        __syncwarp();
    } else if (warp < kWarpLook) {
        // ================= matrix instructions of one slot, one lane issuing.  Per tile: S(j + 1)
        // as soon as the softmax has read S(j), then P.V(j) when the weights are there
        constexpr uint32_t idesc_qk = instr_desc_bf16(kBM, kBN, false), idesc_pv = instr_desc_bf16(kBM, D, true);
        const int slot = warp - kWarpMma, hi = slot_hi(slot);
        // K and V tiles: [half][row] from a contiguous cache, [8 rows][half] from 16-row boxes
        const bool boxes = a.table || a.ring;
        const uint32_t half_step = boxes ? 1024 : L::kHalf, group_step = boxes ? L::kHalves * 1024 : 1024;
        const uint64_t qdesc = smem_desc(smem_u32(sQ) + slot * L::kQTile, 16, 1024), kdesc0 = smem_desc(smem_u32(sK), 16, group_step);
        const uint64_t vdesc0 = smem_desc(smem_u32(sV), half_step, group_step);
        const uint64_t khalf = half_step >> 4, vstep = (2 * group_step) >> 4;
        const uint32_t tS = tmem + L::kColS + kBN * slot, tP = tmem + L::kColP + L::kPStep * slot, tO = tmem + L::kColO + D * slot;
        const bool lead = elect_one();
        auto wait_ok = [&](uint64_t* b, uint32_t parity) -> bool { return __all_sync(0xffffffffu, spin(b, parity, abort_flag)); };
        // S = Q K_j^T, 16 dims per instruction
        auto issue_s = [&](int j) {
            const uint64_t kd = kdesc0 + (uint64_t)((j % L::kStages) * (L::kTile >> 4));
            if (lead) {
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
                    mma_ss(tS, qdesc + (uint64_t)(((s >> 2) * L::kQHalf + (s & 3) * 32) >> 4),
                           kd + (s >> 2) * khalf + (uint64_t)(((s & 3) * 32) >> 4), idesc_qk, s > 0);
                mma_commit(stage_bar(L::kSFull, slot, j));
            }
            __syncwarp();
        };
        // O += P V_j: keys 16 s .. + 15 of P sit in its columns 8 s .. + 7
        auto issue_pv = [&](int j) {
            const uint64_t vd = vdesc0 + (uint64_t)((j % L::kStages) * (L::kTile >> 4));
            if (lead) {
#pragma unroll
                for (int s = 0; s < kBN / 16; ++s)
                    mma_ts(tO, tP + 8 * s, vd + s * vstep, idesc_pv, (j > 0 || s > 0));
                mma_commit(stage_bar(L::kODone, slot, j));
            }
            __syncwarp();
        };
        bool ok = hi == 0 || (wait_ok(&bar[L::kQReady], 0) && wait_ok(&bar[L::kKFull], 0));
        if (ok && hi > 0) {
            fence_after();
            issue_s(0);
        }
        for (int j = 0; j < hi && ok; ++j) {
            const int st = j % L::kStages, next = (j + 1) % L::kStages;
            if (j + 1 < hi) {
                ok = wait_ok(&bar[L::kKFull + next], phase(j + 1)) && wait_ok(&bar[L::kSFree + slot], (uint32_t)(j & 1));
                if (!ok) break;
                fence_after();
                issue_s(j + 1);
            }
            ok = wait_ok(&bar[L::kVFull + st], phase(j));
            if (j < w0 || j >= w1) ok = ok && wait_ok(&bar[L::kVClean + st], phase(j));
            ok = ok && wait_ok(&bar[L::kPFull + slot], (uint32_t)(j & 1));
            if (!ok) break;
            fence_after();
            issue_pv(j);
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0) atomicOr(a.hdr, kErrWait);
        }
        // no product may still target the columns when they are freed
        if (lead) mma_commit(&bar[L::kDone + slot]);
        __syncwarp();
        drain(&bar[L::kDone + slot], 0);
        __syncwarp();
    } else {
        // ================= value rows of boundary tiles: what is not finite becomes 0
        bool ok = true;
        for (int j = 0; j < ntiles; ++j) {
            const int st = j % L::kStages;
            ok = __all_sync(0xffffffffu, wait(&bar[L::kVFull + st], phase(j), abort_flag));
            if (!ok) break;
            if (j >= w0 && j < w1) {
                if (lane == 0) mbar_arrive(&bar[L::kVClean + st]);
                continue;
            }
            unsigned char* tile = sV + st * L::kTile;
            bool any = false;
#pragma unroll 1
            for (int q0 = lane; q0 < L::kTile / 16; q0 += 8 * 32) {
                uint4 u[8];
                uint32_t bad = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = *reinterpret_cast<const uint4*>(tile + 16 * (q0 + 32 * e));
#pragma unroll
                for (int e = 0; e < 8; ++e) bad |= odd_bits(u[e].x) | odd_bits(u[e].y) | odd_bits(u[e].z) | odd_bits(u[e].w);
                if (bad & 0x80008000u) {
                    any = true;
                    for (int q = q0; q < q0 + 8 * 32; q += 32) {
                        uint32_t* w = reinterpret_cast<uint32_t*>(tile + 16 * q);
                        for (int k = 0; k < 4; ++k) {
                            if ((w[k] & 0x7f80u) == 0x7f80u) w[k] &= 0xffff0000u;
                            if ((w[k] & 0x7f800000u) == 0x7f800000u) w[k] &= 0x0000ffffu;
                        }
                    }
                }
            }
            if (any) *spoilt = 1;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[L::kVClean + st]);
        }
        if (!ok) {
            if (lane == 0) atomicOr(a.hdr, kErrWait);
            *abort_flag = 1;
        }
    }
    fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        __syncwarp();
        fence_after();
        tmem_free(tmem, kTmemCols);
    }
}

// Tensor map over `rows` rows of d bf16 values, 128-byte swizzle.  Boxes of `bn` rows by 64 dims;
// or, with `boxes`, of 16 rows and all dims in the order [8 rows][half]: dims (64 of a half, row
// of 8, half, 8-row group), so that one copy brings a page's rows of a head.
bool row_map(CUtensorMap* tm, const void* base, long long rows, int d, bool boxes, int bn) {
    using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                     const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                     CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const EncodeTiled enc = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeTiled>(p) : nullptr;
    }();
    if (!enc) return false;
    const cuuint64_t row = (cuuint64_t)d * 2;
    const cuuint64_t dims2[2] = {(cuuint64_t)d, (cuuint64_t)rows}, strides2[1] = {row};
    const cuuint64_t dims4[4] = {64, 8, (cuuint64_t)(d / 64), (cuuint64_t)(rows / 8)}, strides4[3] = {row, 128, 8 * row};
    const cuuint32_t box2[2] = {64, (cuuint32_t)bn}, box4[4] = {64, 8, (cuuint32_t)(d / 64), 2}, es[4] = {1, 1, 1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, boxes ? 4 : 2, const_cast<void*>(base), boxes ? dims4 : dims2,
               boxes ? strides4 : strides2, boxes ? box4 : box2, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(const CUtensorMap* tm, const AttnArgs& a, int b0, const Items& items, cudaStream_t st) {
    auto kernel = prompt_attn_kernel<D>;
    if (cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), Plan<D>::kBytes)) return e;
    kernel<<<dim3((unsigned)items.n * a.Hkv), kThreads, Plan<D>::kBytes, st>>>(tm[0], tm[1], tm[2], tm[3], a, b0, items);
    return cudaGetLastError();
}

}  // namespace

bool prompt_tc_supported(const Shape& s) {
    const long long rows = s.pages ? (long long)s.pages * s.Hkv * kPage : (long long)s.B * s.Hkv * s.S;
    const long long staged = s.ring ? (long long)s.B * s.Hkv * chunk_ws_rows(s) : 0;
    return s.bf16 && !s.int8 && (s.d == 64 || s.d == 128) && rows < (1ll << 31) - 128 && staged < (1ll << 31);
}

cudaError_t launch_prompt_tc(const kvc_handle* h, const AttnArgs& a, const Packed& g, cudaStream_t st) {
    const Shape& s = h->sh;
    const int bn = s.d == 128 ? Plan<128>::kBN : Plan<64>::kBN;
    CUtensorMap tm[4];
    const bool boxes = s.pages || s.ring;
    const long long rows = s.pages ? (long long)s.pages * s.Hkv * kPage : (long long)s.B * s.Hkv * s.S;
    if (!row_map(&tm[0], a.kc, rows, s.d, boxes, bn) || !row_map(&tm[1], a.vc, rows, s.d, boxes, bn)) return cudaErrorInvalidValue;
    tm[2] = tm[0]; tm[3] = tm[1];
    if (s.ring) {
        const long long staged = (long long)s.B * s.Hkv * a.ws_rows;
        if (!row_map(&tm[2], a.wk, staged, s.d, boxes, bn) || !row_map(&tm[3], a.wv, staged, s.d, boxes, bn))
            return cudaErrorInvalidValue;
    }
    // longest first: an item's work is its number of key tiles.  The host's lengths order the
    // CTAs only; the kernel reads the cut on the device.
    std::vector<std::pair<int, int4>> work;
    for (int i = 0; i < g.nb; ++i) {
        const int n = g.off[i + 1] - g.off[i], cut = h->np[g.b0 + i];
        const long long all = (long long)n * s.g;
        for (long long t = 0; t * kRows < all; ++t) {
            const int first = cut + (int)(t * kRows / s.g), last = cut + (int)((std::min(all, (t + 1) * kRows) - 1) / s.g);
            const int k0 = (s.W > 0 ? std::max(0, first - s.W + 1) : 0) & ~15;
            work.push_back({-((last - k0) / bn + 1), make_int4(i, (int)t, (int)(g.row0 + g.off[i]), n)});
        }
    }
    std::stable_sort(work.begin(), work.end(), [](const auto& x, const auto& y) { return x.first < y.first; });
    static thread_local Items items;      // 8 KB of kernel parameters: not on the stack
    for (size_t i0 = 0; i0 < work.size(); i0 += kItems) {
        items.n = (int)std::min<size_t>(kItems, work.size() - i0);
        for (int i = 0; i < items.n; ++i) items.e[i] = work[i0 + i].second;
        const cudaError_t e = s.d == 128 ? launch<128>(tm, a, g.b0, items, st) : launch<64>(tm, a, g.b0, items, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace kvc
