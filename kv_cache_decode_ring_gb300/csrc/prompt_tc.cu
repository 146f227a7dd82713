// prompt_tc.cu -- attention of packed prompts on tcgen05 (bf16 caches, head_dim 64 or 128).
//
// o = softmax(q K^T / sqrt(d)) V per query row over the keys that it sees, one pass over the
// keys with a running maximum and sum per row (fp32).  A dense contraction: bound by the
// tensor cores, whose pace the softmax between the two products has to keep.
//  * Unit of work: two slots of 128 query rows (token, head of the group; as many whole tokens
//    as fit) of one (request, KV head); both read the same tiles of keys, walked upwards from the first key
//    that any of the rows sees.  A CTA per SM takes units in turn, longest first (host-sorted;
//    every other round in reverse, which evens the CTAs' sums), the KV heads of a tile of rows
//    adjacent.  Where units are few and long, their keys are split over several CTAs
//    and a second kernel joins the parts.
//  * Warps 0-3 and 4-7: softmax of slot 0 and 1, thread = row = tensor-memory lane.  Warp 8
//    issues the tensor copies of keys and values, warp 9 those of the next unit's queries, warps
//    10 and 11 look over the value rows of boundary tiles, warps 12-15 issue the matrix
//    instructions: each slot's two products from a warp of their own (with one warp
//    for both, its waits and issues, one after the other, took longer than the products).
//  * Tensor memory: S of both slots (fp32), their weights P (bf16 pairs, the A operand of P.V) and
//    O (fp32) in columns of their own: with d = 128 that leaves tiles of 80 keys, with d = 64
//    of 128.  So S(j + 1) runs while the softmax works on S(j).  (Tiles of 128 keys with P over S,
//    where S(j + 1) waits for P.V(j), took 2.4 ms a call for 16384 tokens of 32 heads: 1.63 now.)
//  * All operands are bf16: q and the keys as the cache's type holds them, the weights
//    rounded once (relative error 2^-8, at most 2^8 in size).  fp16 weights (2^-11) would
//    need the values in fp16 too: a conversion pass over every tile and a narrower range.
//  * With RoPE the queries come rotated, in d_out's rows (prompt_rows_kernel): a unit copies its
//    queries from the rows that it writes at its end.  Rotating them here, by two warps beside
//    the softmax, took longer than a short unit's products (ragged prompts 0.30 ms a call, 0.178
//    now).
//  * A row's reference maximum moves only when a tile exceeds it by more than 2^8 (log2
//    domain); the softmax thread then rescales its O row itself (no P.V of its slot in flight).
//  * Masked scores are replaced, not added to, so a masked key may hold anything.  A masked
//    weight of 0 times a value that is not finite would still spoil a row, so boundary tiles
//    (where some row sees only some of the keys) have such values replaced by 0 in shared
//    memory before P.V, and the epilogue adds them back to the rows that see them.
//  * Key tiles start on multiples of 16.  A contiguous cache is read in boxes of a tile's rows;
//    paged caches and rings in boxes of 16 rows from the page, the ring slot or the
//    staging rows.  Groups past the last key repeat the last one.
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
constexpr int kThreads = 16 * 32;
constexpr int kWarpCopy = 8, kWarpLoad = 9, kWarpLook = 10, kWarpMma = 12;
constexpr int kLookWarps = 2;
constexpr int kMmaWarps = 4;       // matrix warps: S and P.V of slot 0, then of slot 1
constexpr float kLazyMax = 8.f;     // log2-domain headroom of a row's reference maximum
constexpr int kRegLaunch = 128;
constexpr int kItems = 512;         // items (a tile of rows of a request, a part of its keys) per launch
constexpr uint32_t kTmemCols = 512;
constexpr int kAhead = 8;           // units whose descriptions are kept in shared memory
constexpr int kSplitTiles = 4;      // ... of no fewer tiles than this

struct Items {
    int n, parts;
    int boxed;                      // 32 rows of a slot are whole tokens: tmO has boxes for them
    int4 e[kItems];                 // (index in the group | part << 16, first token, packed row of the request, its tokens)
};

template <int D>
struct Plan {
    static constexpr int kBN = D == 128 ? 80 : 128;        // keys per tile
    static constexpr uint32_t kColS = 0, kColP = 2 * kBN;  // S of slot i at kColS + i kBN (fp32) ...
    static constexpr uint32_t kPStep = D == 128 ? 48 : 64; // ... P at kColP + i kPStep (bf16 pairs)
    static constexpr uint32_t kColO = kTmemCols - 2 * D;   // ... O at kColO + i D (fp32)
    static_assert(kColP + kPStep + kBN / 2 <= kColO, "tensor memory columns");
    static constexpr int kHalves = D / 64;                 // 64-dim halves: 128-byte rows, 128-byte swizzle
    static constexpr int kHalf = kBN * 128;                // of a K or V tile
    static constexpr int kTile = kHalves * kHalf;
    static constexpr int kQHalf = kBM * 128;
    static constexpr int kQTile = kHalves * kQHalf;
    static constexpr int kStages = D == 128 ? 3 : 4;       // of K and of V each
    static constexpr int kQBufs = D == 128 ? 3 : 4;        // Q tiles: slot s of unit i is tile q = 2 i + s, in buffer q mod kQBufs
    static constexpr int kRegSoftmax = 192, kRegIssue = 64, kRegMma = 64;
    static_assert(8 * kRegSoftmax + 4 * kRegIssue + 4 * kRegMma == 16 * kRegLaunch, "register split sums to the launch's registers");
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + kQBufs * kQTile;
    static constexpr int kV = kK + kStages * kTile;
    static constexpr int kBar = kV + kStages * kTile;
    enum {
        kKFull = 0,                          // [stage] K copied
        kVFull = kKFull + kStages,           // [stage] V copied
        kVClean = kVFull + kStages,          // [stage] V looked over (2 warps)
        kSFull = kVClean + kStages,          // [slot][stage] S complete
        kODone = kSFull + kSlots * kStages,  // [slot][stage] P.V complete
        kSFree = kODone + kSlots * kStages,  // [slot] S read (4 warps)
        kPFull = kSFree + kSlots,            // [slot] P written (4 warps)
        kQFree = kPFull + kSlots,            // [Q buffer] the slot's rows of the unit are written (4 warps)
        kQFull = kQFree + kQBufs,            // [slot][unit mod 2] Q copied and the unit's description written
        kDone = kQFull + 2 * kSlots,         // [matrix warp] every product issued so far complete
        kBars = kDone + kMmaWarps
    };
    static constexpr int kUnits = kBar + 8 * kBars;        // descriptions: kAhead of 16 words
    static constexpr int kMisc = kUnits + kAhead * 64;     // tensor memory base, units with spoilt values
    static constexpr int kPlace = kMisc + 8 + 4 * kAhead;  // place of a slot's row in the output, in rows of heads
    static constexpr int kBytes = kPlace + 4 * kBM + 1024; // + alignment of the dynamic base
    static_assert(kBytes <= (int)kMaxSmemPerBlock, "shared memory per block");
    static_assert(kTile % (16 * 8 * 32) == 0, "looked over in rounds of eight chunks a lane");
};

// Bits 15 and 31 tell whether the low and the high bf16 of a pair are not finite.
__device__ __forceinline__ uint32_t odd_bits(uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; }

// One unit of work.
struct Unit {
    int b, kvh, part;
    int row;                        // packed row of the request's first row
    int t0, ntok;                   // first token, tokens
    int cut, p_last;                // position of the request's first row; of the unit's last
    int k0, nt;                     // first key, tiles
    int w0, w1;                     // tiles [w0, w1): every row sees every key; the others are boundary tiles
    int ns, s0, sunk;               // tiles [0, ns) hold the sinks [s0, sunk) that lie before k0 (no key of a later tile)
};

__device__ __forceinline__ int first_key(const AttnArgs& a, int p) { return a.W > 0 ? max(0, p - a.W + 1) : 0; }

// First key of a unit's tile.
template <int D, bool SINKS>
__device__ __forceinline__ int tile_key(const Unit& w, int j) {
    return (SINKS && j < w.ns ? w.s0 : w.k0) + Plan<D>::kBN * j;
}

// SINKS: the first tiles are those of the first positions, up to the window's first tile.  They are
// boundary tiles, and w.k0 counts as if the window's tiles started in their place.
template <int D, bool SINKS>
__device__ __noinline__ Unit unit_of(const AttnArgs& a, const Items& items, int b0, int u) {
    constexpr int kBN = Plan<D>::kBN;
    Unit w;
    const int4 e = items.e[u / a.Hkv];
    w.kvh = u % a.Hkv;
    w.b = b0 + (e.x & 0xffff);
    w.part = e.x >> 16;
    w.row = e.z;
    w.cut = __ldg(a.next_pos + w.b);
    w.t0 = e.y;
    w.ntok = min(kSlots * (kBM / a.g), e.w - e.y);
    const int p_first = w.cut + w.t0;
    w.p_last = p_first + w.ntok - 1;
    w.k0 = first_key(a, p_first) & ~15;
    w.nt = (w.p_last - w.k0) / kBN + 1;
    int first = 0, nsunk = 0;
    if constexpr (SINKS) {
        w.sunk = min(a.sinks, w.k0);
        nsunk = (w.sunk + kBN - 1) / kBN;
        w.nt += nsunk;
    }
    if (items.parts > 1) {
        first = w.nt * w.part / items.parts;
        w.nt = w.nt * (w.part + 1) / items.parts - first;
    }
    w.ns = max(0, nsunk - first);
    w.s0 = kBN * first;
    first -= nsunk;
    w.w0 = max(w.ns, (first_key(a, w.p_last) - w.k0 + kBN - 1) / kBN - first);
    w.w1 = max(w.w0, (p_first - w.k0 + 1) / kBN - first);
    w.k0 += kBN * first;
    return w;
}

template <int D, bool SINKS>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ CUtensorMap tmWK, const __grid_constant__ CUtensorMap tmWV,
                       const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmO,
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
    static_assert(sizeof(Unit) <= 64, "a unit's description");
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
    volatile int* spoilt = reinterpret_cast<volatile int*>(smem + L::kMisc + 8);   // [unit mod kAhead]: 1 + the unit

    int* place = reinterpret_cast<int*>(smem + L::kPlace);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nunits = items.n * a.Hkv, G = gridDim.x, T = kBM / a.g;      // T: tokens a slot
    // The CTA's unit of round r (there may be none in the last).  Every role walks the same
    // units and counts them (i) and their tiles (k) alike: the counts number the barriers' phases.
    auto mine = [&](int r) { return r * G + ((r & 1) ? G - 1 - (int)blockIdx.x : (int)blockIdx.x); };
    auto unit_in = [&](int i) -> Unit& { return *reinterpret_cast<Unit*>(smem + L::kUnits + (i % kAhead) * 64); };
    // A barrier's parity tells neighbouring phases apart only.  So whoever waits on a barrier
    // waits for its every phase in turn, and none completes twice before each waiter saw it:
    // Q tiles are loaded in order, the load of (slot, unit i + 2) comes after that of
    // (1, i + 1), which waits for (0, i) to be done, as (0, i + 2) does for (1, i).
    auto q_full = [&](int slot, int i) { return &bar[L::kQFull + 2 * slot + (i & 1)]; };
    auto q_buf = [](int slot, int i) { return (2 * i + slot) % L::kQBufs; };
    // slot i's barrier for tile k (`which`: kSFull or kODone) and its phase: one per stage, so
    // that the copies, kStages tiles ahead of the products at most, can wait on them too
    auto stage_bar = [&](int which, int i, int k) { return &bar[which + i * L::kStages + k % L::kStages]; };
    auto phase = [](int k) { return (uint32_t)((k / L::kStages) & 1); };
    auto all_ok = [](bool x) -> bool { return __all_sync(0xffffffffu, x); };

    if (tid == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(&bar[L::kKFull + s], 1);
            mbar_init(&bar[L::kVFull + s], 1);
            mbar_init(&bar[L::kVClean + s], kLookWarps);
        }
        for (int i = 0; i < kSlots; ++i) {
            for (int s = 0; s < L::kStages; ++s) {
                mbar_init(&bar[L::kSFull + i * L::kStages + s], 1);
                mbar_init(&bar[L::kODone + i * L::kStages + s], 1);
            }
            mbar_init(&bar[L::kSFree + i], 4);
            mbar_init(&bar[L::kPFull + i], 4);
        }
        for (int i = 0; i < L::kQBufs; ++i) {
            mbar_init(&bar[L::kQFree + i], 4);
        }
        for (int i = 0; i < 2 * kSlots; ++i) mbar_init(&bar[L::kQFull + i], 1);
        for (int i = 0; i < kMmaWarps; ++i) mbar_init(&bar[L::kDone + i], 1);
        for (int i = 0; i < kAhead; ++i) spoilt[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid < kBM) place[tid] = tid / a.g * a.Hq + tid % a.g;
    if (warp == kWarpMma) tmem_alloc(tmem_slot, kTmemCols);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    dep_wait();                                        // launched dependent (see launch_dep): global memory from here on
    // every warpgroup changes its register share together
    if (warp < 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kRegSoftmax));
    else if (warp < kWarpMma) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kRegIssue));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kRegMma));

    bool ok = true;
    if (warp < 8) {
        // ================= softmax: warp w serves slot w / 4, rows 32 (w % 4) .. + 31
        const int slot = warp >> 2, lg = warp & 3;
        const uint32_t lane_off = (uint32_t)(32 * lg) << 16;
        const uint32_t tS = tmem + L::kColS + kBN * slot + lane_off;
        const uint32_t tP = tmem + L::kColP + L::kPStep * slot + lane_off;
        const uint32_t tO = tmem + L::kColO + D * slot + lane_off;
        const int r = 32 * lg + lane, mine_tok = slot * T + r / a.g;               // the row's token in the unit
        const float sc = a.scale_log2, lazy = kLazyMax / sc;
        int k = 0;                                              // tiles so far
        for (int rd = 0, i = 0; rd * G < nunits && ok; ++rd) {
            if (mine(rd) >= nunits) continue;
            if (!(ok = all_ok(wait(q_full(slot, i), (uint32_t)((i >> 1) & 1))))) break;
            const Unit& w = unit_in(i);
            const int nt = w.nt, ntok = w.ntok, k0 = w.k0, w0 = w.w0, w1 = w.w1;
            const bool valid = r < T * a.g && mine_tok < ntok, some = slot * T < ntok;     // this row's, the slot's
            const int p0 = w.cut + w.t0, p = p0 + mine_tok, key_lo = first_key(a, p);
            // all rows of the slot see all keys from sl to sh
            const int sh = p0 + slot * T, sl = first_key(a, p0 + min(ntok, (slot + 1) * T) - 1);
            const bool full = T * a.g == kBM && ntok >= (slot + 1) * T;
            float m_ref = -INFINITY, l = 0.f;                   // m_ref: of the scores, before scaling
            for (int j = 0; j < nt; ++j, ++k) {
                if (!(ok = all_ok(wait(stage_bar(L::kSFull, slot, k), phase(k))))) break;
                fence_after();
                // P.V of the tile before reads P and adds to O: usually done long before the weights are
                auto done = [&]() -> bool {
                    return j == 0 || all_ok(wait(stage_bar(L::kODone, slot, k - 1), phase(k - 1)));
                };
                if (!some) {                                    // no rows: the products run on, nothing is read
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar[L::kSFree + slot]);
                    if (!(ok = done())) break;
                    if (lane == 0) mbar_arrive(&bar[L::kPFull + slot]);
                    continue;
                }
                float s[kBN];
#pragma unroll
                for (int c = 0; c + 32 <= kBN; c += 32) tmem_ld32(tS + c, s + c);
                if constexpr (kBN % 32 == 16) tmem_ld16(tS + kBN - 16, s + kBN - 16);
                tmem_wait_ld();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[L::kSFree + slot]);          // the next S may overwrite it
                const int kb = SINKS ? tile_key<D, SINKS>(w, j) : k0 + kBN * j;
                if (!(kb >= sl && sh - kb >= kBN - 1) || !full) {
                    // (a word of visible keys per 16, which the compiler spreads over predicates: two
                    // comparisons a key took 3 to 6 % longer on short prompts; skipping groups that
                    // all or none of the warp's rows see costs the other tiles registers)
                    const bool sunk = SINKS && j < w.ns;
                    const int c0 = valid && !sunk ? key_lo - kb : kBN, c1 = valid ? p - kb : -1;       // visible: c0 .. c1
                    const int cs = SINKS && valid ? (sunk ? w.sunk : min(a.sinks, p + 1)) - kb : 0;    // ... and 0 .. cs - 1
#pragma unroll
                    for (int q = 0; q < kBN; q += 16) {
                        const int x0 = min(max(c0 - q, 0), 16), x1 = min(max(c1 - q + 1, 0), 16);
                        uint32_t seen = (0xffffffffu << x0) & ~(0xffffffffu << x1);
                        if constexpr (SINKS) seen |= ~(0xffffffffu << min(max(cs - q, 0), 16));
#pragma unroll
                        for (int c = 0; c < 16; ++c) s[q + c] = seen >> c & 1 ? s[q + c] : -INFINITY;
                    }
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
                if (any) {
                    if (!(ok = done())) break;
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
                if (!any && !(ok = done())) break;
                fence_after();
#pragma unroll
                for (int c = 0; c + 32 <= kBN / 2; c += 32) tmem_st32(tP + c, pk + c);
#pragma unroll
                for (int c = kBN / 64 * 32; c < kBN / 2; c += 8) tmem_st8(tP + c, pk + c);
                tmem_wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[L::kPFull + slot]);
            }
            const bool parts = items.parts > 1;                 // unnormalised sums with their maximum, to be joined
            const float inv = parts ? 1.f : 1.f / l;
            const bool bf16 = a.out_bf16 && !parts;
            // through the warp's own rows of the unit's Q tile (its scores are all done): where the
            // warp's rows are whole tokens, all there and bf16, a tensor copy takes them out; else
            // 128 bytes of each row at a time (32 dims as fp32, 64 as bf16), lines stored whole
            unsigned char* tile = sQ + q_buf(slot, i) * L::kQTile + 32 * lg * 128;
            const int c = lane & 7, nv = min(T, ntok - slot * T) * a.g;        // the slot's rows
            const size_t orow = (size_t)(w.row + w.t0 + slot * T) * a.Hq + w.kvh * a.g;
            const long long row_bytes = parts ? (long long)items.parts * D * 4 : D * (bf16 ? 2 : 4);
            char* dst = (parts ? reinterpret_cast<char*>(a.part_acc + (size_t)w.part * D) : static_cast<char*>(a.out)) +
                        orow * row_bytes + 16 * c;
            if (ok && nt > 0) ok = all_ok(wait(stage_bar(L::kODone, slot, k - 1), phase(k - 1)));
            if (!ok) break;
            if (some) {
                fence_after();
                const bool spoilt_unit = nt > 0 && spoilt[i % kAhead] == i + 1;
                const bool boxed = items.boxed && !spoilt_unit && bf16 && 32 * lg + 32 <= nv;
                if (parts && valid)
                    a.part_ml[(orow + place[r]) * items.parts + w.part] =
                        make_float2(m_ref == -INFINITY ? -INFINITY : m_ref * sc, l);
                auto lines_out = [&](const unsigned char* stage) {       // 128 bytes of each of the warp's rows
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int rr = (lane >> 3) + 4 * e;
                        const uint4 u = *reinterpret_cast<const uint4*>(stage + rr * 128 + ((c ^ (rr & 7)) << 4));
                        if (32 * lg + rr < nv) *reinterpret_cast<uint4*>(dst + (long long)place[32 * lg + rr] * row_bytes) = u;
                    }
                    dst += 128;
                    __syncwarp();
                };
#pragma unroll 1
                for (int x0 = 0; x0 < D; x0 += 64) {
                    float o[64];
                    if (nt > 0) {
                        tmem_ld32(tO + x0, o);
                        tmem_ld32(tO + x0 + 32, o + 32);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int e = 0; e < 64; ++e) o[e] = 0.f;
                    }
                    if (bf16) {
                        unsigned char* stage = boxed ? tile + x0 / 64 * L::kQHalf : tile;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            uint32_t u[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const __nv_bfloat162 t2 = __floats2bfloat162_rn(o[8 * e + 2 * q] * inv, o[8 * e + 2 * q + 1] * inv);
                                u[q] = *reinterpret_cast<const uint32_t*>(&t2);
                            }
                            *reinterpret_cast<uint4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
                        }
                        if (!boxed) lines_out(stage);
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                *reinterpret_cast<float4*>(tile + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                                    make_float4(o[32 * h + 4 * e] * inv, o[32 * h + 4 * e + 1] * inv, o[32 * h + 4 * e + 2] * inv,
                                                o[32 * h + 4 * e + 3] * inv);
                            lines_out(tile);
                        }
                    }
                }
                fence_before();                                 // O is read before the next unit's products write it
                if (boxed) {
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
#pragma unroll
                        for (int half = 0; half < L::kHalves; ++half)
                            tma_store_3d(&tmO, tile + half * L::kQHalf, 64 * half, w.kvh * a.g,
                                         w.row + w.t0 + slot * T + 32 * lg / a.g);
                        tma_store_read();
                    }
                    __syncwarp();
                }
                if (spoilt_unit && valid) {
                    // values that are not finite, left out of boundary tiles: those that the row sees are
                    // added to what it wrote (positions past the capacity have no rows to read)
                    const int c_last = min((a.ring ? p : min(p, a.S - 1)) - k0, nt * kBN - 1);
                    char* at = static_cast<char*>(parts ? static_cast<void*>(a.part_acc + (size_t)w.part * D) : a.out) + (orow + place[r]) * row_bytes;
#pragma unroll 1
                    for (int c = SINKS ? 0 : max(key_lo - k0, 0); c <= (SINKS ? nt * kBN - 1 : c_last); ++c) {
                        const int j = c / kBN, key = SINKS ? tile_key<D, SINKS>(w, j) + c % kBN : k0 + c;
                        if (j >= w0 && j < w1) { c = w1 * kBN - 1; continue; }
                        if (SINKS && !(j < w.ns ? key < w.sunk : key <= min(p, a.S - 1) && (key >= key_lo || key < a.sinks))) continue;
                        const bool staged = a.ring && key >= (w.cut & ~15);
                        const __nv_bfloat16* v = staged ? a.wv + stage_row(w.b, w.kvh, key, w.cut, a.Hkv, a.ws_rows) * D
                                                        : static_cast<const __nv_bfloat16*>(a.vc) +
                                                              kv_row(a.table, w.b, w.kvh, a.ring ? key % a.S : key, a.Hkv, a.S) * D;
#pragma unroll 1
                        for (int x = 0; x < D; ++x) {
                            const float add = __bfloat162float(v[x]);
                            if (isfinite(add)) continue;
                            if (bf16) {
                                __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(at) + x;
                                *o = __float2bfloat16_rn(__bfloat162float(*o) + add);
                            } else {
                                reinterpret_cast<float*>(at)[x] += add;
                            }
                        }
                    }
                }
            }
            fence_async_smem();                                 // the tile's rows held output: the next copy comes after
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[L::kQFree + q_buf(slot, i)]);
            ++i;
        }
    } else if (warp == kWarpCopy) {
        // ================= tensor copies of K and V tiles: one box of kBN rows a half on a
        // contiguous cache; else a box per 16 rows, both halves, whose number a lane looks up
        const bool boxes = a.table || a.ring, lead = elect_one();
        auto load_tile = [&](const CUtensorMap* tm, const CUtensorMap* tmw, unsigned char* dst, uint64_t* full, int row) {
            if (lead) mbar_arrive_expect_tx(full, L::kTile);
            if (!boxes) {
                if (lead) {
#pragma unroll
                    for (int half = 0; half < L::kHalves; ++half) tma_load_2d(dst + half * L::kHalf, tm, 64 * half, row, full);
                }
            } else {
                // (every box's row at hand before the first is issued, one tensor map unless the cache
                // is a ring: with a shuffle before each, two maps to choose from, a tile's boxes took
                // longer than its products, ragged prompts 0.192 ms a call against 0.177)
                int r[kBN / 16];
#pragma unroll
                for (int gi = 0; gi < kBN / 16; ++gi) r[gi] = __shfl_sync(0xffffffffu, row, gi);
                if (lead) {
                    if (a.ring) {
#pragma unroll
                        for (int gi = 0; gi < kBN / 16; ++gi)
                            tma_load_4d(dst + gi * L::kHalves * 2048, r[gi] < 0 ? tmw : tm, 0, 0, 0, (r[gi] < 0 ? -1 - r[gi] : r[gi]) / 8, full);
                    } else {
#pragma unroll
                        for (int gi = 0; gi < kBN / 16; ++gi) tma_load_4d(dst + gi * L::kHalves * 2048, tm, 0, 0, 0, r[gi] / 8, full);
                    }
                }
            }
            __syncwarp();
        };
        // a stage is free when both slots are done with its tile
        auto free_again = [&](int which, int k) -> bool {
            return all_ok(wait(stage_bar(which, 0, k), phase(k)) && wait(stage_bar(which, 1, k), phase(k)));
        };
        auto looked = [&](int k) -> bool { return all_ok(wait(&bar[L::kVClean + k % L::kStages], phase(k))); };
        int k = 0, k_issued = 0, v_issued = 0;
        for (int rd = 0; rd * G < nunits && ok; ++rd) {
            if (mine(rd) >= nunits) continue;
            const Unit w = unit_of<D, SINKS>(a, items, b0, mine(rd));
            const int head_row0 = (w.b * a.Hkv + w.kvh) * a.S, cal = w.cut & ~15;
            const int ws_row0 = (w.b * a.Hkv + w.kvh) * a.ws_rows;
            // where the lane's group of tile j lies: its page (read a tile ahead), or its first row
            auto group_of = [&](int j) { return min(tile_key<D, SINKS>(w, j) + 16 * lane, w.p_last & ~15); };
            auto page_of = [&](int j) {
                return a.table && lane < kBN / 16 && j < w.nt
                           ? __ldg(a.table + (size_t)w.b * (a.S / kPage) + (group_of(j) / kPage) % (a.S / kPage))
                           : 0;
            };
            int page = page_of(0);
            for (int j = 0; j < w.nt; ++j, ++k) {
                const int st = k % L::kStages;
                const int ahead = page_of(j + 1);
                int row = head_row0 + tile_key<D, SINKS>(w, j);
                if (boxes) {
                    const int pos = group_of(j);
                    if (a.ring && pos >= cal) row = -1 - (ws_row0 + (pos - cal));      // a staged row
                    else row = a.table ? (max(page, 0) * a.Hkv + w.kvh) * kPage : head_row0 + pos % a.S;
                }
                if (k >= L::kStages && !(ok = free_again(L::kSFull, k - L::kStages))) break;
                load_tile(&tmK, &tmWK, sK + st * L::kTile, &bar[L::kKFull + st], row);
                k_issued = k + 1;
                if (k >= L::kStages && !(ok = free_again(L::kODone, k - L::kStages) && looked(k - L::kStages))) break;
                load_tile(&tmV, &tmWV, sV + st * L::kTile, &bar[L::kVFull + st], row);
                v_issued = k + 1;
                page = ahead;
            }
        }
        if (!ok) {
            // the last copy issued into each stage lands before the CTA can exit
            for (int q = max(0, k_issued - L::kStages); q < k_issued; ++q) wait(&bar[L::kKFull + q % L::kStages], phase(q));
            for (int q = max(0, v_issued - L::kStages); q < v_issued; ++q) wait(&bar[L::kVFull + q % L::kStages], phase(q));
        }
        __syncwarp();
    } else if (warp >= kWarpMma) {
        // ================= matrix instructions, one lane issuing: warps 12 and 14 S of slot 0 and
        // 1, as soon as the softmax has read the S before; warps 13 and 15 P.V when the weights
        // are there
        constexpr uint32_t idesc_qk = instr_desc_bf16(kBM, kBN, false), idesc_pv = instr_desc_bf16(kBM, D, true);
        const int slot = (warp - kWarpMma) >> 1;
        const bool scores = ((warp - kWarpMma) & 1) == 0, lead = elect_one();
        // K and V tiles: [half][row] from a contiguous cache, [8 rows][half] from 16-row boxes
        const bool boxes = a.table || a.ring;
        const uint32_t half_step = boxes ? 1024 : L::kHalf, group_step = boxes ? L::kHalves * 1024 : 1024;
        auto wait_ok = [&](uint64_t* b, uint32_t parity) -> bool { return all_ok(wait(b, parity)); };
        int k = 0;
        if (scores) {
            const uint32_t q0 = desc_lo(smem_u32(sQ), 16), qhi = desc_hi(1024);
            const uint32_t kd0 = desc_lo(smem_u32(sK), 16), khi = desc_hi(group_step), khalf = half_step >> 4;
            const uint32_t tS = tmem + L::kColS + kBN * slot;
            for (int rd = 0, i = 0; rd * G < nunits && ok; ++rd) {
                if (mine(rd) >= nunits) continue;
                if (!(ok = wait_ok(q_full(slot, i), (uint32_t)((i >> 1) & 1)))) break;
                const int nt = unit_in(i).nt;
                const uint32_t qd = q0 + q_buf(slot, i) * (L::kQTile >> 4);
                for (int j = 0; j < nt; ++j, ++k) {
                    const int st = k % L::kStages;
                    ok = wait_ok(&bar[L::kKFull + st], phase(k)) && (k == 0 || wait_ok(&bar[L::kSFree + slot], (uint32_t)((k - 1) & 1)));
                    if (!ok) break;
                    fence_after();
                    const uint32_t kd = kd0 + st * (L::kTile >> 4);
                    if (lead) {
#pragma unroll
                        for (int s = 0; s < D / 16; ++s)         // 16 dims per instruction
                            mma_ss(tS, qd + (((s >> 2) * L::kQHalf + (s & 3) * 32) >> 4), qhi,
                                   kd + (s >> 2) * khalf + (((s & 3) * 32) >> 4), khi, idesc_qk, s > 0);
                        mma_commit(stage_bar(L::kSFull, slot, k));
                    }
                    __syncwarp();
                }
                ++i;
            }
        } else {
            const uint32_t vd0 = desc_lo(smem_u32(sV), half_step), vhi = desc_hi(group_step), vstep = (2 * group_step) >> 4;
            const uint32_t tP = tmem + L::kColP + L::kPStep * slot, tO = tmem + L::kColO + D * slot;
            for (int rd = 0, i = 0; rd * G < nunits && ok; ++rd) {
                if (mine(rd) >= nunits) continue;
                if (!(ok = wait_ok(q_full(slot, i), (uint32_t)((i >> 1) & 1)))) break;
                const int nt = unit_in(i).nt, w0 = unit_in(i).w0, w1 = unit_in(i).w1;
                for (int j = 0; j < nt; ++j, ++k) {
                    const int st = k % L::kStages;
                    ok = wait_ok(&bar[L::kVFull + st], phase(k)) &&
                         ((j >= w0 && j < w1) || wait_ok(&bar[L::kVClean + st], phase(k))) &&
                         wait_ok(&bar[L::kPFull + slot], (uint32_t)(k & 1));
                    if (!ok) break;
                    fence_after();
                    const uint32_t vd = vd0 + st * (L::kTile >> 4);
                    if (lead) {
#pragma unroll
                        for (int s = 0; s < kBN / 16; ++s)       // keys 16 s .. + 15 of P sit in its columns 8 s .. + 7
                            mma_ts(tO, tP + 8 * s, vd + s * vstep, vhi, idesc_pv, (j > 0 || s > 0));
                        mma_commit(stage_bar(L::kODone, slot, k));
                    }
                    __syncwarp();
                }
                ++i;
            }
        }
        // no product may still target the columns when they are freed
        if (lead) mma_commit(&bar[L::kDone + warp - kWarpMma]);
        __syncwarp();
        wait(&bar[L::kDone + warp - kWarpMma], 0);
        __syncwarp();
    } else if (warp >= kWarpLook) {
        // ================= value rows of boundary tiles: what is not finite becomes 0
        int k = 0;
        for (int rd = 0, i = 0; rd * G < nunits && ok; ++rd) {
            if (mine(rd) >= nunits) continue;
            const Unit w = unit_of<D, SINKS>(a, items, b0, mine(rd));
            for (int j = 0; j < w.nt; ++j, ++k) {
                const int st = k % L::kStages;
                // (every tile in turn: a barrier's parity tells neighbouring phases apart only)
                if (!(ok = all_ok(wait(&bar[L::kVFull + st], phase(k))))) break;
                if (j >= w.w0 && j < w.w1) {
                    if (lane == 0) mbar_arrive(&bar[L::kVClean + st]);
                    continue;
                }
                unsigned char* tile = sV + st * L::kTile;
                bool any = false;
#pragma unroll 1
                for (int q0 = 8 * 32 * (warp - kWarpLook) + lane; q0 < L::kTile / 16; q0 += 8 * 32 * kLookWarps) {
                    uint4 u[8];
                    uint32_t bad = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) u[e] = *reinterpret_cast<const uint4*>(tile + 16 * (q0 + 32 * e));
#pragma unroll
                    for (int e = 0; e < 8; ++e) bad |= odd_bits(u[e].x) | odd_bits(u[e].y) | odd_bits(u[e].z) | odd_bits(u[e].w);
                    if (bad & 0x80008000u) {
                        any = true;
                        for (int q = q0; q < q0 + 8 * 32; q += 32) {
                            uint32_t* x = reinterpret_cast<uint32_t*>(tile + 16 * q);
                            for (int e = 0; e < 4; ++e) {
                                if ((x[e] & 0x7f80u) == 0x7f80u) x[e] &= 0xffff0000u;
                                if ((x[e] & 0x7f800000u) == 0x7f800000u) x[e] &= 0x0000ffffu;
                            }
                        }
                    }
                }
                if (any) spoilt[i % kAhead] = i + 1;
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[L::kVClean + st]);
            }
            ++i;
        }
    } else if (warp == kWarpLoad) {
        // ================= queries of the next unit (rows of 128 bytes a half, token-major)
        const bool lead = elect_one();
        int q = 0;
        for (int rd = 0; rd * G < nunits && ok; ++rd) {
            if (mine(rd) >= nunits) continue;
            const Unit w = unit_of<D, SINKS>(a, items, b0, mine(rd));
            for (int slot = 0; slot < kSlots; ++slot, ++q) {
                const int i = q >> 1, buf = q % L::kQBufs, uses = q / L::kQBufs;
                if (uses > 0 && !(ok = all_ok(wait(&bar[L::kQFree + buf], (uint32_t)((uses - 1) & 1))))) break;
                if (lead) {
                    if (slot == 0) unit_in(i) = w;
                    mbar_arrive_expect_tx(q_full(slot, i), L::kHalves * T * a.g * 128);
#pragma unroll
                    for (int half = 0; half < L::kHalves; ++half)
                        tma_load_3d(sQ + buf * L::kQTile + half * L::kQHalf, &tmQ, 64 * half, w.kvh * a.g, w.row + w.t0 + slot * T,
                                    q_full(slot, i));
                }
                __syncwarp();
            }
        }
        // the last copies land before the CTA can exit
        for (int p = max(0, q - L::kQBufs); p < q; ++p) wait(q_full(p & 1, p >> 1), (uint32_t)((p >> 2) & 1));
        __syncwarp();
    }
    if (!ok && lane == 0) atomicOr(a.hdr, kErrWait);
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
cudaError_t launch(const CUtensorMap* tm, const AttnArgs& a, int b0, const Items& items, int sms, cudaStream_t st) {
    auto kernel = a.sinks ? prompt_attn_kernel<D, true> : prompt_attn_kernel<D, false>;
    if (cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), Plan<D>::kBytes)) return e;
    const long long units = (long long)items.n * a.Hkv;
    return launch_dep(kernel, dim3((unsigned)std::min<long long>(units, sms)), dim3(kThreads), Plan<D>::kBytes, st, tm[0], tm[1], tm[2],
                      tm[3], tm[4], tm[5], a, b0, items);
}

}  // namespace

bool prompt_tc_supported(const Shape& s) {
    const long long rows = s.pages ? (long long)s.pages * s.Hkv * kPage : (long long)s.B * s.Hkv * s.S;
    const long long staged = s.ring ? (long long)s.B * s.Hkv * chunk_ws_rows(s) : 0;
    return s.bf16 && !s.int8 && !s.int4 && (s.d == 64 || s.d == 128) && rows < (1ll << 31) - 128 && staged < (1ll << 31) && s.g <= kBM &&
           s.Hkv < (1 << 20);
}

cudaError_t launch_prompt_tc(const kvc_handle* h, const AttnArgs& a, const Packed& g, cudaStream_t st) {
    const Shape& s = h->sh;
    const int bn = s.d == 128 ? Plan<128>::kBN : Plan<64>::kBN;
    CUtensorMap tm[6];
    const bool boxes = s.pages || s.ring;
    const long long rows = s.pages ? (long long)s.pages * s.Hkv * kPage : (long long)s.B * s.Hkv * s.S;
    if (!row_map(&tm[0], a.kc, rows, s.d, boxes, bn) || !row_map(&tm[1], a.vc, rows, s.d, boxes, bn)) return cudaErrorInvalidValue;
    tm[2] = tm[0]; tm[3] = tm[1];
    if (s.ring) {
        const long long staged = (long long)s.B * s.Hkv * a.ws_rows;
        if (!row_map(&tm[2], a.wk, staged, s.d, boxes, bn) || !row_map(&tm[3], a.wv, staged, s.d, boxes, bn))
            return cudaErrorInvalidValue;
    }
    // queries: dims (64 of a half, head, packed row), boxes of a group's heads and a slot's tokens
    const int T = kBM / s.g;
    {
        const cuuint64_t dims[3] = {(cuuint64_t)s.d, (cuuint64_t)s.Hq, (cuuint64_t)(g.row0 + g.off[g.nb])};
        // (rotated ones lie in d_out, at the start of each head's output)
        const cuuint64_t head = (cuuint64_t)s.d * (s.rope && !s.out_bf16 ? 4 : 2);
        const cuuint64_t strides[2] = {head, s.rope ? head * s.Hq : (cuuint64_t)a.q_stride * 2};
        const cuuint32_t box[3] = {64, (cuuint32_t)s.g, (cuuint32_t)T};
        if (!make_tensor_map_bf16(&tm[4], s.rope ? a.out : const_cast<void*>(a.q), 3, dims, strides, box)) return cudaErrorInvalidValue;
    }
    // outputs, for units whose rows are bf16 and there in full: boxes of a warp's 32 rows
    static thread_local Items items;      // 8 KB of kernel parameters: not on the stack
    items.boxed = s.out_bf16 && 32 % s.g == 0;
    tm[5] = tm[4];
    if (items.boxed) {
        const cuuint64_t dims[3] = {(cuuint64_t)s.d, (cuuint64_t)s.Hq, (cuuint64_t)(g.row0 + g.off[g.nb])};
        const cuuint64_t strides[2] = {(cuuint64_t)s.d * 2, (cuuint64_t)s.d * 2 * s.Hq};
        const cuuint32_t box[3] = {64, (cuuint32_t)s.g, (cuuint32_t)(32 / s.g)};
        if (!make_tensor_map_bf16(&tm[5], a.out, 3, dims, strides, box)) return cudaErrorInvalidValue;
    }
    // longest first: an item's work is its number of key tiles.  The host's lengths order the
    // units and choose the split only; the kernel reads the cut on the device.
    std::vector<std::pair<int, int4>> work;
    for (int i = 0; i < g.nb; ++i) {
        const int n = g.off[i + 1] - g.off[i], cut = h->np[g.b0 + i];
        for (int t = 0; t < n; t += kSlots * T) {
            const int first = cut + t, last = cut + std::min(n, t + kSlots * T) - 1;
            const int k0 = (s.W > 0 ? std::max(0, first - s.W + 1) : 0) & ~15;
            const int sunk = (std::min(s.sinks, k0) + bn - 1) / bn;
            work.push_back({-((last - k0) / bn + 1 + sunk), make_int4(i, t, (int)(g.row0 + g.off[i]), n)});
        }
    }
    std::stable_sort(work.begin(), work.end(), [](const auto& x, const auto& y) { return x.first < y.first; });
    // fewer units than SMs and long ones: split their keys, as far as the cache's split-K
    // workspace reaches (rows of this group only: they are packed from 0 in it)
    const long long units = (long long)work.size() * s.Hkv, packed = g.off[g.nb];
    const int longest = work.empty() ? 0 : -work[0].first;
    long long parts = 1;
    if (units * 2 <= h->num_sms && longest >= 2 * kSplitTiles)
        parts = std::min<long long>({h->num_sms / units, (long long)longest / kSplitTiles, (long long)s.B * s.max_splits / packed, kMaxKeyParts,
                                     kItems / (long long)work.size()});
    items.parts = (int)std::max(1ll, parts);
    AttnArgs part = a;
    if (items.parts > 1) split_workspace(h, g, items.parts, &part);
    const size_t per = kItems / items.parts;
    for (size_t i0 = 0; i0 < work.size(); i0 += per) {
        const int m = (int)std::min<size_t>(per, work.size() - i0);
        items.n = m * items.parts;
        for (int i = 0; i < m; ++i)
            for (int q = 0; q < items.parts; ++q) {
                items.e[i * items.parts + q] = work[i0 + i].second;
                items.e[i * items.parts + q].x |= q << 16;
            }
        const cudaError_t e = s.d == 128 ? launch<128>(tm, part, g.b0, items, h->num_sms, st) : launch<64>(tm, part, g.b0, items, h->num_sms, st);
        if (e != cudaSuccess) return e;
    }
    if (items.parts > 1) return launch_join(part, g, st);
    return cudaSuccess;
}

}  // namespace kvc
