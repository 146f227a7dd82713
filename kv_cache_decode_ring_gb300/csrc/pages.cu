// pages.cu -- the block table of paged caches ([LEAN] §6.1; [LOOP] §六, §八 Q1), and whole
// requests forked, copied, freed and compacted.
//
// [LOOP] §八 Q1: requests that branch from one prompt share its pages until one of them
// writes.  Every physical page counts the block-table entries that name it.  A fork copies
// table entries only; whoever is about to write into a page that others also hold first
// gets a page of its own (map_pages), with the old page's bytes copied where it still
// holds rows of that request.  A page is free once its last holder gave it up.
//
// A page is a physical page index into every per-page array of the state: K and V rows
// [pages][Hkv][16], or for the INT8 tiers codes, scales and witnesses, one quantization
// block per KV head.
#include <algorithm>
#include <cstring>
#include <new>
#include <vector>

#include "int4.h"
#include "kvc_internal.h"

namespace kvc {
namespace {

// Table entries and page pairs ride in kernel parameters, few or many per launch.
constexpr int kFew = 64, kMany = 1024;

template <int N>
struct TableUpdates {
    int n;
    int2 e[N];                            // (table index, physical page)
};

template <int N>
__global__ void table_update_kernel(const __grid_constant__ TableUpdates<N> u, int32_t* table) {
    dep_wait();                           // launched dependent, as every kernel here: see launch_dep
    dep_release();
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < u.n) table[u.e[i].x] = u.e[i].y;
}

template <int N>
cudaError_t update_some(int32_t* table, const int2* upd, size_t n, cudaStream_t st) {
    static thread_local TableUpdates<N> u;
    u.n = (int)n;
    std::memcpy(u.e, upd, n * sizeof(int2));
    return launch_dep(table_update_kernel<N>, dim3(((int)n + 255) / 256), dim3(256), 0, st, u, table);
}

cudaError_t send_table(kvc_handle* h, cudaStream_t st) {
    return cudaMemcpyAsync(h->state + h->L.table, h->table_h.data(), h->table_h.size() * 4, cudaMemcpyHostToDevice, st);
}

// The changed entries; very many at once (a large prefill), the whole table.
cudaError_t update_table(kvc_handle* h, const int2* upd, size_t count, cudaStream_t st) {
    int32_t* table = reinterpret_cast<int32_t*>(h->state + h->L.table);
    if (count > 4 * (size_t)kMany) return send_table(h, st);
    for (size_t i0 = 0; i0 < count; i0 += kMany) {
        const size_t n = std::min<size_t>(kMany, count - i0);
        const cudaError_t e = n <= kFew ? update_some<kFew>(table, upd + i0, n, st)
                                        : update_some<kMany>(table, upd + i0, n, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t update_table(kvc_handle* h, const std::vector<int2>& upd, cudaStream_t st) {
    return update_table(h, upd.data(), upd.size(), st);
}

// ---- copies of whole pages -------------------------------------------------------
constexpr int kMaxParts = 5;              // per-page arrays: K, V or codes, scales, witnesses

// One per-block array: `bytes` per 16 slots of one KV head.
struct Part {
    char* base;
    long long bytes;
};

// Page `to` takes the bytes of page `from` (< 0: none); table entry `entry` (< 0: none) names it.
struct Move {
    int entry, from, to;
};

template <int N>
struct Moves {
    Part part[kMaxParts];
    int32_t* table;
    int parts, Hkv;
    Move e[N];
};

// Bound by HBM: four 16-byte units in flight a thread (eight: no faster), 983 pages of 64 KB in
// 18 us.  grid (moves, parts); a page is Hkv * bytes contiguous bytes of each part.  The pages written
// are disjoint from the pages read.
template <int N>
__global__ void __launch_bounds__(256) move_pages_kernel(const __grid_constant__ Moves<N> m) {
    const Move e = m.e[blockIdx.x];
    dep_wait();
    if (e.entry >= 0 && blockIdx.y == 0 && threadIdx.x == 0) m.table[e.entry] = e.to;
    if (e.from < 0) return;
    const Part p = m.part[blockIdx.y];
    const size_t page = (size_t)m.Hkv * p.bytes;
    const char* from = p.base + (size_t)e.from * page;
    char* to = p.base + (size_t)e.to * page;
    if (page % 16 == 0) {
        const uint4* f = reinterpret_cast<const uint4*>(from);
        uint4* t = reinterpret_cast<uint4*>(to);
        const int n = (int)(page / 16);
        for (int base = threadIdx.x; base < n; base += 4 * 256) {
            uint4 x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (base + j * 256 < n) x[j] = f[base + j * 256];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (base + j * 256 < n) t[base + j * 256] = x[j];
        }
    } else {                              // scales: 4 bytes per KV head
        for (int i = threadIdx.x; i < (int)(page / 4); i += 256)
            reinterpret_cast<uint32_t*>(to)[i] = reinterpret_cast<const uint32_t*>(from)[i];
    }
}

// The per-block arrays of a cache.
int parts_of(const kvc_handle* h, Part* p) {
    const Shape& s = h->sh;
    const Layout& L = h->L;
    auto part = [&](size_t off, long long bytes) { return Part{h->state + off, bytes}; };
    int n = 0;
    if (!s.int8) {
        p[n++] = part(L.k, (long long)(kPage * row_bytes(s)));
        p[n++] = part(L.v, (long long)(kPage * row_bytes(s)));
        return n;
    }
    p[n++] = part(L.kq, (long long)kQBlock * s.d);
    p[n++] = part(L.vq, (long long)kQBlock * s.d);
    p[n++] = part(L.sk, 4);
    p[n++] = part(L.sv, 4);
    if (!s.dither) p[n++] = part(L.wit, kQBlock * kBands * 2);
    return n;
}

template <int N>
cudaError_t move_some(const kvc_handle* h, const Move* moves, size_t n, cudaStream_t st) {
    static thread_local Moves<N> m;
    m.parts = parts_of(h, m.part);
    m.Hkv = h->sh.Hkv;
    m.table = reinterpret_cast<int32_t*>(h->state + h->L.table);
    std::memcpy(m.e, moves, n * sizeof(Move));
    return launch_dep(move_pages_kernel<N>, dim3((unsigned)n, m.parts), dim3(256), 0, st, m);
}

cudaError_t move_pages(const kvc_handle* h, const std::vector<Move>& moves, cudaStream_t st) {
    for (size_t i0 = 0; i0 < moves.size(); i0 += kMany) {
        const size_t n = std::min<size_t>(kMany, moves.size() - i0);
        const cudaError_t e = n <= kFew ? move_some<kFew>(h, moves.data() + i0, n, st) : move_some<kMany>(h, moves.data() + i0, n, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// ---- copies of whole requests ------------------------------------------------------
constexpr int kCopyBlocks = 8;            // 16-slot blocks per CTA: 128 rows, as the store's copies
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;
constexpr int kCopyGroups = 64;           // sources per launch
constexpr int kCopyTargets = 512;         // destinations per launch

struct CopyGroup {
    int src;                              // request of the source cache (-1: the destinations become empty)
    int first, n;                         // its destinations: target[first .. first + n)
    int rows;                             // slots [0, rows) hold rows to copy (0: none, as on a fork of pages)
    int len;                              // next_position after the copy
    int tail;                             // rows of the exact tail (INT8)
    uint32_t req_id;                      // Tier B
};

struct CopySide {
    Part part[kMaxParts];
    int32_t* table;                       // paged: block table, else nullptr
    int32_t* pos;
    int32_t* next_pos;
    __nv_bfloat16* ktail; __nv_bfloat16* vtail;
    uint32_t* req_id;
    int S;
};

struct CopyArgs {
    CopySide from, to;
    int parts, Hkv, d, ring, int8;
    int share;                            // destinations take the source's pages (none: give theirs up)
    CopyGroup group[kCopyGroups];
    int target[kCopyTargets];
};

// Bound by HBM: eight units of K and eight of V in flight a thread; 4096 rows of 8 bf16 heads of 128
// into 16 branches in 44 us (6.5 TB/s, 268 MB of it written).
// grid (max of ceil(rows / 128) and destinations, Hkv + 1, groups).  Plane y < Hkv: KV head
// y's rows of the group's source, read once and written to each of its destinations; its
// scales, witnesses and exact tail for the INT8 tiers.  Plane Hkv, a CTA per destination:
// positions, next_position, request ID and (share) block-table entries.
__device__ __forceinline__ void copy_books(const CopyArgs& a, const CopyGroup& g, const int* target) {
    for (int j = blockIdx.x; j < g.n; j += gridDim.x) {
        const int b = target[j];
        int32_t* pb = a.to.pos + (size_t)b * a.to.S;
        // a ring's slots move with their positions (equal S on both sides); a contiguous
        // cache holds position s in slot s, and nothing from next_position on
        const int old = a.to.next_pos[b];
        const int hi = a.ring ? a.to.S : min(a.to.S, max(g.len, old));
        for (int s = threadIdx.x; s < hi; s += kCopyThreads)
            pb[s] = g.src < 0 ? -1 : a.ring ? a.from.pos[(size_t)g.src * a.from.S + s] : s < g.len ? s : -1;
        if (a.share) {
            const int npg = a.to.S / kPage;
            for (int lp = threadIdx.x; lp < npg; lp += kCopyThreads)
                a.to.table[(size_t)b * npg + lp] = g.src < 0 ? -1 : a.from.table[(size_t)g.src * npg + lp];
        }
        __syncthreads();                  // every thread has read the old next_position
        if (threadIdx.x == 0) {
            a.to.next_pos[b] = g.len;
            if (a.to.req_id && g.src >= 0) a.to.req_id[b] = g.req_id;
        }
    }
}

template <typename U>
__global__ void __launch_bounds__(kCopyThreads) copy_requests_kernel(const __grid_constant__ CopyArgs a) {
    dep_wait();
    dep_release();
    const CopyGroup g = a.group[blockIdx.z];
    const int h = blockIdx.y;
    const int* target = a.target + g.first;
    if (h == a.Hkv) {
        copy_books(a, g, target);
        return;
    }
    if (g.src < 0) return;
    const int s0 = blockIdx.x * kCopyBlocks * kPage;
    const int rows = min(g.rows - s0, kCopyBlocks * kPage);
    if (a.int8 && blockIdx.x == 0) {
        // exact tail rows [0, tail) of 2 d bytes, K and V
        const size_t from = ((size_t)g.src * a.Hkv + h) * kQBlock * a.d;
        const int n = g.tail * a.d / 8;
        for (int i = threadIdx.x; i < n; i += kCopyThreads) {
            const uint4 k = reinterpret_cast<const uint4*>(a.from.ktail + from)[i];
            const uint4 v = reinterpret_cast<const uint4*>(a.from.vtail + from)[i];
            for (int j = 0; j < g.n; ++j) {
                const size_t to = ((size_t)target[j] * a.Hkv + h) * kQBlock * a.d;
                reinterpret_cast<uint4*>(a.to.ktail + to)[i] = k;
                reinterpret_cast<uint4*>(a.to.vtail + to)[i] = v;
            }
        }
    }
    if (rows <= 0) return;
    // byte offset of unit u of row r (from s0) in an array of `row` bytes per slot
    const int row = (int)(a.from.part[0].bytes / kPage), upr = row / (int)sizeof(U), total = rows * upr;
    const char* fk = a.from.part[0].base;
    const char* fv = a.from.part[1].base;
    char* tk = a.to.part[0].base;
    char* tv = a.to.part[1].base;
    for (int base = threadIdx.x; base < total; base += kCopyUnroll * kCopyThreads) {
        U kx[kCopyUnroll], vx[kCopyUnroll];
#pragma unroll
        for (int j = 0; j < kCopyUnroll; ++j) {
            const int i = base + j * kCopyThreads;
            if (i >= total) continue;
            const size_t o = kv_row(a.from.table, g.src, h, s0 + i / upr, a.Hkv, a.from.S) * row + (size_t)(i % upr) * sizeof(U);
            kx[j] = *reinterpret_cast<const U*>(fk + o);
            vx[j] = *reinterpret_cast<const U*>(fv + o);
        }
        for (int t = 0; t < g.n; ++t) {
#pragma unroll
            for (int j = 0; j < kCopyUnroll; ++j) {
                const int i = base + j * kCopyThreads;
                if (i >= total) continue;
                const size_t o = kv_row(a.to.table, target[t], h, s0 + i / upr, a.Hkv, a.to.S) * row + (size_t)(i % upr) * sizeof(U);
                *reinterpret_cast<U*>(tk + o) = kx[j];
                *reinterpret_cast<U*>(tv + o) = vx[j];
            }
        }
    }
    // INT8: scales and witnesses of the blocks (rows is a multiple of 16 there)
    for (int q = 2; q < a.parts; ++q) {
        const int words = (int)(a.from.part[q].bytes / 4), n = rows / kQBlock * words;
        for (int i = threadIdx.x; i < n; i += kCopyThreads) {
            const int k = s0 / kQBlock + i / words;
            const size_t from = int8_block(a.from.table, g.src, h, k, a.Hkv, a.from.S) * words + i % words;
            const uint32_t x = reinterpret_cast<const uint32_t*>(a.from.part[q].base)[from];
            for (int t = 0; t < g.n; ++t)
                reinterpret_cast<uint32_t*>(a.to.part[q].base)[int8_block(a.to.table, target[t], h, k, a.Hkv, a.to.S) * words +
                                                               i % words] = x;
        }
    }
}

// The same between a bf16 cache and an INT4 one of D dims: rows are quantised (QUANT) or read back
// as bf16 (m + u s rounded once) on the way.  A thread takes 16 dims of a row, K and V, as int4.h
// lays them out, kConvertUnroll rows in flight.  64000 rows of 8 heads of 128: quantised in 57 us, read back
// in 48 (6.0 and 7.2 TB/s, part of it in L2); 8 dims a thread and divisions took 89 and 53.
constexpr int kConvertUnroll = 2;

template <int D, bool QUANT>
__global__ void __launch_bounds__(kCopyThreads) convert_requests_kernel(const __grid_constant__ CopyArgs a) {
    dep_wait();
    dep_release();
    const CopyGroup g = a.group[blockIdx.z];
    const int h = blockIdx.y;
    const int* target = a.target + g.first;
    if (h == a.Hkv) {
        copy_books(a, g, target);
        return;
    }
    constexpr int kVec = D / 16, kRow4 = int4::row_size(D), kStep = kCopyThreads / kVec;
    const int s0 = blockIdx.x * kCopyBlocks * kPage, rows = min(g.rows - s0, kCopyBlocks * kPage);
    if (g.src < 0 || rows <= 0) return;
    const int e = threadIdx.x % kVec;
    // row r from s0 of request b, as kv_row
    auto head_row = [&](const CopySide& c, int b) { return c.table ? (size_t)h * kPage : ((size_t)b * a.Hkv + h) * c.S + s0; };
    auto row_of = [&](const CopySide& c, int b, size_t head, int r) -> size_t {
        if (!c.table) return head + r;
        const int page = max(c.table[(size_t)b * (c.S / kPage) + (s0 + r) / kPage], 0);
        return (size_t)page * (a.Hkv * kPage) + head + r % kPage;
    };
    const size_t from = head_row(a.from, g.src);
    for (int r0 = threadIdx.x / kVec; r0 - (int)threadIdx.x / kVec < rows; r0 += kConvertUnroll * kStep) {
        uint4 kx[kConvertUnroll][2], vx[kConvertUnroll][2];
        int4::Unit u[kConvertUnroll];
#pragma unroll
        for (int j = 0; j < kConvertUnroll; ++j) {
            const int r = r0 + j * kStep;
            kx[j][0] = kx[j][1] = vx[j][0] = vx[j][1] = make_uint4(0, 0, 0, 0);
            u[j] = int4::Unit{};
            if (r >= rows) continue;
            const size_t row = row_of(a.from, g.src, from, r);
            if constexpr (QUANT) {
                const uint4* k = reinterpret_cast<const uint4*>(a.from.part[0].base) + row * (D / 8) + int4::chunk_of(e);
                const uint4* v = reinterpret_cast<const uint4*>(a.from.part[1].base) + row * (D / 8) + int4::chunk_of(e);
                kx[j][0] = k[0]; kx[j][1] = k[2];
                vx[j][0] = v[0]; vx[j][1] = v[2];
            } else {
                u[j] = int4::load<D>(a.from.part[0].base + row * kRow4, a.from.part[1].base + row * kRow4, e);
            }
        }
#pragma unroll
        for (int j = 0; j < kConvertUnroll; ++j) {
            const int r = r0 + j * kStep;
            if constexpr (QUANT) {
                u[j] = int4::quantise(kx[j], vx[j], e);
            } else {
                kx[j][0] = int4::values_bf16(u[j].k.x, u[j].kp); kx[j][1] = int4::values_bf16(u[j].k.y, u[j].kp);
                vx[j][0] = int4::values_bf16(int4::v_codes(u[j].v.x, e), u[j].vp);
                vx[j][1] = int4::values_bf16(int4::v_codes(u[j].v.y, e), u[j].vp);
            }
            if (r >= rows) continue;
            for (int t = 0; t < g.n; ++t) {
                const size_t row = row_of(a.to, target[t], head_row(a.to, target[t]), r);
                if constexpr (QUANT) {
                    int4::store<D>(a.to.part[0].base + row * kRow4, a.to.part[1].base + row * kRow4, e, u[j]);
                } else {
                    uint4* k = reinterpret_cast<uint4*>(a.to.part[0].base) + row * (D / 8) + int4::chunk_of(e);
                    uint4* v = reinterpret_cast<uint4*>(a.to.part[1].base) + row * (D / 8) + int4::chunk_of(e);
                    k[0] = kx[j][0]; k[2] = kx[j][1];
                    v[0] = vx[j][0]; v[2] = vx[j][1];
                }
            }
        }
    }
}

void side_of(kvc_handle* h, CopySide* c) {
    const Shape& s = h->sh;
    parts_of(h, c->part);
    c->table = s.pages ? reinterpret_cast<int32_t*>(h->state + h->L.table) : nullptr;
    c->pos = reinterpret_cast<int32_t*>(h->state + h->L.pos);
    c->next_pos = reinterpret_cast<int32_t*>(h->state + h->L.next_pos);
    if (s.int8) {
        c->ktail = reinterpret_cast<__nv_bfloat16*>(h->state + h->L.ktail);
        c->vtail = reinterpret_cast<__nv_bfloat16*>(h->state + h->L.vtail);
    }
    c->req_id = s.dither ? reinterpret_cast<uint32_t*>(h->state + h->L.req_id) : nullptr;
    c->S = s.S;
}

// Copies in the order of their sources (worked out before anything changes).
std::vector<int> by_source(const std::vector<int>& src) {
    std::vector<int> order(src.size());
    for (size_t i = 0; i < order.size(); ++i) order[i] = (int)i;
    std::stable_sort(order.begin(), order.end(), [&](int x, int y) { return src[x] < src[y]; });
    return order;
}

// Destinations dst[i] of `to` take the rows of requests src[i] of `from` (src[i] < 0:
// nothing).  rows_of(b): slots whose rows move.  Destinations of one source share its reads.
// share: a paged cache's destinations name the source's pages (the host table already does).
template <typename Rows>
cudaError_t copy_requests(kvc_handle* to, kvc_handle* from, const std::vector<int>& src, const std::vector<int>& dst,
                          const std::vector<int>& order, Rows rows_of, bool share, cudaStream_t st) {
    const Shape& s = to->sh;
    static thread_local CopyArgs a;       // 5 KB of kernel parameters: not on the stack
    a = CopyArgs{};
    side_of(from, &a.from);
    side_of(to, &a.to);
    Part parts[kMaxParts];
    a.parts = parts_of(to, parts);
    a.Hkv = s.Hkv; a.d = s.d; a.ring = s.ring; a.int8 = s.int8; a.share = share;
    const bool wide = (s.int8 ? s.d : row_bytes(s)) % 16 == 0;
    size_t i = 0;
    while (i < order.size()) {
        int ng = 0, nt = 0, most = 0, widest = 1;
        while (i < order.size() && nt < kCopyTargets) {
            const int b = src[order[i]];
            if (ng == 0 || a.group[ng - 1].src != b) {
                if (ng == kCopyGroups) break;
                CopyGroup& g = a.group[ng++];
                g = CopyGroup{b, nt, 0, 0, 0, 0, 0};
                if (b >= 0) {
                    g.rows = rows_of(b);
                    g.len = from->np[b];
                    g.tail = s.int8 ? g.len % kQBlock : 0;
                    g.req_id = s.dither ? from->req_id_h[b] : 0;
                }
                most = std::max(most, g.rows);
            }
            a.target[nt++] = dst[order[i++]];
            widest = std::max(widest, ++a.group[ng - 1].n);
        }
        const int per = kCopyBlocks * kPage;
        dim3 grid(std::max((most + per - 1) / per, widest), s.Hkv + 1, ng);
        auto kernel = wide ? copy_requests_kernel<uint4> : copy_requests_kernel<uint32_t>;
        if (s.int4 != from->sh.int4)
            kernel = s.d == 128 ? (s.int4 ? convert_requests_kernel<128, true> : convert_requests_kernel<128, false>)
                                : (s.int4 ? convert_requests_kernel<64, true> : convert_requests_kernel<64, false>);
        const cudaError_t e = launch_dep(kernel, grid, dim3(kCopyThreads), 0, st, a);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Slots of request b that hold rows to copy: complete blocks only for the INT8 tiers
// (the rest is the exact tail).
int held_rows(const kvc_handle* h, int b) {
    const Shape& s = h->sh;
    const int n = s.int8 ? h->np[b] / kQBlock * kQBlock : h->np[b];
    return std::min(n, s.S);
}

// No block-table entry of request b from this one on names a page: a contiguous cache maps no
// page behind its rows.
int held_pages(const kvc_handle* h, int b) {
    const Shape& s = h->sh;
    return s.ring ? s.S / kPage : (h->np[b] + kPage - 1) / kPage;
}

// Restored INT8 blocks live in a pool of their own, which copies do not follow.
bool has_restored(const kvc_handle* h, int b) {
    if (h->xn_h.empty()) return false;
    for (int k = 0; k < h->sh.Hkv; ++k)
        if (h->xn_h[(size_t)b * h->sh.Hkv + k] > 0) return true;
    return false;
}

// Restored blocks of the listed requests return to the pool.
cudaError_t drop_restored(kvc_handle* h, const std::vector<int>& reqs, cudaStream_t st) {
    bool any = false;
    for (int b : reqs) any |= has_restored(h, b);
    if (!any) return cudaSuccess;
    std::vector<int32_t> cut(h->np);
    for (int b : reqs) cut[b] = 0;
    return int8_drop_restored(h, cut.data(), st);
}

// n distinct requests of [0, B)
bool distinct(const int32_t* list, int32_t n, int B, std::vector<char>* seen) {
    seen->assign(B, 0);
    for (int i = 0; i < n; ++i) {
        if (list[i] < 0 || list[i] >= B || (*seen)[list[i]]) return false;
        (*seen)[list[i]] = 1;
    }
    return true;
}

}  // namespace

void drop_page(kvc_handle* h, int32_t& entry) {
    if (entry < 0) return;
    if (--h->page_ref[entry] == 0) h->page_free.push_back(entry);
    entry = -1;
}

// Nothing is allocated (page_free has room for every page).  More entries than one launch takes go with the whole table where
// that is not much larger: 32 requests of 512 table entries each that give up 125 pages, 38 us a trim, in four launches 52.
cudaError_t unmap_pages(kvc_handle* h, const int32_t* cut, cudaStream_t st) {
    static thread_local int2 upd[4 * kMany];
    const Shape& s = h->sh;
    const int npg = s.S / kPage;
    size_t n = 0;
    for (int b = 0; b < s.B; ++b)
        for (int lp = (cut[b] + kPage - 1) / kPage; lp < npg; ++lp, ++n) {
            const size_t idx = (size_t)b * npg + lp;
            if (h->table_h[idx] < 0) break;                // (no page is mapped behind the rows)
            if (n < 4 * kMany) upd[n] = make_int2((int)idx, -1);
            drop_page(h, h->table_h[idx]);
        }
    if (n == 0) return cudaSuccess;
    // (a graph gets the entries themselves: a captured copy would read the host's table at each replay)
    return n > kMany && h->table_h.size() <= 16 * n && !capturing(st) ? send_table(h, st) : update_table(h, upd, n, st);
}

// Too few pages: nothing changes and *status = KVC_ERR_CAPACITY.  Everything is allocated before
// the books change, here and below: a call that runs out of host memory leaves them as they were.
cudaError_t remap_pages(kvc_handle* h, const std::vector<int>& reqs, const std::vector<int>& lo,
                        const std::vector<int>& hi, cudaStream_t st, int* status) {
    const Shape& s = h->sh;
    const size_t npg = s.S / kPage, n = reqs.size();
    std::vector<int32_t> left(h->page_ref);
    std::vector<int2> upd;                 // entries that were mapped or will be: the new page
    upd.reserve(n * npg);
    long long need = 0, released = 0;
    for (size_t i = 0; i < n; ++i)
        for (size_t lp = 0; lp < npg; ++lp) {
            const size_t idx = reqs[i] * npg + lp;
            const int32_t e = h->table_h[idx];
            const bool touched = page_touched(s, (int)lp, lo[i], hi[i]);
            need += touched;
            if (e >= 0 && --left[e] == 0) ++released;
            if (e >= 0 || touched) upd.push_back(make_int2((int)idx, touched ? 1 : -1));
        }
    *status = need > released + (long long)h->page_free.size() ? KVC_ERR_CAPACITY : KVC_OK;
    if (*status != KVC_OK) return cudaSuccess;
    for (const int2& u : upd) drop_page(h, h->table_h[u.x]);
    for (int2& u : upd) {
        if (u.y < 0) continue;
        u.y = h->table_h[u.x] = h->page_free.back();
        h->page_free.pop_back();
        h->page_ref[u.y] = 1;
    }
    return update_table(h, upd, st);
}

// From the host free list; the device table follows on `st`.  On exhaustion nothing
// changes and *status = KVC_ERR_CAPACITY.  A shared page is copied where the request may
// still hold rows in it: always on a ring (its slots are reused), below from[b] on a
// contiguous bf16/fp32 cache, and never on a contiguous INT8 cache (the rows of an
// incomplete block sit in the exact tail, its page is written when the block completes).
// A copy is refused under stream capture (KVC_ERR_UNSUPPORTED): a replay would bring the
// old page's bytes back over rows that earlier replays wrote.  On a ring so is a write by a
// request that shares any page: replays advance on the device and come round to it, where no
// host looks who else holds it.  (A contiguous cache's later pages are unmapped: the kernels
// flag rows there.)
cudaError_t map_pages(kvc_handle* h, const std::vector<int>& from, const std::vector<int>& to, cudaStream_t st,
                      int* status) {
    const Shape& s = h->sh;
    const int np = s.S / kPage;
    if (s.ring && capturing(st))
        for (int b = 0; b < s.B; ++b)
            for (int lp = 0; to[b] > from[b] && lp < np; ++lp) {
                const int32_t e = h->table_h[(size_t)b * np + lp];
                if (e >= 0 && h->page_ref[e] > 1) { *status = KVC_ERR_UNSUPPORTED; return cudaSuccess; }
            }
    struct Need { int idx, old; bool keep; };
    std::vector<Need> need;                // table indices to map, in request and page order
    auto undo = [&] {
        for (const Need& x : need)
            if (x.old >= 0) ++h->page_ref[x.old];
    };
    std::vector<int2> upd;
    std::vector<Move> moves;
    bool copies = false;
    *status = KVC_OK;
    try {
        for (int b = 0; b < s.B; ++b) {
            const long long lo = from[b], hi = to[b];
            if (hi <= lo) continue;
            const long long first = lo / kPage, count = std::min<long long>((hi - 1) / kPage - first + 1, np);
            for (long long q = 0; q < count; ++q) {
                const int lp = (int)((first + q) % np);
                const size_t idx = (size_t)b * np + lp;
                const int32_t e = h->table_h[idx];
                if (e >= 0 && h->page_ref[e] == 1) continue;
                need.push_back(Need{(int)idx, e, e >= 0 && (s.ring || (!s.int8 && (long long)lp * kPage < lo))});
                if (e >= 0) --h->page_ref[e];
                copies |= e >= 0;
            }
        }
        upd.reserve(need.size());
        moves.reserve(copies ? need.size() : 0);
    } catch (...) {
        undo();
        throw;
    }
    if (need.empty()) return cudaSuccess;
    if (need.size() > h->page_free.size()) *status = KVC_ERR_CAPACITY;
    else if (copies && capturing(st)) *status = KVC_ERR_UNSUPPORTED;
    if (*status != KVC_OK) {
        undo();
        return cudaSuccess;
    }
    // one launch for copies and their table entries
    for (const Need& x : need) {
        const int page = h->page_free.back();
        h->page_free.pop_back();
        h->page_ref[page] = 1;
        h->table_h[x.idx] = page;
        if (x.keep) moves.push_back(Move{x.idx, x.old, page});
        else upd.push_back(make_int2(x.idx, page));
    }
    if (!moves.empty() && upd.size() <= kFew) {
        for (const int2& u : upd) moves.push_back(Move{u.x, -1, u.y});
        upd.clear();
    }
    const cudaError_t e = move_pages(h, moves, st);
    return e != cudaSuccess || upd.empty() ? e : update_table(h, upd, st);
}

}  // namespace kvc

using namespace kvc;

extern "C" {

int kvc_fork(kvc_t h, int32_t n, const int32_t* h_src, const int32_t* h_dst, kvc_stream_t stream) try {
    if (!h || !on_device(h) || n < 0 || (n > 0 && (!h_src || !h_dst))) return KVC_ERR_ARG;
    const Shape& s = h->sh;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    std::vector<char> is_dst;
    if (!distinct(h_dst, n, s.B, &is_dst)) return KVC_ERR_ARG;
    for (int i = 0; i < n; ++i)
        if (h_src[i] < 0 || h_src[i] >= s.B || is_dst[h_src[i]]) return KVC_ERR_ARG;
    for (int i = 0; i < n; ++i)
        if (has_restored(h, h_src[i])) return KVC_ERR_UNSUPPORTED;
    if (n == 0) return KVC_OK;
    if (capturing(st) || s.Hkv > kMaxGridHeads) return KVC_ERR_UNSUPPORTED;
    const std::vector<int> src(h_src, h_src + n), dst(h_dst, h_dst + n), order = by_source(src);
    if (drop_restored(h, dst, st) != cudaSuccess) return KVC_ERR_CUDA;
    if (s.pages) {
        const int npg = s.S / kPage;
        for (int i = 0; i < n; ++i)
            for (int lp = 0, held = std::max(held_pages(h, src[i]), held_pages(h, dst[i])); lp < held; ++lp) {
                const int32_t page = h->table_h[(size_t)src[i] * npg + lp];
                int32_t& e = h->table_h[(size_t)dst[i] * npg + lp];
                if (e == page) continue;
                if (page >= 0) ++h->page_ref[page];
                drop_page(h, e);
                e = page;
            }
    }
    const bool shared = s.pages > 0;       // rows stay where they are
    if (copy_requests(h, h, src, dst, order, [&](int b) { return shared ? 0 : held_rows(h, b); }, shared, st) != cudaSuccess)
        return KVC_ERR_CUDA;
    for (int i = 0; i < n; ++i) {
        h->np[dst[i]] = h->np[src[i]];
        h->held_lo[dst[i]] = h->held_lo[src[i]];
        if (s.dither) h->req_id_h[dst[i]] = h->req_id_h[src[i]];
    }
    return KVC_OK;
} catch (...) {
    return KVC_ERR_ARG;      // out of host memory
}

int kvc_copy(kvc_t to, kvc_t from, int32_t n, const int32_t* h_src, const int32_t* h_dst, kvc_stream_t stream) try {
    if (!to || !from || !on_device(to) || from->device != to->device || n < 0 || (n > 0 && (!h_src || !h_dst)))
        return KVC_ERR_ARG;
    const Shape &s = to->sh, &f = from->sh;
    // (INT4 caches are bf16 ones here: the copy converts)
    if (s.bf16 != f.bf16 || s.int8 != f.int8 || s.dither != f.dither || s.Hkv != f.Hkv || s.d != f.d || s.ring != f.ring ||
        (s.ring && s.S != f.S) || to->cfg.rope_base != from->cfg.rope_base ||
        (s.dither && (to->cfg.layer_index != from->cfg.layer_index || to->cfg.dither_key_lo != from->cfg.dither_key_lo ||
                      to->cfg.dither_key_hi != from->cfg.dither_key_hi)))
        return KVC_ERR_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    std::vector<char> is_dst;
    if (!distinct(h_dst, n, s.B, &is_dst)) return KVC_ERR_ARG;
    for (int i = 0; i < n; ++i)
        if (h_src[i] < 0 || h_src[i] >= f.B || (to == from && is_dst[h_src[i]])) return KVC_ERR_ARG;
    for (int i = 0; i < n; ++i)
        if (has_restored(from, h_src[i])) return KVC_ERR_UNSUPPORTED;
    for (int i = 0; i < n; ++i) {
        const int len = from->np[h_src[i]];
        if ((!s.ring && len > s.S) || (s.rope && len > s.P)) return KVC_ERR_CAPACITY;
    }
    if (n == 0) return KVC_OK;
    if (capturing(st) || s.Hkv > kMaxGridHeads) return KVC_ERR_UNSUPPORTED;
    const std::vector<int> src(h_src, h_src + n), dst(h_dst, h_dst + n), order = by_source(src);
    if (s.pages) {
        // the destinations give back their pages and map those that the rows need
        std::vector<int> lo(n), hi(n);
        for (int i = 0; i < n; ++i) {
            hi[i] = from->np[src[i]];
            lo[i] = s.ring && hi[i] > s.S ? hi[i] - s.S : 0;
        }
        int rc = KVC_OK;
        if (remap_pages(to, dst, lo, hi, st, &rc) != cudaSuccess) return KVC_ERR_CUDA;
        if (rc) return rc;
    } else if (drop_restored(to, dst, st) != cudaSuccess) {      // (the gate's pool: unpaged caches)
        return KVC_ERR_CUDA;
    }
    if (copy_requests(to, from, src, dst, order, [&](int b) { return held_rows(from, b); }, false, st) != cudaSuccess) return KVC_ERR_CUDA;
    for (int i = 0; i < n; ++i) {
        to->np[dst[i]] = from->np[src[i]];
        to->held_lo[dst[i]] = from->held_lo[src[i]];
        if (s.dither) to->req_id_h[dst[i]] = from->req_id_h[src[i]];
    }
    return KVC_OK;
} catch (...) {
    return KVC_ERR_ARG;      // out of host memory
}

int kvc_free(kvc_t h, int32_t n, const int32_t* h_b, kvc_stream_t stream) try {
    if (!h || !on_device(h) || n < 0 || (n > 0 && !h_b)) return KVC_ERR_ARG;
    const Shape& s = h->sh;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    std::vector<char> seen;
    if (!distinct(h_b, n, s.B, &seen)) return KVC_ERR_ARG;
    if (n == 0) return KVC_OK;
    if (capturing(st) || s.Hkv > kMaxGridHeads) return KVC_ERR_UNSUPPORTED;
    const std::vector<int> dst(h_b, h_b + n), none(n, -1), order = by_source(none);
    if (drop_restored(h, dst, st) != cudaSuccess) return KVC_ERR_CUDA;
    if (s.pages) {
        const int npg = s.S / kPage;
        for (int b : dst)
            for (int lp = 0, held = held_pages(h, b); lp < held; ++lp) drop_page(h, h->table_h[(size_t)b * npg + lp]);
    }
    if (copy_requests(h, h, none, dst, order, [](int) { return 0; }, s.pages > 0, st) != cudaSuccess) return KVC_ERR_CUDA;
    for (int b : dst) h->np[b] = h->held_lo[b] = 0;
    return KVC_OK;
} catch (...) {
    return KVC_ERR_ARG;      // out of host memory
}

int kvc_compact(kvc_t h, int32_t* h_used, kvc_stream_t stream) try {
    if (!h || !on_device(h) || !h_used) return KVC_ERR_ARG;
    const Shape& s = h->sh;
    if (!s.pages) return KVC_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (capturing(st)) return KVC_ERR_UNSUPPORTED;
    const int used = s.pages - (int)h->page_free.size();
    // pages at and past `used` move into the free ones below it: sources and destinations
    // are disjoint, and no page moves that need not
    std::vector<int32_t> to(s.pages, -1);
    std::vector<Move> moves;
    int hole = 0;
    for (int p = used; p < s.pages; ++p) {
        if (h->page_ref[p] == 0) continue;
        while (h->page_ref[hole] != 0) ++hole;
        to[p] = hole;
        moves.push_back(Move{-1, p, hole});
        ++hole;
    }
    if (!moves.empty()) {
        std::vector<int2> upd;
        for (size_t i = 0; i < h->table_h.size(); ++i) {
            const int32_t e = h->table_h[i];
            if (e >= 0 && to[e] >= 0) upd.push_back(make_int2((int)i, to[e]));
        }
        if (move_pages(h, moves, st) != cudaSuccess) return KVC_ERR_CUDA;
        for (const int2& u : upd) h->table_h[u.x] = u.y;
        for (const Move& m : moves) {
            h->page_ref[m.to] = h->page_ref[m.from];
            h->page_ref[m.from] = 0;
        }
        if (update_table(h, upd, st) != cudaSuccess) return KVC_ERR_CUDA;
    }
    h->page_free.clear();
    for (int p = s.pages - 1; p >= used; --p) h->page_free.push_back(p);   // the lowest is taken first
    *h_used = used;
    return KVC_OK;
} catch (...) {
    return KVC_ERR_ARG;      // out of host memory
}

int kvc_page_counts(kvc_t h, int32_t* h_free, int32_t* h_shared) {
    if (!h || !h_free || !h_shared) return KVC_ERR_ARG;
    if (!h->sh.pages) return KVC_ERR_UNSUPPORTED;
    *h_free = (int32_t)h->page_free.size();
    *h_shared = (int32_t)std::count_if(h->page_ref.begin(), h->page_ref.end(), [](int32_t r) { return r > 1; });
    return KVC_OK;
}

}  // extern "C"
