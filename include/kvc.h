/*
 * kvc.h -- C ABI of libkvc, a single-GPU (GB300, sm_103a) library for one
 * autoregressive decode step over a KV cache.
 *
 * Sources of the operations, cited by page title and section:
 *   [LEAN]    "用Lean4形式化验证滑动窗口KV Cache的正确性" (framerc.cn/news/4505248)
 *   [PREFIX]  "LLM 機制實驗（五）：改了歷史，能否只重算變化的後綴？"
 *             (huhohoo.com/zh-TW/docs/llm/longest-prefix-reuse)
 *   [LOOP]    "KV Cache 自回归生成推理（增量更新与状态拼接）" (airsota.com/?p=549)
 *   [WITCERT] "WitCert: Sound Runtime Risk Observability and Gating for
 *             KV-Cache Quantization" (agifrontier.github.io tutorial)
 *
 * Conventions
 *  - Ownership: the caller owns every device buffer (the cache state, inputs,
 *    outputs) and the stream.  The library owns only the small host handle.
 *    kvc_create() and kvc_destroy() neither allocate nor free device memory.
 *  - Pointers named d_* are device pointers, h_* host pointers.  Device
 *    inputs must be 16-byte aligned and densely packed in the stated layout.
 *  - Devices: a handle lives on the device that was current at kvc_create();
 *    every later call on it that touches the device must run with that device
 *    current, else it returns KVC_ERR_ARG and enqueues nothing.
 *  - Streams: kvc_stream_t is a cudaStream_t (NULL = the legacy default
 *    stream).  Compute calls only enqueue work and return; none waits for the
 *    GPU, except kvc_create (uploads tables), kvc_export and
 *    kvc_device_status (read back).  One handle serves one stream at a time:
 *    calls on one handle from different streams race on its state.  The
 *    decode-path kernels (append, decode, combine) start as programmatic
 *    dependent launches.  They may be scheduled while the previous kernel on the
 *    stream drains, but they wait for it to complete before touching memory.
 *    So the order of work on a stream, and CUDA graph capture, behave as with
 *    ordinary launches.
 *  - Element types: KVC_F32 = IEEE fp32, KVC_BF16 = bfloat16.  q, k and v
 *    use the cache dtype; outputs use kvc_config.out_dtype (default: the
 *    cache dtype).
 *  - Positions are absolute, 0-based, signed 32-bit; -1 marks an empty slot.
 *  - Errors: every entry point returns a KVC_* status.  Arguments are checked
 *    on the host before anything is enqueued; a failed call changes nothing.
 *    Kernels also check their own bounds and set a sticky device error word
 *    (read by kvc_device_status) instead of writing out of bounds.
 */
#ifndef KVC_H
#define KVC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct kvc_handle* kvc_t;
typedef void* kvc_stream_t; /* a cudaStream_t */

/* ---- status codes ---------------------------------------------------- */
#define KVC_OK 0
#define KVC_ERR_ARG 1          /* null pointer, bad shape/dtype/size, call out of order,
                                  or out of host memory */
#define KVC_ERR_CAPACITY 2     /* contiguous cache full: position >= max_seq_len
                                  ([LOOP] §三 "assert pos < max_seq_len"), or a
                                  position beyond the RoPE table */
#define KVC_ERR_EVICTED 3      /* trim needs rows the cache no longer holds exactly:
                                  evicted from a ring ([PREFIX] "為什麼滑窗部分命中必須回退")
                                  or already folded into an INT8 block */
#define KVC_ERR_CUDA 4         /* a CUDA runtime call failed */
#define KVC_ERR_UNSUPPORTED 5  /* valid request this build does not implement */
#define KVC_ERR_DEVICE 6       /* a kernel flagged an error (see kvc_device_status) */

/* ---- configuration --------------------------------------------------- */
enum { KVC_F32 = 0, KVC_BF16 = 1 };
enum { KVC_CONTIGUOUS = 0, KVC_RING = 1 };
enum { KVC_QUANT_NONE = 0, KVC_QUANT_INT8 = 1, KVC_QUANT_INT8_DITHER = 2, KVC_QUANT_INT4 = 3 };

typedef struct {
    int32_t dtype;        /* KVC_F32 or KVC_BF16 */
    int32_t layout;       /* KVC_CONTIGUOUS: slot = position, capacity = max_seq_len
                             ([LOOP] §三, preallocated (B, H, max_S, D) buffers);
                             KVC_RING: slot = position mod W, capacity = W
                             ([LEAN] §3.4 ring buffer, §2.3 lastWindow) */
    int32_t kv_quant;     /* KVC_QUANT_NONE, KVC_QUANT_INT4 (see "4-bit rows" below),
                             KVC_QUANT_INT8_DITHER (Tier B, see
                             dither_key_lo below) or KVC_QUANT_INT8 ([WITCERT]; bf16
                             caches, contiguous with any window or a ring.  Blocks are
                             16 positions; a ring of W slots, W % 16 == 0, keeps block n
                             in block slot n mod W/16 and holds the newest W/16
                             complete blocks plus the exact rows of the incomplete
                             one, which covers its window [LEAN] §3.4) */
    int32_t batch;        /* B >= 1 requests */
    int32_t n_q_heads;    /* Hq >= 1 */
    int32_t n_kv_heads;   /* Hkv >= 1, Hq % Hkv == 0; query head h reads KV head h / (Hq/Hkv).
                             Shapes served by the generic decode (fp32 caches; bf16 with d
                             other than 64/128 or more than 8 query heads per KV head)
                             need g (d + 64) 4 <= 232448 bytes of shared memory, g = Hq/Hkv */
    int32_t head_dim;     /* d: even, 2..256; INT8 needs d % 16 == 0 */
    int32_t capacity;     /* slots per (request, KV head); INT8 needs capacity % 16 == 0 */
    int32_t window;       /* attention window W: 0 = full history (contiguous only);
                             a ring must use 0 or its capacity.  The query at
                             position t sees positions [max(0, t-W+1), t] ([LEAN] §2.1). */
    int32_t max_position; /* RoPE table length; every position must stay below it.
                             0 = capacity (contiguous).  Required for a ring with RoPE. */
    float rope_base;      /* rotary base (e.g. 10000); 0 = keys and queries not rotated */
    int32_t max_chunk;    /* largest n for kvc_chunk_attn (sizes a ring's staging rows) */
    int32_t out_dtype;    /* attention outputs: 0 = the cache dtype, else KVC_F32 or
                             KVC_BF16 (+1 is added so that 0 keeps the default):
                             pass KVC_F32 + 1 or KVC_BF16 + 1 */
    int32_t int8_exact_blocks; /* INT8 only: capacity of the pool of blocks restored
                             to full precision by kvc_int8_restore (0 = none).
                             Contiguous caches with window 0 only. */
    int32_t page_pool;    /* paged K/V storage ([LEAN] §6.1 block table; [LOOP] §八 Q1,
                             16-token pages mapped on demand): 0 = each
                             request owns `capacity` slots; > 0 = K and V live in a pool
                             of page_pool pages of 16 slots (all KV heads of one request)
                             mapped by a per-request block table, allocated on append and
                             freed by trim; capacity (the per-request logical
                             slots) must be a multiple of 16.  With INT8 a page holds
                             one quantization block of every KV head (codes, scales,
                             witnesses); the exact tail stays per request; no gate pool. */
    int32_t store_slots;  /* device slots for saved prefills (kvc_store_save /
                             kvc_store_load), each holding one request's K, V and
                             positions; 0 = none.  Not with INT8. */
    int32_t layer_index;  /* KVC_QUANT_INT8_DITHER: the layer in the dither counter */
    uint32_t dither_key_lo, dither_key_hi;
                          /* KVC_QUANT_INT8_DITHER (Tier B, [WITCERT] subtractive-
                             dither paragraph; counter from "SGLang 生产级落地与闭环门控修复"):
                             the Philox4x32-10 key.  Same shapes and limits as
                             KVC_QUANT_INT8, without witnesses: key element (token t,
                             channel c) of a block is stored as
                               code = clamp(rint(x/s + u), -127, 127), read as (code - u) s,
                             u = r/256 - 1/2 with r byte c mod 16 of the call
                               Philox4x32-10(counter = (t, c/16,
                                                       kv_head + 65536 layer_index,
                                                       request ID), key)
                             (byte i = bits 8(i mod 4) .. of word i/4); values keep the
                             plain block quantizer.  The request ID is b unless set by
                             kvc_set_request_id. */
    int32_t int8_split;   /* INT8 tiers: positions per quantized split of the decode (a
                             CTA's share of one request and KV head), a multiple of 64
                             in [1024, 2048]; 0 = 2048 when the cache (or a contiguous
                             cache's window + 32) spans 16384 slots or more, else 1024.
                             A tuning knob only: results do not depend on it beyond
                             fp32 rounding order.  Must be 0 without INT8. */
    int32_t sinks;        /* first positions that stay visible behind the window: the query at
                             position t sees [max(0, t-W+1), t] and [0, min(sinks, t+1)).  0 = none.
                             Contiguous caches with a window, all tiers but INT8 (a ring overwrites
                             its first rows); decode and prompts, not kvc_chunk_attn */
} kvc_config;

/* Bytes of the device state buffer for `cfg` (cache rows, positions,
 * next_position, RoPE table, INT8 arrays, split-K workspace).
 * Returns KVC_ERR_ARG for an invalid configuration. */
int kvc_state_bytes(const kvc_config* cfg, size_t* bytes);

/* Bind a handle to a caller-allocated device buffer of at least
 * kvc_state_bytes() bytes (256-byte aligned) on the current device.  Sets
 * every position to -1 and every next_position to 0, and uploads the RoPE
 * table; waits for `stream`.  The buffer must outlive the handle. */
int kvc_create(const kvc_config* cfg, void* d_state, size_t bytes, kvc_stream_t stream,
               kvc_t* out);

/* Release the host handle (the device buffer stays the caller's). */
int kvc_destroy(kvc_t h);

/* Append one token to every request ([LOOP] §三 step: write cache[pos];
 * [LEAN] §3.3 step).  d_k, d_v: [B][Hkv][d], keys not yet rotated.  For each
 * request: pos = next_position; the key is rotated at pos (if RoPE) and
 * rounded to the cache dtype; k, v go to slot pos (contiguous) or pos mod W
 * (ring); positions[slot] = pos; next_position = pos + 1.  INT8: the row goes
 * to the request's exact tail block; the 16th row of a block quantizes the
 * block and writes its witnesses.  KVC_ERR_CAPACITY if a contiguous cache is
 * full (nothing is written).  A captured call appends at the device's next_position; a
 * replay past the capacity or the RoPE table, or on a paged cache past the pages mapped at
 * capture, writes nothing for that request and sets the error word that
 * kvc_device_status reads. */
int kvc_append(kvc_t h, const void* d_k, const void* d_v, kvc_stream_t stream);

/* Append up to n tokens per request, in order, from d_k, d_v [B][Hkv][n][d]
 * (prefill).  h_counts (host, B entries, NULL = n for all) limits request b to
 * its first h_counts[b] rows.  Same per-row semantics as kvc_append; on a ring
 * only the rows that stay resident are written.  Replays write no row past the capacity
 * or the mapped pages either, but next_position counts every row. */
int kvc_append_rows(kvc_t h, const void* d_k, const void* d_v, int32_t n,
                    const int32_t* h_counts, kvc_stream_t stream);

/* Decode attention for the newest token of every request ([LOOP] §三 step;
 * [LEAN] §2.1).  d_q: [B][Hq][d] not yet rotated; the query sits at
 * t = next_position - 1, is rotated at t (if RoPE) in fp32, and attends to the
 * cached positions [max(0, t-W+1), t]:
 *     out = softmax(q . K^T / sqrt(d)) . V            d_out: [B][Hq][d]
 * (and to positions [0, sinks) of a cache with sinks),
 * evaluated as split-K flash decoding with an online softmax and a cross-split
 * combine, fp32 accumulation, rounded once to the output dtype.  Needs at least
 * one cached token per request; KVC_ERR_ARG too while a request of a ring lacks a key of
 * that window: a bf16 or fp32 ring that wrapped and was then trimmed (or loaded short of a
 * slot's end) has overwritten it, until the request itself appends.
 * INT8 caches also return, per (request, query head), the witness bound
 * ([WITCERT] "频带酉性与双层证书"):
 *     c_t = (1/sqrt d) sum_b ||q_b|| w_{t,b}   for every cached token in the window,
 *     d_cmax[b][h] = max_t c_t,  d_tanh[b][h] >= tanh(max_t c_t),
 * computed with upward rounding so that c_t >= |q . r_t| / sqrt(d) for the
 * stored residual r_t, hence attention total variation <= d_tanh
 * ([WITCERT] "为什么在线监控 KV 误差如此困难？").  d_ct (nullable) receives c_t
 * as [B][Hq][capacity] indexed by slot: the tokens of the window, and 0 for the
 * tokens before the window start that share its first block; other slots are not
 * written.  With a window (or a ring), max_t runs over the window only.
 * For non-quantized caches d_cmax/d_tanh (nullable) receive 0 and d_ct must
 * be NULL. */
int kvc_decode_attn(kvc_t h, const void* d_q, void* d_out, float* d_cmax, float* d_tanh,
                    float* d_ct, kvc_stream_t stream);
/* Tier B (KVC_QUANT_INT8_DITHER) caches regenerate every dither from its counter,
 * attend over the rows (code - u) s and the exact tail, and return no bound: the
 * tier's probabilistic certificate needs a per-request failure budget and a
 * concentration formula that the page does not give.  d_cmax, d_tanh and d_ct
 * must be NULL (KVC_ERR_ARG otherwise). */

/* Tier B: the request ID of request b in the dither counters, so that a
 * request's stream does not depend on its batch slot.  Only while request b holds
 * no rows (KVC_ERR_ARG otherwise, and for other tiers). */
int kvc_set_request_id(kvc_t h, int32_t b, uint32_t request_id, kvc_stream_t stream);

/* Decode attention that allocates nothing (the pages have no counterpart; this
 * is a deployment variant of kvc_decode_attn).
 *
 * Who it is for: callers that cannot call cudaMalloc while they decode. Examples:
 *   - a serving engine that reserved all device memory for its KV pool;
 *   - a runtime whose own allocator owns every device buffer;
 *   - host code that must not wait on the allocator's device synchronisation.
 *
 * What it does: the same computation and result as kvc_decode_attn (out
 * only; bf16/fp32 caches, not INT8).  The split-K partials go to a fixed
 * array of KVC_NOALLOC_SCRATCH_BYTES inside the library, not to the state
 * buffer's workspace.  The caller passes q and out; the cache is the handle's.
 *
 * The fixed array:
 *   - Every GPU that loads the library holds it until the process exits.
 *   - The first call on a device looks up the array's device address with that
 *     device current.  Make that first call before any stream capture.
 *   - Every call shares the array and overwrites it.  Each call writes every
 *     partial it reads, so nothing has to start at zero.
 *   - Calls that overlap on the GPU race on the array, even on different
 *     handles or streams: serialise them.
 *   - The looked-up address is kept for the life of the process.  A device
 *     reset (cudaDeviceReset, or the primary context torn down and made again)
 *     unloads the array, so this entry point must not be called after one.
 *
 * Errors:
 *   - KVC_ERR_CAPACITY if the problem needs more than the array holds, that is
 *     if B*Hq*splits*(8 + 4*d) bytes (+ 256 bytes of alignment) exceed
 *     KVC_NOALLOC_SCRATCH_BYTES, with
 *       splits = ceil(min(capacity, window) / split) + (page_pool > 0 ? 1 : 0)
 *                + ceil(min(sinks, max(0, capacity - window)) / split)
 *     (window 0 = capacity), where split is the decode kernel's keys per split:
 *       1024, or 2048 when min(capacity, window) >= 16384, for bf16 caches with
 *         d = 64 or 128 and 4 or 8 query heads per KV head;
 *       128 for the other bf16 caches with d = 64 or 128 and at most 8 query
 *         heads per KV head;
 *       64 otherwise.
 *   - KVC_ERR_ARG for the cases kvc_decode_attn refuses, or if the current device
 *     is not the handle's.
 *   - KVC_ERR_UNSUPPORTED for an INT8 or INT4 cache.
 * It calls no cudaMalloc, cudaFree or other allocating routine. */
#define KVC_NOALLOC_SCRATCH_BYTES (64u << 20)
/* See the comment above KVC_NOALLOC_SCRATCH_BYTES: d_q, d_out as for kvc_decode_attn. */
int kvc_decode_attn_noalloc(kvc_t h, const void* d_q, void* d_out, kvc_stream_t stream);

/* Continue every request from next_position = h_cut[b] ([PREFIX]
 * "哪些東西必須一起裁剪": keep k[:cut], v[:cut], positions[:cut]; next_position
 * = cut).  h_cut: host, B entries, 0 <= cut <= next_position.  Rows at
 * positions >= cut are dropped (positions set to -1).  A ring accepts the cut
 * only if every position the next query needs is still resident, i.e. with
 * lo = max(0, cut-W+1): lo == cut, or lo >= max(0, next_position-W) and no row that
 * an earlier trim dropped had overwritten lo; an INT8 cache only if no quantized
 * block is split (cut % 16 == 0 or cut within the exact tail).  Otherwise
 * KVC_ERR_EVICTED and nothing changes. */
int kvc_trim(kvc_t h, const int32_t* h_cut, kvc_stream_t stream);

/* Chunked causal suffix attention after a trim ([PREFIX] model.chunk(tokens[cut:],
 * cache)).  Appends n rows per request at positions cut .. cut+n-1 (as
 * kvc_append_rows) and answers every suffix query i at p = cut + i over
 * positions [max(0, p-W+1), p]:
 *     d_q [B][n][Hq][d], d_k, d_v [B][n][Hkv][d]  ->  d_out [B][n][Hq][d].
 * Row i equals what kvc_decode_attn returns for that query after appending
 * rows 0..i.  bf16 caches with head_dim 128, without INT8, INT4 or sinks: contiguous, or a ring
 * whose size W is a multiple of 16 (paged or not); n <= max_chunk.  On a ring the
 * suffix may be longer than W: appending it first would evict rows that early
 * suffix queries need ([LEAN] §3.4), so the call stages the rotated suffix rows
 * in the state buffer (sized by max_chunk), attends, and then appends them; the
 * ring ends as n one-token appends would leave it.
 * The tensor-core products take fp16 operands: the query (rotated, times
 * log2(e)/sqrt(d)), the softmax weights and the K and V rows.  Every K and V row
 * of the keys the call reads, and every scaled query, must be below 65520 in
 * magnitude (the fp16 range); otherwise bit 2 of the device error word is set and
 * the output is not valid.  Nothing else is lost: K and V values in
 * [2^-14, 65504] are exact in fp16, smaller ones keep an absolute error of at
 * most 2^-25. */
int kvc_chunk_attn(kvc_t h, const void* d_q, const void* d_k, const void* d_v, int32_t n,
                   void* d_out, kvc_stream_t stream);

/* Packed prompts ([PREFIX] model.chunk(tokens[cut:], cache) for a batch whose requests
 * have cuts and lengths of their own).  Request b brings h_counts[b] >= 0 rows (host, B
 * entries); the rows lie packed, request after request, T = the sum of the counts in all:
 *     d_q [T][Hq][d], d_k, d_v [T][Hkv][d]  ->  d_out [T][Hq][d].
 * q_stride and kv_stride are the elements from one packed row to the next (0 = dense, Hq d
 * and Hkv d), so that the three may be views of one projection's output (aligned to an
 * element where a head's row is no multiple of 16 bytes); the heads of a row are dense.
 * Appends every row as kvc_append_rows does and answers row i of request b at
 * p = next_position + i over positions [max(0, p-W+1), p], and over [0, min(sinks, p+1)) of a cache
 * with sinks.  The query is rotated in fp32 and
 * rounded to the cache's type, as the keys are; sums and softmax are fp32.  bf16 caches with
 * head_dim 64 or 128 (below 2^31 rows of all heads, at most 128 query heads a KV head) run on
 * the tensor cores, where the softmax weights are rounded to bf16 too (relative error at most
 * 2^-8 each; their sum is fp32); other shapes run on the CUDA cores in fp32 throughout, far
 * slower.  Where a call's rows fill few SMs, the keys of a row are split over several, as far
 * as the state's split-K workspace reaches: it holds the decode's partial sums, those of a
 * few rows a request.  Calls of some hundred rows behind long prefixes run unsplit.  What a
 * masked key or value row holds, infinities and NaN among it, does not reach the result.
 * d_out must not overlap the ranges that the inputs span (from their first row to their last);
 * its rows hold intermediate values during the call.
 * Rows of d_out at and after T, and requests with a count of 0, are left as they are.
 * All tiers but INT8 and INT4; a ring needs a bf16 cache with W a multiple of 16, and counts of at
 * most max_chunk (its rows are staged, as kvc_chunk_attn's are).
 * A captured call appends at the device's next_position.  A replay that passes the capacity, or
 * on a paged cache the pages mapped at capture (those of that one call), writes no row there
 * and sets the error word that kvc_device_status reads.
 * KVC_ERR_ARG: a negative count, a count above max_chunk on a ring, T > 2^31 - 1, a stride
 * below the row or of 2^38 elements, or one that is no multiple of 16 bytes where a head's
 * row is one, or an overlap.
 * KVC_ERR_CAPACITY: as kvc_append_rows; nothing is written.  KVC_ERR_UNSUPPORTED: INT8 and
 * INT4 caches, other rings, more than 65534 query heads. */
int kvc_prompt_attn(kvc_t h, const void* d_q, int64_t q_stride, const void* d_k, const void* d_v,
                    int64_t kv_stride, const int32_t* h_counts, void* d_out, kvc_stream_t stream);

/* ---- whole requests: fork, copy, free; pages: compact --------------------------
 * [LOOP] §八 Q1, [LEAN] §6.1: requests that branch from one prompt share its pages.  A
 * physical page of a paged cache may be named by the block tables of several requests.
 * Any call that is about to write rows into a shared page (append, prompt, chunk) first
 * maps a page of its own for that request and copies the rows it keeps: forked requests
 * are independent, and only what they write costs memory.  Such a call needs a free page
 * for each page it copies (KVC_ERR_CAPACITY otherwise; nothing changes); under stream
 * capture it returns KVC_ERR_UNSUPPORTED (a replay would copy again, over newer rows):
 * append once before capturing.  Replays on a ring go round to each of its pages, so there a
 * captured call is refused while a request that it brings rows for shares any page: append W
 * rows first, or branch with kvc_copy, whose pages are the branch's own.  Trim, free and the
 * store give up a request's hold on a page; the page is free when its last holder gave it up.
 * These calls keep books on the host (the lengths that kvc_next_positions reports and
 * the block table): they return KVC_ERR_UNSUPPORTED on a stream under capture, and a
 * handle whose captured calls were replayed has lengths on the device that the host does
 * not know.  On a paged cache a graph holds the page numbers of its capture: after any of
 * them (but kvc_page_counts) capture anew.  All but kvc_compact and kvc_page_counts return
 * KVC_ERR_UNSUPPORTED with more than 65534 KV heads. */

/* Requests h_dst[i] become copies of requests h_src[i] (host, n entries each, of [0, B)):
 * rows, positions, next_position and, in Tier B, the request ID (a branch draws the same
 * dithers as its source).  What the destinations held is given up.  A source may appear
 * more than once; a destination may not, nor may it be a source.  A paged cache copies no
 * rows (see above) and needs no free page; an unpaged one reads the source's rows once and
 * writes them for every destination.
 * KVC_ERR_ARG: bad index.  KVC_ERR_UNSUPPORTED: a source with blocks restored by
 * kvc_int8_restore, or stream capture. */
int kvc_fork(kvc_t h, int32_t n, const int32_t* h_src, const int32_t* h_dst, kvc_stream_t stream);

/* Requests h_dst[i] of cache `to` become copies of requests h_src[i] of cache `from`, with
 * rows of their own (on a paged cache, pages of their own).  Both caches on the current
 * device, with the same dtype, kv_quant (but for bf16 and INT4, which convert: "4-bit rows"),
 * layout, n_kv_heads, head_dim and rope_base (and, in Tier B, layer and key); paged or not, batch, query heads and, on contiguous caches,
 * capacity and window may differ; rings are of the same W.  to == from is allowed: a
 * destination must not be a source then.  The caller orders the streams of the two handles.
 * KVC_ERR_ARG: other caches or a bad index.  KVC_ERR_CAPACITY: rows beyond the capacity
 * or RoPE table of `to`, or too few free pages; nothing changes.  KVC_ERR_UNSUPPORTED: as
 * kvc_fork. */
int kvc_copy(kvc_t to, kvc_t from, int32_t n, const int32_t* h_src, const int32_t* h_dst,
             kvc_stream_t stream);

/* Empties the n distinct requests h_b: next_position 0, positions -1, every page given up
 * (a ring's too).  Other requests are untouched. */
int kvc_free(kvc_t h, int32_t n, const int32_t* h_b, kvc_stream_t stream);

/* Paged caches: moves pages so that every page in use lies below *h_used, their number:
 * the first *h_used pages of each per-page array (kvc_region) then hold everything.  No
 * more pages move than have to; requests see no change.  Free pages are taken in ascending
 * order afterwards.  KVC_ERR_UNSUPPORTED: an unpaged cache, or stream capture. */
int kvc_compact(kvc_t h, int32_t* h_used, kvc_stream_t stream);

/* Paged caches, host only: free pages, and pages that more than one request holds.
 * KVC_ERR_UNSUPPORTED: an unpaged cache. */
int kvc_page_counts(kvc_t h, int32_t* h_free, int32_t* h_shared);

/* ---- rotary positions with several axes -----------------------------------------
 * Tokens of images and video carry a position on each of several axes (time, height,
 * width), where a cache's own RoPE knows one.  With rope_base 0 a cache stores keys as
 * they are given: rotate queries and keys here, then append, decode or prompt.
 *     y[r][h] = R(angles of row r) x[r][h],    x, y [rows][heads][head_dim] of `dtype`
 * Row strides x_stride, y_stride in elements (0 = dense); heads of a row are dense.
 * d_pos: int32 [n_axes][rows], any value; 1 <= n_axes <= 8.  h_sections: host, pairs of each
 * axis in turn; their sum P <= head_dim/2, the dims from 2P on pass through.  Pair p
 * belongs to the axis a whose section it lies in, as the section's pair j, and turns by
 *     d_pos[a][r] * base^(-p/P),  with KVC_ROPE_PER_AXIS  d_pos[a][r] * base^(-j/h_sections[a]).
 * Its dims are (2p, 2p+1), with KVC_ROPE_HALVES (p, P+p).  The frequency is a double and the
 * position times it is reduced to a turn exactly, then rounded to fp32: an angle of x radians is
 * off by x 2^-51 + 1e-7 at most.  Products and sums in fp32, each rounded once, then rounded to
 * dtype.
 * d_y may be d_x (same strides); otherwise the two ranges must not overlap.  d_x and d_y
 * need the alignment of an element; 16-byte aligned rows are faster.
 * KVC_ERR_ARG: a bad size (heads * head_dim up to 2^24, rows and strides up to 2^31, head_dim
 * even and up to 256), section, flag, stride, base (positive and finite, as every frequency has
 * to be) or overlap. */
enum { KVC_ROPE_HALVES = 1, KVC_ROPE_PER_AXIS = 2 };
int kvc_rope_axes(const void* d_x, int64_t x_stride, void* d_y, int64_t y_stride, int32_t dtype,
                  int64_t rows, int32_t heads, int32_t head_dim, const int32_t* d_pos,
                  int32_t n_axes, const int32_t* h_sections, double base, int32_t flags,
                  kvc_stream_t stream);

/* ---- 4-bit rows (KVC_QUANT_INT4) ------------------------------------------------
 * A cache of bf16 inputs and outputs whose rows are quantised as they are written: 4-bit codes u
 * with a scale s and a minimum m per 32 dims of a row,
 *     m = min x,  s = bf16((max x - min x) / 15),  u = rint((x - m) / s) in 0..15,  x ~ m + u s
 * (differences and quotients in fp32, ties to even; s = 0 gives u = 0).  |x - (m + u s)| <= s / 2 for
 * s >= 2^-126; at most the group's range max x - min x for smaller s.  Keys
 * are quantised as the bf16 cache would store them, rotated and rounded.  A group of 32 that
 * holds an infinity or NaN (or spans more than fp32 holds) reads as NaN.
 * 5 bits an element: a row takes 5 d / 8 bytes, the codes (d / 2 bytes) and then the bf16 pair
 * (s, m) of each group in turn.  With G = d / 32 groups, dim 32 g + x of a K row is nibble x mod 8 of
 * 32-bit word (x / 8) G + g, of a V row nibble x mod 4 of 16-bit word (x / 4) G + g (nibble 0 the lowest
 * four bits).
 * No row depends on another: kvc_append, kvc_append_rows, kvc_trim, kvc_fork, kvc_copy, kvc_free,
 * kvc_compact and the store take this tier as they take a bf16 cache, contiguous with any window or a
 * ring, paged or not.  head_dim 64 or 128, capacity a multiple of 16, any number of query heads a KV head (at
 * most 65534 groups of 8 in all).
 * kvc_copy between a bf16 cache and one of this tier converts: rows written are quantised, rows
 * read back are m + u s, rounded once to bf16.  (A prompt runs on a bf16 cache and is handed over.)
 * kvc_decode_attn attends to the rows m + u s with fp32 sums; query and weights meet the codes in two fp16 parts
 * (relative error 2^-21 at most; of a query's dim 2^-39 of its head's largest, of a weight times its scale 2^-32 of
 * the largest in its group, where that is more); d_cmax and d_tanh receive 0 and d_ct must be NULL.
 * kvc_prompt_attn, kvc_chunk_attn and kvc_decode_attn_noalloc return KVC_ERR_UNSUPPORTED. */

/* ---- gated fallback of the INT8 tier ----------------------------------
 * [WITCERT] "SGLang 生产级落地与闭环门控修复": once the risk of a head or a block
 * crosses the water line, the lossless block is swapped in from the full-precision
 * backing store and its witness is zeroed; in the saturated zone blocks are ranked by
 * risk and truncated.  Three steps, each usable alone:
 *   kvc_int8_block_risk  (device) the risk of every complete block from a decode's c_t;
 *   kvc_int8_gate        (host)   which blocks to restore;
 *   kvc_int8_restore     (device) restore them.
 * A restored block is served exactly (bf16) from a pool inside the state buffer
 * (kvc_config.int8_exact_blocks entries); its tokens get c_t = 0 from then on.  A
 * trim that drops a restored block returns its pool entry. */

/* d_risk[b][h][k] = max over the query heads of KV head h and the 16 tokens of block
 * k of d_ct[b][hq][t] (the per-token bound of the last kvc_decode_attn on this cache,
 * [B][Hq][capacity] fp32), for every complete block of request b; 0 elsewhere.
 * d_risk: fp32 [B][Hkv][capacity/16], device.  Async on `stream`.
 * KVC_ERR_ARG: not an INT8 cache, or a null pointer.  KVC_ERR_UNSUPPORTED: Tier B,
 * a ring or a window (the gated fallback serves contiguous caches that attend to
 * their whole history). */
int kvc_int8_block_risk(kvc_t h, const float* d_ct, float* d_risk, kvc_stream_t stream);

/* Host only.  Every (request, KV head, block) of h_risk ([B][Hkv][nblk] fp32, host)
 * with tanh(risk) > tau (both in double), highest risk first, ties broken by the smaller
 * (request, head, block); at most max_blocks of them into h_sel ([max_blocks][3]
 * int32 triples); their number into *h_n_sel.  KVC_ERR_ARG: bad sizes or pointers. */
int kvc_int8_gate(const float* h_risk, int32_t B, int32_t Hkv, int32_t nblk, double tau, int32_t max_blocks,
                  int32_t* h_sel, int32_t* h_n_sel);

/* Restore the n blocks listed in h_blocks ([n][3] int32 (request, KV head, block),
 * host): copy each block's 16 rows of K and V from the full-precision backing store
 * d_k_full / d_v_full (bf16 [B][Hkv][capacity][d], device: the rows an exact cache
 * holds, keys rotated) into the pool, zero the block's witnesses, and serve its
 * tokens from the pool in every later decode.  Blocks already restored are skipped.
 * KVC_ERR_ARG: not an INT8 cache, null pointer, or a block that is not complete;
 * KVC_ERR_CAPACITY: the pool has too few free entries, or a (request, KV head) would
 * hold more than 1024 restored blocks (nothing is restored then). */
int kvc_int8_restore(kvc_t h, const int32_t* h_blocks, int32_t n, const void* d_k_full, const void* d_v_full,
                     kvc_stream_t stream);

/* Bit-exact readback of one state array for tests and debug asserts
 * ([LEAN] §6.3: export the cache and compare it with the specification).
 * Copies into h_dst (exactly kvc_export_bytes() bytes) and waits for `stream`. */
enum {
    KVC_EXPORT_K = 0,             /* [B][Hkv][capacity][d] cache dtype (non-INT8) */
    KVC_EXPORT_V = 1,
    KVC_EXPORT_POSITIONS = 2,     /* int32 [B][capacity] */
    KVC_EXPORT_NEXT_POSITION = 3, /* int32 [B] */
    KVC_EXPORT_KQ = 4,            /* int8 [B][Hkv][capacity][d] signed codes (INT8; stored
                                     biased and in the decode's block order, converted here) */
    KVC_EXPORT_VQ = 5,            /* int8 [B][Hkv][capacity][d], as KQ */
    KVC_EXPORT_SK = 6,            /* fp32 [B][Hkv][capacity/16]           (INT8) */
    KVC_EXPORT_SV = 7,
    KVC_EXPORT_WITNESS = 8,       /* fp16 [B][Hkv][capacity][16]          (INT8) */
    KVC_EXPORT_KTAIL = 9,         /* bf16 [B][Hkv][16][d] exact tail rows (INT8) */
    KVC_EXPORT_VTAIL = 10,
    KVC_EXPORT_XMAP = 11,         /* int32 [B][Hkv][capacity/16]: pool entry of a restored
                                     block, -1 = quantized (INT8) */
    KVC_EXPORT_K4 = 13,           /* [B][Hkv][capacity] rows of 5 d / 8 bytes (INT4: "4-bit rows") */
    KVC_EXPORT_V4 = 14,
    KVC_EXPORT_PAGE_TABLE = 12    /* int32 [B][capacity/16]: physical page of each logical
                                     page, -1 = none (paged caches; K, V, K4 and V4 exports are
                                     gathered through it into [B][Hkv][capacity]) */
};
/* *bytes = the size of export `which` for this handle.  KVC_ERR_ARG for a null
 * pointer or an export the cache does not hold (K/V of an INT8 or INT4 cache, INT8 arrays
 * of another, K4/V4 of any but INT4, the page table of an unpaged cache). */
int kvc_export_bytes(kvc_t h, int32_t which, size_t* bytes);
/* Copy export `which` into h_dst (host, `bytes` = kvc_export_bytes exactly, else
 * KVC_ERR_ARG), after the work already queued on `stream`; returns when the copy
 * is complete. */
int kvc_export(kvc_t h, int32_t which, void* h_dst, size_t bytes, kvc_stream_t stream);

/* Host only: where array `which` (KVC_EXPORT_*) lies inside the state buffer, as stored:
 * byte offset and size.  K and V: [B][Hkv][capacity][d], paged [page_pool][Hkv][16][d] in
 * physical page order; K4 and V4 the same with rows of 5 d / 8 bytes.  For reading on the device, ordered behind the calls that write.
 * KVC_ERR_ARG: a null pointer or an array the cache does not hold. */
int kvc_region(kvc_t h, int32_t which, size_t* offset, size_t* bytes);

/* Host mirror of next_position (B entries), kept by the handle.  Enqueued but
 * unexecuted work is already counted. */
int kvc_next_positions(kvc_t h, int32_t* h_out);

/* Waits for `stream`, then returns the device error word (0 = none; bit 0: a
 * kernel met a position outside the cache or RoPE table; bit 1: a bounded wait
 * gave up; bit 2: kvc_chunk_attn met an operand beyond the fp16 range) and
 * clears it. */
int kvc_device_status(kvc_t h, kvc_stream_t stream, int32_t* h_status);

/* Health check of the failure path: enqueues one CTA that waits, with the bounded
 * waits the kernels use for their copies (by time, and by tries in kvc_prompt_attn),
 * on a barrier that nothing signals.  Both give up after their bound (about one
 * second), bit 1 of the device error word is set and the kernel returns; nothing
 * faults and the context stays usable.  A following kvc_device_status reports the bit (and clears it). */
int kvc_check_wait_path(kvc_t h, kvc_stream_t stream);

/* Host only.  Rows of a stored prefill that a new query can reuse ([PREFIX]
 * "先看一次歷史編輯", "查詢流程與快取所有權", "為什麼滑窗部分命中必須回退"):
 * cut = length of the longest contiguous common prefix of old and new IDs,
 * at most n_new - 1 (the last query token is always recomputed).  With ring != 0
 * only a full match of the cached prefix followed by new tokens is reused
 * (cut = n_old), otherwise cut = 0.  KVC_ERR_ARG if n_new < 1, n_old < 0 or a
 * pointer is NULL where its count is positive. */
int kvc_prefix_cut(const int64_t* h_old_ids, int32_t n_old, const int64_t* h_new_ids,
                   int32_t n_new, int32_t ring, int32_t* h_cut);

/* ---- prefix store ([PREFIX] "查詢流程與快取所有權") -------------------------
 * Policy and data are split.  A kvc_pstore_t (host only, no GPU needed) decides
 * which stored prefill a query reuses and how many of its rows; the rows
 * themselves live in the store slots of a handle's state (kvc_config.store_slots)
 * and move with kvc_store_save / kvc_store_load.  A pstore slot index names the
 * handle's store slot that holds that entry's rows. */
typedef struct kvc_pstore* kvc_pstore_t;

/* Host only.  A store of at most `capacity` prefills of caches configured as
 * `cfg` ([PREFIX]: at most two).  The configuration (dtype, layout, window, head
 * shape, RoPE base) is part of every entry's computation signature; a ring
 * layout selects the sliding-window reuse rule.  KVC_ERR_ARG for capacity < 1 or
 * an invalid cfg. */
int kvc_pstore_create(const kvc_config* cfg, int32_t capacity, kvc_pstore_t* out);
/* Host only.  Frees the store (its entries' IDs, scopes and signatures); the rows
 * in the handle's store slots are untouched.  KVC_ERR_ARG for NULL. */
int kvc_pstore_destroy(kvc_pstore_t ps);

/* Host only.  Records a prefill of the n_ids >= 1 token IDs h_ids under the
 * application scope `scope` (NUL-terminated, compared byte for byte) and the
 * caller's part of the computation signature (sig_bytes bytes at h_sig, e.g. a
 * hash of the weights and of the implementation; h_sig may be NULL when
 * sig_bytes is 0).  *h_slot = the slot used: the lowest free one, else the slot
 * of the oldest entry, which is replaced (the page is silent on eviction). */
int kvc_pstore_insert(kvc_pstore_t ps, const int64_t* h_ids, int32_t n_ids, const char* scope,
                      const void* h_sig, int32_t sig_bytes, int32_t* h_slot);

/* Host only.  Lookup of a query of n_ids >= 1 token IDs, in the page's order:
 * entries with the same scope and signature are eligible; each offers the cut
 * of kvc_prefix_cut (longest contiguous common prefix, at most n_ids - 1; on a
 * ring only a whole-prefix match); the largest cut wins, ties going to the most
 * recently inserted entry.  *h_slot = that entry's slot and *h_cut its cut, or
 * -1 and 0 when no entry offers a row. */
int kvc_pstore_lookup(kvc_pstore_t ps, const int64_t* h_ids, int32_t n_ids, const char* scope,
                      const void* h_sig, int32_t sig_bytes, int32_t* h_slot, int32_t* h_cut);

/* Copies request b's cache into store slot `slot` of the state: K and V rows
 * and positions (every slot of a ring).  n must equal request b's next_position
 * (the prefill's length, n >= 1).  KVC_ERR_UNSUPPORTED without store slots. */
int kvc_store_save(kvc_t h, int32_t slot, int32_t b, int32_t n, kvc_stream_t stream);

/* Request b continues from rows [0, cut) of store slot `slot` ([PREFIX] step 4:
 * the kept K, V and positions are copied out of the store, which keeps its
 * own): the slot's rows at positions below cut are copied into request b,
 * every other slot of b is emptied, and next_position[b] = cut.  slot = -1 with
 * cut = 0 empties request b.  Other requests are untouched.  KVC_ERR_ARG if the
 * slot holds nothing or cut exceeds its length; KVC_ERR_EVICTED if a ring slot no
 * longer holds rows that the token at `cut` would attend to (the kvc_trim rule);
 * KVC_ERR_CAPACITY if a paged cache lacks pages (nothing changes).  On a ring, as
 * after kvc_trim, the request may have to append before the next decode. */
int kvc_store_load(kvc_t h, int32_t slot, int32_t b, int32_t cut, kvc_stream_t stream);

/* kvc_store_load for n requests at once (h_slots, h_b, h_cuts: host arrays of n
 * entries; the requests distinct), in one launch per 64 requests.  Every entry
 * is checked before anything changes; the statuses are those of kvc_store_load. */
int kvc_store_load_batch(kvc_t h, int32_t n, const int32_t* h_slots, const int32_t* h_b,
                         const int32_t* h_cuts, kvc_stream_t stream);

/* Static description of a status code. */
const char* kvc_strerror(int code);

#ifdef __cplusplus
}
#endif
#endif /* KVC_H */
