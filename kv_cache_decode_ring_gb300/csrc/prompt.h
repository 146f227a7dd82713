// prompt.h -- what the kernels of a packed prompt call share (prompt.cu, prompt_tc.cu).
#pragma once

#include "kvc_internal.h"

namespace kvc {

constexpr int kPromptGroup = 1024;        // requests per launch: their offsets ride in the parameters

// What every kernel of a call knows about its requests [b0, b0 + nb).
struct Packed {
    long long row0;                       // packed row of request b0's first row
    int b0, nb;
    int off[kPromptGroup + 1];            // request b0 + i brings rows [off[i], off[i + 1]) from row0 on
};

struct AttnArgs {
    const void* q;
    void* out;
    long long q_stride;
    const void* kc; const void* vc;       // cache rows
    const __nv_bfloat16* wk; const __nv_bfloat16* wv;   // ring staging [B][Hkv][ws_rows][d]
    const int32_t* table;
    const int32_t* next_pos;              // the cut
    const float2* rope;
    uint32_t* hdr;
    float2* part_ml;                      // split keys: {maximum (log2 domain), sum} and unnormalised sums
    float* part_acc;                      // of [packed row][Hq][part]
    int Hq, Hkv, g, d, S, W, P, ring, bf16, out_bf16, ws_rows;
    int parts;                            // 1: no split
    int sinks;                            // first positions that every row sees behind its window (0: none)
    float scale_log2;                     // log2(e) / sqrt(d)
};

// Row of the staging area that holds position p >= cut rounded down to 16.
__device__ __forceinline__ size_t stage_row(int b, int h, int p, int cut, int Hkv, int ws_rows) {
    return ((size_t)b * Hkv + h) * ws_rows + (p - (cut & ~15));
}

constexpr int kMaxKeyParts = 32;             // parts that a request's keys are split into

// The split's workspace in the state (rows of this group only: they are packed from 0 in it) as
// the attention kernels address it, by packed row, and the kernel that joins the parts.
void split_workspace(const kvc_handle* h, const Packed& g, int parts, AttnArgs* a);
cudaError_t launch_join(const AttnArgs& a, const Packed& g, cudaStream_t st);

// Tensor-core attention (prompt_tc.cu): bf16, d = 64 or 128.  `rows` of the cache (of the
// staging area) are addressed with 32-bit coordinates.
bool prompt_tc_supported(const Shape& s);
cudaError_t launch_prompt_tc(const kvc_handle* h, const AttnArgs& a, const Packed& g, cudaStream_t st);

}  // namespace kvc
