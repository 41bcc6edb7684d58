// Attention of new tokens over a paged cache: what its kernels share.
#pragma once

#include "decoder.h"

namespace mnb {
namespace attn {

struct AttnParams {
    const void* q;
    void* o;
    float* lse;
    const void* k;
    const void* v;
    const int32_t* tables;
    const int32_t* kv_lens;
    const int32_t* q_start;
    int64_t T, table_stride;
    int64_t q_ts, q_hs, o_ts, o_hs;                  // elements
    int64_t page_stride, token_stride, head_stride;  // elements
    int batch, q_heads, kv_heads, group;             // group = q_heads / kv_heads
    int D, page_shift, num_pages;
    int max_q, max_kv;
    int window, causal;                              // window 0: none
    float scale, scale_log2;                         // scale, scale * log2(e)
    int* status;
    void* workspace;
    size_t workspace_bytes;
    uint32_t wait_limit;  // tries without a hint
    int dtype;
};

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Keys [lo, hi) that some row of the new tokens [i0, i1) of a sequence sees
// (n new tokens, len keys); hi <= lo: none.
__host__ __device__ inline void visible_range(const AttnParams& p, int n, int len, int i0, int i1, int* lo, int* hi) {
    const int first = len - n + i0, last = len - n + i1 - 1;  // positions of the first and last row
    *hi = p.causal ? (last + 1 < len ? last + 1 : len) : len;
    *lo = p.window > 0 && first >= p.window ? first - p.window + 1 : 0;  // (first may be negative and the window 2^31 - 1)
}

// A sequence of tokens [q0, q1) and len keys that is no sequence, or exceeds the call's bounds.
__device__ inline bool bad_sequence(const AttnParams& p, int q0, int q1, int len) {
    return q0 < 0 || q1 < q0 || q1 - q0 > p.max_q || q1 > p.T || len < 0 || len > p.max_kv;
}

// Few rows a key head, bf16 / f16 (attn_mma.cuh); its workspace.
cudaError_t launch_mma(const AttnParams& p, cudaStream_t s);
size_t mma_workspace_bytes(int D);
// Many rows, bf16 / f16, head_dim up to 128 (attn_tc.cuh); cudaErrorNotSupported
// (nothing launched) where a stride or size has no tensor map.  keys: those
// that the new tokens of a sequence see, at most.
bool tc_serves(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t D, int64_t max_q, int64_t keys, int dtype);
cudaError_t launch_tc(const AttnParams& p, cudaStream_t s);
size_t tc_workspace_bytes(int64_t batch, int64_t T, int64_t q_heads, int64_t kv_heads, int64_t D, int64_t max_kv);
// f32, CUDA cores (attn_f32.cu).
cudaError_t launch_f32(const AttnParams& p, cudaStream_t s);

}  // namespace attn
}  // namespace mnb
