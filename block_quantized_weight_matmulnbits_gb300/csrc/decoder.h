// Shared by the decoder-layer operators (rotary positions, paged attention,
// cache pages): argument checks and launches with programmatic dependence.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <utility>

#include "mnb.h"
#include "mnb_internal.h"

namespace mnb {
namespace dec {

inline bool valid_dt(int d) { return d == kF32 || d == kF16 || d == kBF16; }
inline int dt_bytes(int d) { return d == kF32 ? 4 : 2; }
inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool pow2(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }
constexpr int kSms = 152;  // SMs the grids are sized for

// Launch with programmatic stream serialisation.  Every kernel of these
// operators runs griddep_wait() before its first access to memory that another
// kernel may write, so the attribute never changes a result: it lets the
// launch itself (and a kernel's address set-up) overlap the preceding kernel.
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, int cluster, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)(cluster > 1 ? cluster : 1);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<A>(args)...);
}

inline mnb_status status_of(cudaError_t e) {
    if (e == cudaSuccess) return MNB_OK;
    cudaGetLastError();  // clear a launch error so the next call starts clean
    return MNB_ERR_CUDA;
}

// The fields of a cache descriptor that every call checks.
inline bool valid_cache(const mnb_kv_cache* c) {
    if (!c || !c->k_pages || !c->v_pages || !c->tables || !c->kv_lens) return false;
    if (c->batch < 1 || c->batch >= (int64_t(1) << 31) || c->table_stride < 1 || c->table_stride >= (int64_t(1) << 31))
        return false;
    if (c->num_pages < 1 || c->num_pages >= (int64_t(1) << 31)) return false;
    if (!pow2(c->page_size) || c->page_size < 8 || c->page_size > 1024) return false;
    if (c->kv_heads < 1 || c->kv_heads > 65535 || c->head_dim < 1 || c->head_dim > 4096 || !valid_dt(c->dtype)) return false;
    const int64_t v = 16 / dt_bytes(c->dtype);
    const int64_t st[3] = {c->page_stride, c->token_stride, c->head_stride};
    for (int64_t x : st)
        if (x < 0 || x % v != 0 || x >= (int64_t(1) << 39)) return false;
    return aligned_to(c->k_pages, 16) && aligned_to(c->v_pages, 16) && aligned_to(c->tables, 4) &&
           aligned_to(c->kv_lens, 4);
}

// Sequence of token t: q_start is ascending, so the last b with q_start[b] <= t
// (and q_start[b + 1] > t).  A decode batch has one token per sequence, b == t.
__device__ __forceinline__ int sequence_of(const int32_t* q_start, int batch, int64_t t) {
    if (t < batch && q_start[t] == t && q_start[t + 1] == t + 1) return (int)t;
    int lo = 0, hi = batch;  // invariant: q_start[lo] <= t (q_start[0] == 0)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (q_start[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

}  // namespace dec
}  // namespace mnb
