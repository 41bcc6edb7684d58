// Paged attention in f32, on CUDA cores: any head_dim that is a multiple of 8
// up to 256.
//
// One CTA of 8 warps per (token, query head).  Each warp walks every eighth
// block of 32 keys with an online softmax: a lane scores one key (its whole
// row against the query in shared memory), the warp takes the block's maximum
// and sum with shuffles, then the lanes turn to the depths and add p_j V[j].
// The 8 partial (m, l, O) are joined at the end in a fixed order.
//
// The plain kernel for a type that decoders rarely cache in.  Nothing is shared
// between rows or the heads of a group, so it is bound by its loads from L2 (a
// lane reads a key row by itself).  Measured on a GB300, 32 / 8 heads x 128: 8
// single tokens over 2000 keys 305 us (19 us of DRAM time), a prompt of 256
// tokens 293 us, one of 2048 11.7 ms (3 TFLOP/s).
#include <cmath>

#include "attention.h"

namespace mnb {
namespace attn {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxD = 256;
constexpr int kPer = kMaxD / 32;  // depths a lane owns

__device__ __forceinline__ float at(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }

__global__ void __launch_bounds__(kWarps * 32) attn_f32_kernel(const AttnParams p) {
    __shared__ float qs[kMaxD];
    __shared__ float os[kWarps][kMaxD];
    __shared__ float ms[kWarps], ls[kWarps];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t t = blockIdx.x / (unsigned)p.q_heads;
    const int h = (int)(blockIdx.x % (unsigned)p.q_heads), hk = h / p.group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x == 0)  // reports bad sequences, those without a new token among them
        for (int b = threadIdx.x; b < p.batch; b += kWarps * 32)
            if (bad_sequence(p, p.q_start[b], p.q_start[b + 1], p.kv_lens[b])) set_status(p.status, MNB_ERR_INVALID_ARG);
    if (t >= p.q_start[p.batch]) return;
    const int b = dec::sequence_of(p.q_start, p.batch, t);
    const int n = p.q_start[b + 1] - p.q_start[b], len = p.kv_lens[b];
    if (bad_sequence(p, p.q_start[b], p.q_start[b + 1], len)) return;
    const int i = (int)(t - p.q_start[b]);
    int lo, hi;
    visible_range(p, n, len, i, i + 1, &lo, &hi);
    for (int d = threadIdx.x; d < p.D; d += kWarps * 32) qs[d] = at(p.q, t * p.q_ts + h * p.q_hs + d) * p.scale;
    __syncthreads();

    float m = -INFINITY, l = 0.f, o[kPer] = {};
    const int ps = 1 << p.page_shift;
    for (int j0 = lo + warp * 32; j0 < hi; j0 += kWarps * 32) {
        const int j = j0 + lane;
        int64_t row = -1;
        float s = -INFINITY;
        if (j < hi) {
            const int col = j >> p.page_shift;
            const int page = col < p.table_stride ? p.tables[(int64_t)b * p.table_stride + col] : -1;
            s = 0.f;
            if ((unsigned)page < (unsigned)p.num_pages) {
                row = page * p.page_stride + (j & (ps - 1)) * p.token_stride + hk * p.head_stride;
                for (int d = 0; d < p.D; d += 4) {
                    const float4 kk = *reinterpret_cast<const float4*>(static_cast<const float*>(p.k) + row + d);
                    s = fmaf(qs[d], kk.x, s);
                    s = fmaf(qs[d + 1], kk.y, s);
                    s = fmaf(qs[d + 2], kk.z, s);
                    s = fmaf(qs[d + 3], kk.w, s);
                }
            } else {
                set_status(p.status, MNB_ERR_INVALID_ARG);
            }
        }
        float top = s;
#pragma unroll
        for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
        const float mn = fmaxf(m, top);
        const float base = mn == -INFINITY ? 0.f : mn;  // every score of the block may be -inf
        const float scale = expf(m - base), e = expf(s - base);
        float sum = e;
#pragma unroll
        for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(~0u, sum, x);
        l = l * scale + sum;
        m = mn;
#pragma unroll
        for (int c = 0; c < kPer; ++c) o[c] *= scale;
        const int cnt = min(32, hi - j0);
        for (int k = 0; k < cnt; ++k) {
            const int64_t r = __shfl_sync(~0u, row, k);
            const float w = __shfl_sync(~0u, e, k);
            if (r < 0) continue;
#pragma unroll
            for (int c = 0; c < kPer; ++c) {
                const int d = c * 32 + lane;
                if (d < p.D) o[c] = fmaf(w, at(p.v, r + d), o[c]);
            }
        }
    }
    if (lane == 0) {
        ms[warp] = m;
        ls[warp] = l;
    }
#pragma unroll
    for (int c = 0; c < kPer; ++c)
        if (c * 32 + lane < p.D) os[warp][c * 32 + lane] = o[c];
    __syncthreads();
    float top = -INFINITY;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ms[w]);
    const float base = top == -INFINITY ? 0.f : top;
    float total = 0.f;
    for (int w = 0; w < kWarps; ++w) total += ls[w] * expf(ms[w] - base);
    for (int d = threadIdx.x; d < p.D; d += kWarps * 32) {
        float a = 0.f;
        for (int w = 0; w < kWarps; ++w) a = fmaf(os[w][d], expf(ms[w] - base), a);
        static_cast<float*>(p.o)[t * p.o_ts + h * p.o_hs + d] = total == 0.f ? 0.f : a / total;  // (no key, or none above -inf)
    }
    if (threadIdx.x == 0 && p.lse) p.lse[t * p.q_heads + h] = total == 0.f ? -INFINITY : base + logf(total);
}

}  // namespace

cudaError_t launch_f32(const AttnParams& p, cudaStream_t s) {
    const int64_t blocks = p.T * p.q_heads;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks), block(kWarps * 32);
    return dec::launch_pdl(attn_f32_kernel, grid, block, 0, s, 1, p);
}

}  // namespace attn
}  // namespace mnb
