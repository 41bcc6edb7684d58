// mnb_moe_route and mnb_moe: argument checks, the routing kernel and the choice
// of the kernels in moe.cuh.
#include <algorithm>
#include <cmath>

#include "decoder.h"
#include "moe.h"
#include "moe_route.cuh"

namespace mnb {
namespace moe {
namespace {

constexpr int kRouteWarps = 4;

// mnb_moe_route: a warp a token.
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(Route r, int64_t T, int32_t* ids, float* w) {
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    griddep_wait();
    griddep_launch_dependents();
    if (t >= T) return;
    int e;
    float v;
    route_any(r, t, e, v);
    if (lane < r.S) {
        const int64_t at = t * r.S + lane;
        if (ids) ids[at] = e;
        if (w) w[at] = v;
    }
}

// Routing of mnb_moe's tokens and its lists, in one CTA: a warp a token, then one warp counts the pairs of each expert,
// 32 pairs at a time (equal ones find each other by a match), and cuts them into segments.
constexpr int kPlanThreads = 512;

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(Route r, Plan* g, int32_t* ids_out, float* w_out) {
    __shared__ int ids[kMaxPairs], place[kMaxPairs], cnt[kMaxExperts], first[kMaxExperts];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = r.S, P = r.T * S, E = r.E;
    for (int i = tid; i < E; i += kPlanThreads) cnt[i] = 0;
    griddep_wait();
    griddep_launch_dependents();
    for (int t = warp; t < r.T; t += kPlanThreads / 32) {
        int e;
        float w;
        route_any(r, t, e, w);
        if (lane < S) {
            const int at = t * S + lane;
            ids[at] = e;
            g->w[at] = w;
            if (ids_out) ids_out[at] = e;
            if (w_out) w_out[at] = w;
        }
    }
    __syncthreads();
    if (warp == 0) {
        for (int i0 = 0; i0 < P; i0 += 32) {
            const int i = i0 + lane;
            const int e = i < P ? ids[i] : -1 - lane;
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
            const int rank = __popc(same & ((1u << lane) - 1u));
            const int before = i < P ? cnt[e] : 0;
            __syncwarp();
            if (i < P) {
                place[i] = before + rank;  // among its expert's
                if (rank == 0) cnt[e] = before + __popc(same);
            }
            __syncwarp();
        }
    }
    __syncthreads();
    if (warp < 2) {
        PlanSegs& to = warp == 0 ? g->by8 : g->by4;
        const int cap = warp == 0 ? 8 : 4;
        int pairs = 0, segs = 0, most = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane, c = e < E ? cnt[e] : 0, n = (c + cap - 1) / cap;
            int fs = c, ss = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(0xFFFFFFFFu, fs, o), b = __shfl_up_sync(0xFFFFFFFFu, ss, o);
                if (lane >= o) {
                    fs += a;
                    ss += b;
                }
            }
            const int f = pairs + fs - c, s = segs + ss - n;
            for (int k = 0; k < n; ++k) to.seg[s + k] = Seg{e, f + k * cap, min(cap, c - k * cap)};
            if (warp == 0 && e < E) first[e] = f;
            most = max(most, min(cap, c));
            pairs += __shfl_sync(0xFFFFFFFFu, fs, 31);
            segs += __shfl_sync(0xFFFFFFFFu, ss, 31);
        }
        most = __reduce_max_sync(0xFFFFFFFFu, most);
        if (lane == 0) {
            to.n = segs;
            to.most = most;
        }
    }
    __syncthreads();
    for (int i = tid; i < P; i += kPlanThreads) g->sorted[first[ids[i]] + place[i]] = i;
}

mnb_status check_route(const mnb_moe_route_args* a) {
    if (!a || a->T < 0 || a->E < 1 || a->S < 1 || a->S > a->E || !dec::valid_dt(a->dtype)) return MNB_ERR_INVALID_ARG;
    if ((a->scoring != MNB_MOE_SOFTMAX && a->scoring != MNB_MOE_SIGMOID) || (a->renormalize != 0 && a->renormalize != 1) ||
        !std::isfinite(a->scale))
        return MNB_ERR_INVALID_ARG;
    if (a->bias && a->scoring != MNB_MOE_SIGMOID) return MNB_ERR_INVALID_ARG;
    if (a->T > 1 && (a->logits_stride < a->E || a->logits_stride >= (int64_t(1) << 38))) return MNB_ERR_INVALID_ARG;
    if (a->E > kMaxExperts || a->S > kMaxTopK || a->T >= (int64_t(1) << 31)) return MNB_ERR_UNSUPPORTED;
    if (a->T == 0) return MNB_OK;
    if (!a->logits || !dec::aligned_to(a->logits, dec::dt_bytes(a->dtype)) || !dec::aligned_to(a->bias, 4) ||
        !dec::aligned_to(a->ids, 4) || !dec::aligned_to(a->weights, 4))
        return MNB_ERR_INVALID_ARG;
    return MNB_OK;
}

Route make_route(const mnb_moe_route_args* a) {
    Route r{};
    r.logits = a->logits;
    r.bias = a->bias;
    r.stride = a->T > 1 ? a->logits_stride : a->E;
    r.dt = a->dtype;
    r.E = (int)a->E;
    r.S = (int)a->S;
    r.T = (int)a->T;
    r.sigmoid = a->scoring == MNB_MOE_SIGMOID;
    r.renorm = a->renormalize;
    r.scale = a->scale;
    return r;
}

bool valid_weights(const mnb_expert_weights* w, int64_t E) {
    return w && w->E == E && mnb_packed_size(w->N, w->K, w->bits, w->block_size) != 0 && dec::valid_dt(w->scale_dtype) && w->packed_b &&
           w->scales && dec::aligned_to(w->packed_b, 256) && dec::aligned_to(w->scales, dec::dt_bytes(w->scale_dtype));
}

Weights make_weights(const mnb_expert_weights* w) {
    Layout L;
    L.init(w->N, w->K, w->bits, w->block_size);
    Weights q{};
    q.packed = static_cast<const uint8_t*>(w->packed_b);
    q.scales = static_cast<const uint8_t*>(w->scales);
    q.zp = w->zero_points;
    q.expert_bytes = L.total_bytes();
    q.scale_bytes = (size_t)w->N * (size_t)L.KB * dec::dt_bytes(w->scale_dtype);
    q.zp_bytes = (size_t)w->N * (size_t)L.zp_row;
    q.row_tiles = L.NT;
    q.k_tiles = L.KTILES;
    q.N = (int)w->N;
    q.K = (int)w->K;
    q.KB = (int)L.KB;
    q.zp_row = (int)L.zp_row;
    return q;
}

size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace
}  // namespace moe
}  // namespace mnb

using namespace mnb;

extern "C" {

mnb_status mnb_moe_route(const mnb_moe_route_args* a) {
    const mnb_status st = moe::check_route(a);
    if (st != MNB_OK || a->T == 0) return st;
    if (!a->ids && !a->weights) return MNB_ERR_INVALID_ARG;
    if (inject_launch_failure()) return MNB_ERR_CUDA;
    const cudaStream_t s = (cudaStream_t)a->stream;
    ProfileScope prof("mnb_moe_route", s);
    const unsigned grid = (unsigned)((a->T + moe::kRouteWarps - 1) / moe::kRouteWarps);
    const cudaError_t e = dec::launch_pdl(moe::route_kernel, dim3(grid), dim3(32 * moe::kRouteWarps), 0, s, 1, moe::make_route(a), a->T,
                                          a->ids, a->weights);
    if (e == cudaSuccess) prof.done("moe_route");
    return dec::status_of(e);
}

size_t mnb_moe_workspace_size(int64_t T, int64_t S, int64_t E, int64_t hidden, int64_t inner) {
    if (T < 1 || T > moe::kMaxTokens || S < 1 || S > moe::kMaxTopK || T * S > moe::kMaxPairs || E < S || E > moe::kMaxExperts ||
        hidden < 1 || hidden >= (int64_t(1) << 30) || inner < 1 || inner >= (int64_t(1) << 30))
        return 0;
    const size_t pairs = (size_t)(T * S);
    // (the kernels count row tiles of segments, and their depths' chunks, in 32 bits)
    const int64_t longest = hidden > inner ? hidden : inner;
    if ((longest / 16 + 1) * T * S >= (int64_t(1) << 31)) return 0;
    return moe::round256(sizeof(moe::Plan)) + moe::round256(pairs * 4 * (((size_t)inner + 15) / 16 * 16));
}

mnb_status mnb_moe(const mnb_moe_args* a, const mnb_moe_route_args* route) {
    const mnb_status st = moe::check_route(route);
    if (st != MNB_OK) return st;
    if (!a) return MNB_ERR_INVALID_ARG;
    const mnb_expert_weights *g = a->gate, *u = a->up, *d = a->down;
    if (!moe::valid_weights(g, route->E) || !moe::valid_weights(u, route->E) || !moe::valid_weights(d, route->E)) return MNB_ERR_INVALID_ARG;
    if (g->N != u->N || g->K != u->K || d->N != g->K || d->K != g->N) return MNB_ERR_INVALID_ARG;
    if (!dec::valid_dt(a->act_dtype) || !dec::valid_dt(a->out_dtype) || (a->activation != MNB_ACT_SILU && a->activation != MNB_ACT_GELU_TANH))
        return MNB_ERR_INVALID_ARG;
    if (route->T > 1 && (a->x_stride < g->K || a->y_stride < g->K || a->x_stride >= (int64_t(1) << 38) || a->y_stride >= (int64_t(1) << 38)))
        return MNB_ERR_INVALID_ARG;
    const bool same = g->bits == u->bits && g->bits == d->bits && g->block_size == u->block_size && g->block_size == d->block_size &&
                      g->scale_dtype == u->scale_dtype && g->scale_dtype == d->scale_dtype;
    if (!same || a->act_dtype == MNB_F32 || route->T > moe::kMaxTokens || route->T * route->S > moe::kMaxPairs ||
        g->K >= (int64_t(1) << 30) || g->N >= (int64_t(1) << 30) || g->block_size > (1 << 30))
        return MNB_ERR_UNSUPPORTED;
    if (route->T == 0) return MNB_OK;
    if (!a->x || !a->y || !dec::aligned_to(a->x, 2) || !dec::aligned_to(a->y, dec::dt_bytes(a->out_dtype))) return MNB_ERR_INVALID_ARG;
    const size_t need = mnb_moe_workspace_size(route->T, route->S, route->E, g->K, g->N);
    if (need == 0) return MNB_ERR_UNSUPPORTED;
    if (!a->workspace || a->workspace_bytes < need) return MNB_ERR_NO_MEM;
    if (!dec::aligned_to(a->workspace, 256)) return MNB_ERR_INVALID_ARG;

    moe::Params p{};
    p.status = device_status_word();
    if (!p.status) return dec::status_of(cudaErrorUnknown);
    p.r = moe::make_route(route);
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    moe::Plan* plan = reinterpret_cast<moe::Plan*>(ws);
    p.h = reinterpret_cast<uint16_t*>(ws + moe::round256(sizeof(moe::Plan)));
    p.inner = (g->N + 15) / 16 * 16;
    p.x = a->x;
    p.x_stride = p.r.T > 1 ? a->x_stride : g->K;
    p.x_wide = dec::aligned_to(a->x, 16) && g->K % 8 == 0 && p.x_stride % 8 == 0;
    p.y = a->y;
    p.y_stride = p.r.T > 1 ? a->y_stride : g->K;
    p.y_dt = a->out_dtype;
    p.act = a->activation;
    p.sdt = g->scale_dtype;
    while ((1 << p.bs_shift) < g->block_size) ++p.bs_shift;
    moe::Params q = p;  // down
    p.a = moe::make_weights(g);
    p.b = moe::make_weights(u);
    q.a = q.b = moe::make_weights(d);
    if (inject_launch_failure()) return MNB_ERR_CUDA;
    const cudaStream_t s = (cudaStream_t)a->stream;
    ProfileScope prof("mnb_moe", s);
    cudaError_t e = cudaSuccess;
    if ((int64_t)p.r.T * p.r.E * p.r.E > moe::kInsideScores || p.r.T * p.r.S > moe::kInsidePairs) {
        e = dec::launch_pdl(moe::plan_kernel, dim3(1), dim3(moe::kPlanThreads), 0, s, 1, p.r, plan, route->ids, route->weights);
        p.plan = q.plan = plan;
    } else {
        p.ids_out = route->ids;
        p.w_out = route->weights;
    }
    if (e == cudaSuccess) {
        switch (g->bits) {
            case 2: e = moe::launch_b2(p, q, a->act_dtype == MNB_BF16, s); break;
            case 4: e = moe::launch_b4(p, q, a->act_dtype == MNB_BF16, s); break;
            default: e = moe::launch_b8(p, q, a->act_dtype == MNB_BF16, s); break;
        }
    }
    if (e == cudaSuccess) prof.done("moe");
    return dec::status_of(e);
}

}  // extern "C"
