// Selection of a token's experts, by one warp or by a thread a score.
//
// The router's scores are the logits (softmax) or sigmoid(logit) + bias; the S
// largest are taken in descending order, equal ones by ascending expert, a NaN
// after everything else.  A token's weights are exp(l - max) of its experts,
// divided by the sum over its experts (renormalised) or over all of them, or
// the sigmoids, divided by their sum or not, times a scale.  An expert of logit
// -inf weighs 0; where all do, every weight is 0.
#pragma once

#include "moe.h"

namespace mnb {
namespace moe {

// Ascending order of floats as unsigned integers; 1 for a NaN, 0 never.
__device__ __forceinline__ uint32_t order_key(float f) {
    f += 0.f;  // -0 and 0 are equal
    const uint32_t u = __float_as_uint(f);
    return isnan(f) ? 1u : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float sigmoid(float v) { return 1.f / (1.f + expf(-v)); }

// Key of expert e of logit l: what is ordered.
__device__ __forceinline__ uint32_t route_key(const Route& r, float l, int e) {
    if (r.sigmoid && r.bias) l = sigmoid(l) + __ldg(r.bias + e);
    return order_key(l);
}

// Weight of place s of a token with the given logits, whose experts are ids[0 .. S - 1].
__device__ __forceinline__ float route_weight(const Route& r, const float* logit, const int* ids, int s) {
    const float top = logit[ids[0]];
    auto score = [&](float l) { return r.sigmoid ? sigmoid(l) : l != -INFINITY ? expf(l - top) : 0.f; };
    float w = score(logit[ids[s]]), sum = 0.f;
    if (r.renorm) {
        for (int j = 0; j < r.S; ++j) sum += score(logit[ids[j]]);
    } else if (!r.sigmoid) {
        for (int e = 0; e < r.E; ++e) sum += score(logit[e]);
    }
    if (!r.sigmoid || r.renorm) w = sum != 0.f ? __fdiv_rn(w, sum) : 0.f;
    return w * r.scale;
}

// Lane s < S gets expert s and its weight.  VPL: scores a lane holds (E <= 32 VPL).
template <int VPL>
__device__ __forceinline__ void route_token(const Route& r, int64_t t, int& expert, float& weight) {
    const int lane = threadIdx.x & 31;
    uint32_t key[VPL];
    float l[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        const int e = lane + 32 * j;
        l[j] = e < r.E ? load_f32(r.logits, t * r.stride + e, r.dt) : 0.f;
    }
    float all = 0.f, top = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        const int e = lane + 32 * j;
        key[j] = e < r.E ? route_key(r, l[j], e) : 0u;
    }
    expert = 0;
    float logit = 0.f;
    for (int s = 0; s < r.S; ++s) {
        uint32_t best = 0u;
#pragma unroll
        for (int j = 0; j < VPL; ++j) best = max(best, key[j]);
        best = __reduce_max_sync(0xFFFFFFFFu, best);
        int e = 0x7FFFFFFF;
#pragma unroll
        for (int j = VPL - 1; j >= 0; --j)
            if (key[j] == best) e = lane + 32 * j;
        e = __reduce_min_sync(0xFFFFFFFFu, e);
        float le = 0.f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            if (e == lane + 32 * j) {
                key[j] = 0u;
                le = l[j];
            }
        }
        le = __shfl_sync(0xFFFFFFFFu, le, e & 31);
        if (s == 0) top = le;
        if (lane == s) {
            expert = e;
            logit = le;
        }
    }
    float w;
    if (r.sigmoid) {
        w = lane < r.S ? sigmoid(logit) : 0.f;
    } else {
        w = lane < r.S && logit != -INFINITY ? expf(logit - top) : 0.f;
        if (!r.renorm) {
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (lane + 32 * j < r.E && l[j] != -INFINITY) all += expf(l[j] - top);
        }
    }
    float sum = r.sigmoid || r.renorm ? w : all;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (!r.sigmoid || r.renorm) w = sum != 0.f ? __fdiv_rn(w, sum) : 0.f;
    weight = w * r.scale;
}

__device__ __forceinline__ void route_any(const Route& r, int64_t t, int& expert, float& weight) {
    if (r.E <= 64) route_token<2>(r, t, expert, weight);
    else if (r.E <= 256) route_token<8>(r, t, expert, weight);
    else route_token<32>(r, t, expert, weight);
}

}  // namespace moe
}  // namespace mnb
