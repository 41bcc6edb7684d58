// Selection of a token's experts, by one warp or by a thread a score.
//
// The router's scores are the logits (softmax) or sigmoid(logit) + bias; the S
// largest are taken in descending order, equal ones by ascending expert, a NaN
// after everything else.  A token's weights are exp(l - max) of its experts,
// divided by the sum over its experts (renormalised) or over all of them, or
// the sigmoids, divided by their sum or not, times a scale.  An expert of logit
// -inf weighs 0; where all do, every weight is 0.  Sigmoids that are divided by
// their sum and all below exp(-60) are exp(l) to 2^-86 of themselves, and are taken
// relative to the largest, as their sum would be subnormal or 0 in 32 bits.  Where
// it is 0 in 64 bits too (logits below -745, the lowest value of a mask), so are
// the weights.
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

// (below -80 1 + exp(v) is 1, and exp(-v) soon past the range)
__device__ __forceinline__ float sigmoid(float v) {
    const bool far = v <= -80.f;
    const float e = expf(far ? v : -v);
    return far ? e : 1.f / (1.f + e);
}
constexpr float kTail = -60.f, kNone = -745.f;

// Key of expert e of logit l: what is ordered.
__device__ __forceinline__ uint32_t route_key(const Route& r, float l, int e) {
    if (r.sigmoid && r.bias) l = sigmoid(l) + __ldg(r.bias + e);
    return order_key(l);
}

// Weight of place s of a token with the given logits, whose experts are ids[0 .. S - 1].
__device__ __forceinline__ float route_weight(const Route& r, const float* logit, const int* ids, int s) {
    float top = logit[ids[0]];
    if (r.sigmoid && r.renorm)  // (a bias may have put another one first)
#pragma unroll 1
        for (int j = 1; j < r.S; ++j) top = fmaxf(top, logit[ids[j]]);
    const bool plain = r.sigmoid && !(r.renorm && top < kTail);
    const float least = r.sigmoid ? kNone : -INFINITY;
    auto score = [&](float l) {
        const bool far = !plain || l <= -80.f;
        const float e = expf(!plain ? l - top : far ? l : -l);
        return !far ? 1.f / (1.f + e) : !plain && l <= least ? 0.f : e;
    };
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
    bool plain = r.sigmoid;
    if (r.sigmoid && r.renorm) {  // (a bias may have put another one first)
        top = lane < r.S ? logit : -INFINITY;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        plain = !(top < kTail);
    }
    if (plain) {
        w = lane < r.S ? sigmoid(logit) : 0.f;
    } else {
        w = lane >= r.S || logit <= (r.sigmoid ? kNone : -INFINITY) ? 0.f : expf(logit - top);
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
