// A mixture-of-experts layer for a few tokens: parameters shared by the host
// side (moe.cu) and the kernels (moe.cuh, one file for each code width).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "mnb.h"
#include "mnb_internal.h"

namespace mnb {
namespace moe {

constexpr int kMaxTokens = 64, kMaxTopK = 32, kMaxPairs = 1024, kMaxExperts = 1024;
// Every CTA routes for itself up to so many comparisons (T * E^2; 64 a thread) and pairs; more are a launch of their own.
constexpr int64_t kInsideScores = 1 << 14;
constexpr int kInsidePairs = 64;

// Experts' weights, back to back as mnb_matmul_grouped takes them.
struct Weights {
    const uint8_t* packed;  // expert 0's header
    const uint8_t* scales;
    const uint8_t* zp;      // null: 2^(bits - 1)
    size_t expert_bytes, scale_bytes, zp_bytes;  // of one expert
    int64_t row_tiles, k_tiles;
    int N, K, KB, zp_row;
};

// Selection of experts from the router's logits.
struct Route {
    const void* logits;
    const float* bias;  // added to the scores for the selection alone
    int64_t stride;
    int dt, E, S, T;
    int sigmoid, renorm;
    float scale;
};

struct Seg {
    int e, first, cnt;  // expert, place of its first pair in the sorted list, pairs
};

// A routing kernel's lists: pairs sorted by expert, and segments of at most 8 (gate_up) and 4 (down) of them.
struct PlanSegs {
    int n, most;  // segments, pairs of the largest
    Seg seg[kMaxPairs];
};
struct Plan {
    float w[kMaxPairs];
    int sorted[kMaxPairs];
    PlanSegs by8, by4;
};

struct Params {
    Route r;
    const Plan* plan;       // null: route inside
    int32_t* ids_out;       // optional outputs of a kernel that routes
    float* w_out;
    const void* x;
    int64_t x_stride;
    int x_wide;             // rows of x start on 16 bytes and hold whole 16-byte vectors
    Weights a, b;           // gate and up; down is a == b
    int bs_shift, sdt, s_vec, z_vec;
    int act;
    uint16_t* h;            // bf16 [T * S][hi, lo][inner]
    int64_t inner;          // rows of h: inner size rounded up to a row tile
    void* y;
    int64_t y_stride;
    int y_dt;
    int cluster;            // CTAs that share the depths of 32 rows (down)
    int* status;
};

cudaError_t launch_b2(const Params& gate_up, const Params& down, int act_bf16, cudaStream_t s);
cudaError_t launch_b4(const Params& gate_up, const Params& down, int act_bf16, cudaStream_t s);
cudaError_t launch_b8(const Params& gate_up, const Params& down, int act_bf16, cudaStream_t s);

}  // namespace moe
}  // namespace mnb
