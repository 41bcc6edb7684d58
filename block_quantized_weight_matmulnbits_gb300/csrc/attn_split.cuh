// Even division of a ragged batch's attention over a fixed grid: which keys of
// which rows a CTA takes.  The lengths live on the device, so every CTA works
// the division out for itself from q_start and kv_lens.
//
// A unit is one tile of kRows rows (new tokens x the heads of one key head) of
// one sequence; its visible keys are walked in tiles of kKeys.  The tiles of
// all units laid end to end are cut into equal ranges, one per CTA, so a batch
// of very different lengths keeps every SM busy to the end.  A unit inside one
// range is finished by its CTA; one that a boundary cuts leaves partial results
// (m, l, O) in the workspace, at most two per CTA (its first and its last
// piece), and a second kernel joins them in the order of the CTAs, so a result
// does not depend on timing.
#pragma once

#include "attention.h"

namespace mnb {
namespace attn {

// What a unit costs beside its tiles (its lookups, Q and exchange; its first loads fly during the exchange before it), in
// tiles: the division counts each unit that much longer, or a range of many short units would take several times as
// long as one of few long units.  256 sequences of 49 to 600 keys, 8 key heads: 78 us at 0, 58, 54, 55, 57 at 1, 2, 3, 4;
// 512 of up to 1000 keys: 162, 145, 136, 136, 139 us; 64 of up to 8192 keys: 129 us at each.
constexpr int kUnitCost = 2;

struct SplitParams {
    int ctas;        // grid of the first kernel
    int whole_tiles; // units of at most this many tiles are not cut, when each can have a CTA
    int min_tiles;   // otherwise a CTA takes at least this many tiles
    float* part_o;   // [ctas][2][rows][DP]
    float2* part_ml; // [ctas][2][rows]: maximum (log2 units) and sum
    int4* cut;       // [ctas]: the unit that the end of CTA c's range is the first to cut, for the join:
                     // first token of the sequence, first row inside it, key head + rows << 16, pieces * 2 + slot of the first
};

struct Seq {
    int n, len;    // new tokens, keys
    int lo, tiles; // first key of the first tile (a multiple of the tile), tiles of its units
    int row_tiles;
    bool bad;
};

template <int ROWS, int KEYS>
__device__ __forceinline__ Seq load_seq(const AttnParams& p, int b) {
    Seq s;
    s.n = p.q_start[b + 1] - p.q_start[b];
    s.len = p.kv_lens[b];
    s.bad = bad_sequence(p, p.q_start[b], p.q_start[b + 1], s.len);
    if (s.bad) s.n = 0;
    int lo, hi;
    visible_range(p, s.n, s.len, 0, s.n, &lo, &hi);
    s.lo = lo & ~(KEYS - 1);
    s.tiles = s.n == 0 ? 0 : hi > s.lo ? (hi - s.lo + KEYS - 1) / KEYS : 1;  // a unit without keys still writes its rows
    s.row_tiles = (s.n * p.group + ROWS - 1) / ROWS;
    return s;
}

struct Division {
    int64_t total;  // tiles (kUnitCost more for each unit), or units when whole
    int64_t ctas;   // CTAs that have work
    bool whole;     // one unit per CTA, uncut
    __device__ int64_t begin(int64_t c) const { return c >= ctas ? total : whole ? c : c * total / ctas; }
};

// Sums over the batch, by all threads of a block of THREADS.
template <int ROWS, int KEYS, int THREADS>
__device__ Division divide(const AttnParams& p, const SplitParams& sp, bool tell) {
    __shared__ int64_t sh_w[THREADS / 32], sh_u[THREADS / 32];
    __shared__ int sh_t[THREADS / 32];
    int64_t w = 0, u = 0;
    int t = 0;
    for (int b = threadIdx.x; b < p.batch; b += THREADS) {
        const Seq s = load_seq<ROWS, KEYS>(p, b);
        if (s.bad && tell) set_status(p.status, MNB_ERR_INVALID_ARG);
        const int64_t units = (int64_t)s.row_tiles * p.kv_heads;
        u += units;
        if (s.tiles) w += units * (s.tiles + kUnitCost);
        t = max(t, s.tiles);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        w += __shfl_xor_sync(~0u, w, d);
        u += __shfl_xor_sync(~0u, u, d);
        t = max(t, __shfl_xor_sync(~0u, t, d));
    }
    if ((threadIdx.x & 31) == 0) {
        sh_w[threadIdx.x >> 5] = w;
        sh_u[threadIdx.x >> 5] = u;
        sh_t[threadIdx.x >> 5] = t;
    }
    __syncthreads();
    w = u = 0;
    t = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        w += sh_w[i];
        u += sh_u[i];
        t = max(t, sh_t[i]);
    }
    Division d;
    d.whole = u <= sp.ctas && t <= sp.whole_tiles;
    d.total = d.whole ? u : w;
    const int64_t most = d.whole ? u : (w + sp.min_tiles - 1) / sp.min_tiles;
    d.ctas = most < sp.ctas ? most : sp.ctas;
    return d;
}

// A place in the division: unit (b, row tile, key head) and tile inside it.
struct Place {
    int b;
    Seq s;
    int unit;         // row tile * kv_heads + key head, inside the sequence
    int tile;
    int64_t unit_begin;  // index of the unit's first tile
};

// The place of index x, by all threads of the block; b < 0 past the last one.
// WHOLE: x is a unit, not a tile.
template <int ROWS, int KEYS, int THREADS>
__device__ Place locate(const AttnParams& p, bool whole, int64_t x, bool tell) {
    __shared__ int64_t sh_s[THREADS / 32];
    __shared__ int sh_b;
    __shared__ int64_t sh_base;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t base = 0;
    if (threadIdx.x == 0) sh_b = -1;
    for (int b0 = 0; b0 < p.batch; b0 += THREADS) {
        const int b = b0 + threadIdx.x;
        int64_t v = 0;
        if (b < p.batch) {
            const Seq s = load_seq<ROWS, KEYS>(p, b);
            if (s.bad && tell) set_status(p.status, MNB_ERR_INVALID_ARG);
            v = (int64_t)s.row_tiles * p.kv_heads * (whole ? 1 : s.tiles + kUnitCost);
            if (s.tiles == 0) v = 0;
        }
        int64_t incl = v;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int64_t y = __shfl_up_sync(~0u, incl, k);
            if (lane >= k) incl += y;
        }
        __syncthreads();
        if (lane == 31) sh_s[warp] = incl;
        __syncthreads();
        int64_t before = base, sum = 0;
        for (int i = 0; i < THREADS / 32; ++i) {
            if (i < warp) before += sh_s[i];
            sum += sh_s[i];
        }
        if (v > 0 && x >= before + incl - v && x < before + incl) {
            sh_b = b;
            sh_base = before + incl - v;
        }
        base += sum;
        if (x < base && !tell) break;  // (the block that reports bad sequences looks at all of them)
    }
    __syncthreads();
    Place pl;
    pl.b = sh_b;
    if (pl.b < 0) return pl;
    pl.s = load_seq<ROWS, KEYS>(p, pl.b);
    const int64_t r = x - sh_base;
    const int per = whole ? 1 : pl.s.tiles + kUnitCost;
    pl.unit = (int)(r / per);
    const int off = whole ? 0 : (int)(r - (int64_t)pl.unit * per) - kUnitCost;
    pl.tile = off > 0 ? off : 0;
    pl.unit_begin = x - off;
    return pl;
}

// The next unit after pl (the caller knows that there is one).
template <int ROWS, int KEYS>
__device__ __forceinline__ void next_unit(const AttnParams& p, Place& pl) {
    pl.unit_begin += pl.s.tiles + kUnitCost;
    pl.tile = 0;
    if (++pl.unit < pl.s.row_tiles * p.kv_heads) return;
    pl.unit = 0;
    do {
        ++pl.b;
        pl.s = load_seq<ROWS, KEYS>(p, pl.b);
    } while (pl.s.tiles == 0);
}

// Joins the partial results of the units that a boundary cuts: block (c, y)
// takes row y of the unit that CTA c is the first to leave unfinished.  The CTAs
// of the first kernel wrote what it needs to know.  Each of the four warps adds
// every fourth piece, eight loads ahead of their use (one warp a row, a load at a
// time, took 20 us for the 38 pieces of a single long context), and the four sums
// are added in order.
template <int DT, int DP, int ROWS>
__global__ void __launch_bounds__(128) attn_join_kernel(const AttnParams p, const SplitParams sp) {
    constexpr int W = 4, AHEAD = 8, PER = DP / 64;  // warps, pieces loaded ahead, pairs of depths a lane owns
    __shared__ float2 acc_s[W][DP / 2];
    __shared__ float l_s[W];
    griddep_wait();
    griddep_launch_dependents();
    const int c = blockIdx.x, row = blockIdx.y;
    const int4 cut = sp.cut[c];
    const int n = cut.w >> 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (n == 0 || row >= cut.z >> 16) return;
    // CTA c's piece is its last one (slot 1) unless its range begins with the unit; those after it begin inside the unit
    const int64_t at0 = (int64_t)(c * 2 + (cut.w & 1)) * ROWS + row;
    auto piece = [&](int k) { return k == 0 ? at0 : (int64_t)((c + k) * 2) * ROWS + row; };
    float m = -INFINITY;
    for (int k = lane; k < n; k += 32) m = fmaxf(m, sp.part_ml[piece(k)].x);
#pragma unroll
    for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, x));
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float2 acc[PER] = {};
    for (int k0 = warp; k0 < n; k0 += W * AHEAD) {
        float2 v[AHEAD][PER], ml[AHEAD];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const int k = k0 + a * W;
            ml[a] = make_float2(-INFINITY, 0.f);
            if (k < n) {
                const int64_t at = piece(k);
                ml[a] = sp.part_ml[at];
#pragma unroll
                for (int i = 0; i < PER; ++i) v[a][i] = *reinterpret_cast<const float2*>(sp.part_o + at * DP + i * 64 + lane * 2);
            }
        }
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            if (k0 + a * W >= n) continue;
            const float w = exp2f(ml[a].x - base);
            l = fmaf(ml[a].y, w, l);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                acc[i].x = fmaf(v[a][i].x, w, acc[i].x);
                acc[i].y = fmaf(v[a][i].y, w, acc[i].y);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) acc_s[warp][i * 32 + lane] = acc[i];
    if (lane == 0) l_s[warp] = l;
    __syncthreads();
    const int r = cut.y + row;
    const int64_t t = (int64_t)cut.x + r / p.group;
    const int h = (cut.z & 0xFFFF) * p.group + r % p.group;
    l = (l_s[0] + l_s[1]) + (l_s[2] + l_s[3]);
    const float inv = 1.f / l;
    for (int d = threadIdx.x; d * 2 < p.D; d += W * 32) {
        float2 a = acc_s[0][d];
#pragma unroll
        for (int w = 1; w < W; ++w) {
            a.x += acc_s[w][d].x;
            a.y += acc_s[w][d].y;
        }
        const int64_t o = t * p.o_ts + h * p.o_hs + d * 2;
        store_f32(p.o, o, l == 0.f ? 0.f : a.x * inv, DT);  // (without a key a may be 0 * NaN)
        store_f32(p.o, o + 1, l == 0.f ? 0.f : a.y * inv, DT);
    }
    if (threadIdx.x == 0 && p.lse) p.lse[t * p.q_heads + h] = l == 0.f ? -INFINITY : (base + log2f(l)) * kLn2;
}

}  // namespace attn
}  // namespace mnb
