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

struct SplitParams {
    int ctas;        // grid of the first kernel
    int whole_tiles; // units of at most this many tiles are not cut, when each can have a CTA
    int min_tiles;   // otherwise a CTA takes at least this many tiles
    float* part_o;   // [ctas][2][rows][DP]
    float2* part_ml; // [ctas][2][rows]: maximum (log2 units) and sum
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
    s.bad = s.n < 0 || s.n > p.max_q || s.len < 0 || s.len > p.max_kv || p.q_start[b] < 0 || p.q_start[b + 1] > p.T;
    if (s.bad) s.n = 0;
    int lo, hi;
    visible_range(p, s.n, s.len, 0, s.n, &lo, &hi);
    s.lo = lo & ~(KEYS - 1);
    s.tiles = s.n == 0 ? 0 : hi > s.lo ? (hi - s.lo + KEYS - 1) / KEYS : 1;  // a unit without keys still writes its rows
    s.row_tiles = (s.n * p.group + ROWS - 1) / ROWS;
    return s;
}

struct Division {
    int64_t total;  // tiles, or units when whole
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
        w += units * s.tiles;
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
    int64_t unit_begin;  // index of the unit's first tile (or of the unit, when whole)
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
            v = (int64_t)s.row_tiles * p.kv_heads * (whole ? 1 : s.tiles);
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
        if (x < base) break;
    }
    __syncthreads();
    Place pl;
    pl.b = sh_b;
    if (pl.b < 0) return pl;
    pl.s = load_seq<ROWS, KEYS>(p, pl.b);
    const int64_t r = x - sh_base;
    const int per = whole ? 1 : pl.s.tiles;
    pl.unit = (int)(r / per);
    pl.tile = whole ? 0 : (int)(r - (int64_t)pl.unit * per);
    pl.unit_begin = x - pl.tile;
    return pl;
}

// The next unit after pl (the caller knows that there is one).
template <int ROWS, int KEYS>
__device__ __forceinline__ void next_unit(const AttnParams& p, const Division& d, Place& pl) {
    pl.unit_begin += d.whole ? 1 : pl.s.tiles;
    pl.tile = 0;
    if (++pl.unit < pl.s.row_tiles * p.kv_heads) return;
    pl.unit = 0;
    do {
        ++pl.b;
        pl.s = load_seq<ROWS, KEYS>(p, pl.b);
    } while (pl.s.tiles == 0);
}

// Joins the partial results of the units that a boundary cuts.  Block (c, y)
// looks at the boundary between CTA c and c + 1; if it is the first one inside
// its unit, the block joins the unit's rows [y * 4, y * 4 + 4).
template <int DT, int DP, int ROWS, int KEYS>
__global__ void __launch_bounds__(128) attn_join_kernel(const AttnParams p, const SplitParams sp) {
    griddep_wait();
    griddep_launch_dependents();
    const Division d = divide<ROWS, KEYS, 128>(p, sp, false);
    const int64_t c = blockIdx.x;
    if (d.whole || c + 1 >= d.ctas) return;
    const int64_t cut = d.begin(c + 1);
    const Place pl = locate<ROWS, KEYS, 128>(p, d.whole, cut, false);
    if (pl.tile == 0 || d.begin(c) > pl.unit_begin) return;  // no cut, or not the unit's first
    const int64_t unit_end = pl.unit_begin + pl.s.tiles;
    const int row = blockIdx.y * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int rt = pl.unit / p.kv_heads, hk = pl.unit - rt * p.kv_heads;
    const int r = rt * ROWS + row;
    if (r >= pl.s.n * p.group) return;
    // Pieces: CTAs c .. last, the last with begin(x) < unit_end.  CTA c's piece is its last one (slot 1)
    // unless it begins with the unit; the others begin inside the unit (slot 0).
    const int n = (int)((unit_end * d.ctas - 1) / d.total - c) + 1;
    const int64_t at0 = (c * 2 + (d.begin(c) == pl.unit_begin ? 0 : 1)) * ROWS + row;
    auto piece = [&](int k) { return k == 0 ? at0 : ((c + k) * 2) * ROWS + row; };
    float m = -INFINITY;
    for (int k = lane; k < n; k += 32) m = fmaxf(m, sp.part_ml[piece(k)].x);
#pragma unroll
    for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, x));
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    constexpr int PER = DP / 32;
    float acc[PER] = {};
    for (int k0 = 0; k0 < n; k0 += 32) {
        // a lane's weight of piece k0 + lane, then the pieces in order, eight loads in flight
        const float2 ml = k0 + lane < n ? sp.part_ml[piece(k0 + lane)] : make_float2(-INFINITY, 0.f);
        const float w = exp2f(ml.x - base), wl = ml.y * w;
        const int cnt = n - k0 < 32 ? n - k0 : 32;
#pragma unroll 8
        for (int k = 0; k < cnt; ++k) {
            const float wk = __shfl_sync(~0u, w, k);
            l += __shfl_sync(~0u, wl, k);
            const float* o = sp.part_o + piece(k0 + k) * DP + lane * 2;
#pragma unroll
            for (int i = 0; i < PER; i += 2) {
                const float2 v = *reinterpret_cast<const float2*>(o + i * 32);
                acc[i] = fmaf(v.x, wk, acc[i]);
                acc[i + 1] = fmaf(v.y, wk, acc[i + 1]);
            }
        }
    }
    const int64_t t = p.q_start[pl.b] + r / p.group;
    const int h = hk * p.group + r % p.group;
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int64_t ob = t * p.o_ts + h * p.o_hs;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int dd = (i / 2) * 64 + lane * 2 + (i & 1);
        if (dd < p.D) store_f32(p.o, ob + dd, acc[i] * inv, DT);
    }
    if (lane == 0 && p.lse) p.lse[t * p.q_heads + h] = l > 0.f ? (base + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace attn
}  // namespace mnb
