// Paged attention for many rows (chunks of a prompt, drafted tokens of wide
// groups) in bf16 / f16, head_dim up to 128: tcgen05 with TMEM accumulators.
//
// 4 D flops per (row, visible key) against 4 D bytes per key shared by the 256
// rows of a CTA: bound by the tensor pipe once a unit has a few hundred rows,
// by the cache's bytes below that.
//
// A unit is 2 x 128 rows of one sequence and key head, a row being (new token,
// query head of the group), token-major: the Q tile is one TMA box of
// [tokens][heads of the group][64 depths], so a key tile read once serves the
// whole group.  Keys come in tiles of 128, K and V through one ring of TMA
// boxes: a box is the part of a page that lies in the tile, both halves of its
// depths at once where head_dim is 128 and one tensor map can describe that.
//
//   S_X = Q_X K^T        (M 128, N 128; both operands K-major in shared memory)
//   P_X = 2^(s S_X - m)  (written as bf16 / f16 over S_X in TMEM)
//   O_X += P_X V         (A = P_X from TMEM, B = V as stored: MN-major)
//
// The two row tiles X = A, B take turns: while the tensor pipe runs O_B += P_B V
// and S_B of the next keys, the other four softmax warps work on S_A, and the
// other way round.  One thread owns one row (its TMEM lane): no shuffles.  The
// maximum a row is scaled by follows the true one only when it falls more than
// 8 (log2) behind, so O is hardly ever read back for rescaling; PV of the step
// before is complete by then, because S was committed after it.
//   warps 0-3    softmax and epilogue of row tile A
//   warps 4-7    the same for B
//   warp 8       one thread issues all MMAs
//   warp 9       TMA, and the schedule: it takes over blocks of the grid that
//                have not started (cluster launch control) and tells the others
//                what is next, so a unit's first loads and products overlap the
//                epilogue of the one before and nothing is set up twice
//   warp 10      watches the ring, so that the MMA thread polls one barrier a
//                step for it, and zeroes V rows before and past the visible keys,
//                whose pages may hold anything (0 * NaN is NaN); warp 11
//                completes the warpgroup
// Measured on a GB300: two prompts of 4096 tokens, 32 query and 8 key heads x
// 128, bf16, pages of 64: 196 us in bursts, 205 sustained (1340 TFLOP/s, the
// tensor pipe 61 % active); 500 tokens over 32000 keys: 199 us with pages of 16,
// 190 with pages of 64.  A box for each page and half took 224 and 191 us there
// (and the prompts 233 us with pages of 16): the ring waited for 32 boxes a
// step.  A step (128 keys of both row tiles) takes about 2800 cycles against
// 2048 of the tensor pipe: the chain wait, softmax (1350), P V and S (1024) of a
// row tile, and the MMA thread's polls, which take 160 to 250 cycles each.
// Few units (a short chunk over a long context) are cut into ranges of key
// tiles; attn_tc_join adds their (m, l, O) in order.
#pragma once

#include "attention.h"
#include "tc_ptx.cuh"

namespace mnb {
namespace attn {
namespace tca {

constexpr int kRows = 128, kKeys = 128;
constexpr int kSoftWarps = 8, kMmaWarp = 8, kTmaWarp = 9, kRingWarp = 10, kThreads = 384;
// Registers: 384 threads start with 168 each (64512); the third warpgroup (MMA, TMA, zeroing) gives
// 88 of each of its threads back, the softmax warpgroups take 40 more: 256 * 208 + 128 * 80 = 63488.
constexpr int kSoftRegs = 208, kCtlRegs = 80;
constexpr int kReady = 8;              // steps that may be announced ahead: more than the ring holds
constexpr int kBarBytes = 512;         // jobs and barriers
constexpr int kStageBytes = 4096;      // of one softmax warp: its 32 rows, 128 bytes at a time, on their way out
constexpr int kHalfBytes = 128 * 128;  // 128 rows of 64 values: one swizzled half of a Q, K or V tile

// ONE: a box brings both halves of its rows, as [8 rows][half] groups; otherwise a box brings one half, and the halves of
// a tile follow each other.
template <int DP, bool ONE> struct Shape {
    static constexpr int kHalves = DP / 64;
    static constexpr int kGroup = ONE ? 2048 : 1024;        // from 8 rows of a K / V tile to the next 8
    static constexpr int kHalf = ONE ? 1024 : kHalfBytes;   // from one half of a K / V tile to the other
    static constexpr int kTile = kHalves * kHalfBytes;
    static constexpr int kRing = DP == 128 ? 4 : 8;
    static constexpr int kSmem = 1024 + 2 * kTile + kRing * kTile + kSoftWarps * kStageBytes + kBarBytes;
};

struct TcParams {
    int tokens;      // new tokens of a row tile: 128 / group
    int units;       // bound on the units (grid = units * splits)
    int splits;
    float* part_o;   // [units][splits][256][DP]
    float2* part_ml; // [units][splits][256]
    int negate;      // 1: S = -Q K^T
    int box_rows;    // rows of a K / V box: the part of a page in a tile
    int64_t page_step, head_step; // ONE: steps of the box's last coordinate, and
    int head_halves; // of its coordinate of halves with the key head
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, int v, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(smem_u32(bar))
        : "memory");
}

// D[tmem] (+)= A[smem] . B[smem]^T, kind::f16, cta_group::1.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// One thread of the (converged) warp.  Code under this predicate keeps warp-
// uniform operands in uniform registers, where tcgen05.mma takes them from.
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(ok));
    return ok != 0;
}

// K, K-major with a 128-byte swizzle as tc::sdesc_sw128, its groups of 8 rows `group` bytes apart.
__device__ __forceinline__ uint64_t sdesc_k_sw128(uint32_t saddr, int group) {
    return (tc::sdesc_sw128(saddr) & ~(0x3FFFull << 32)) | (uint64_t)(group >> 4) << 32;
}
// V, MN-major, 128-byte swizzle: 64 values of the M / N dimension by 8 of K are a
// 1024-byte atom; atoms follow each other along K every `group` bytes (stride
// byte offset), blocks of 64 along N every `half` bytes (leading byte offset).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, int group, int half) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(half >> 4) << 16;
    d |= (uint64_t)(group >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Bounded waits on an mbarrier phase: false when one ran out (the role then
// records it and gives up), or when another role of the CTA gave up.  Kept to a
// few instructions: the roles share the instruction cache with the unrolled
// softmax, and the MMA thread's time is mostly instruction fetches.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort, const AttnParams& p) {
    for (uint32_t i = 0; i < p.wait_limit; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
    }
    return false;
}
// Polling: a thread that try_wait has put to sleep was seen to wake about 300
// cycles after the arrival.  It does not look at the abort flag, not even every
// 2^16 polls (two prompts of 4096: 209 -> 222 us): when another role has given
// up no MMA streams, and 2^26 polls end within 2.1 s.
__device__ __forceinline__ bool spin_for(uint64_t* bar, uint32_t parity, uint32_t limit) {
    for (uint32_t i = 0; i < limit; ++i)
        if (mbar_test_wait(bar, parity)) return true;
    return false;
}
__device__ __forceinline__ void give_up(volatile int* abort, const AttnParams& p) {
    if (!*abort) set_status(p.status, MNB_ERR_TIMEOUT);
    *abort = 1;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
template <int DT>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    uint32_t d;
    if constexpr (DT == kBF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Largest of 32 scores.
__device__ __forceinline__ float largest32(const uint32_t (&v)[32]) {
    float a = __uint_as_float(v[0]), b = __uint_as_float(v[1]);
#pragma unroll
    for (int k = 2; k < 32; k += 4) {
        a = max3(a, __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
        if (k + 3 < 32) b = max3(b, __uint_as_float(v[k + 2]), __uint_as_float(v[k + 3]));
    }
    return fmaxf(a, b);
}

// Unit `idx`: sequence, row-tile pair and key head.  The pairs of a sequence
// come last first, so that the longest ranges start first.  By one whole warp.
struct Unit {
    int b, n, len, pair, hk, tok;
    bool ok;
};
__device__ __forceinline__ Unit find_unit(const AttnParams& p, int tokens, int64_t idx, bool tell) {
    const int lane = threadIdx.x & 31;
    Unit u{};
    int64_t base = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
        const int b = b0 + lane;
        int n = 0, len = 0, q0 = 0;
        if (b < p.batch) {
            q0 = p.q_start[b];
            const int q1 = p.q_start[b + 1];
            n = q1 - q0;
            len = p.kv_lens[b];
            if (bad_sequence(p, q0, q1, len)) {
                set_status(p.status, MNB_ERR_INVALID_ARG);
                n = 0;
            }
        }
        const int64_t v = (int64_t)((n + 2 * tokens - 1) / (2 * tokens)) * p.kv_heads;
        int64_t incl = v;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int64_t y = __shfl_up_sync(~0u, incl, k);
            if (lane >= k) incl += y;
        }
        const int64_t first = base + incl - v;
        const uint32_t hit = __ballot_sync(~0u, !u.ok && v > 0 && idx >= first && idx < first + v);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const int64_t r = idx - __shfl_sync(~0u, first, src), all = __shfl_sync(~0u, v, src);
            u.b = b0 + src;
            u.n = __shfl_sync(~0u, n, src);
            u.len = __shfl_sync(~0u, len, src);
            u.tok = __shfl_sync(~0u, q0, src);
            u.pair = (int)(all / p.kv_heads - 1 - r / p.kv_heads);
            u.hk = (int)(r % p.kv_heads);
            u.ok = true;
            if (!tell) break;
        }
        base += __shfl_sync(~0u, incl, 31);
    }
    return u;
}

// Key tiles of a unit's range: [first, first + n_a) for row tile A, n_b for B.
struct Range {
    int first, na, nb;
    int lo, hi;  // visible keys of the unit
};
__device__ __forceinline__ Range unit_range(const AttnParams& p, const TcParams& tp, const Unit& u, int split) {
    Range r;
    const int a0 = u.pair * 2 * tp.tokens;
    const int a1 = a0 + tp.tokens < u.n ? a0 + tp.tokens : u.n;
    const int b1 = a1 + tp.tokens < u.n ? a1 + tp.tokens : u.n;
    int lo_a, hi_a, lo_b = 0, hi_b = 0;
    visible_range(p, u.n, u.len, a0, a1, &lo_a, &hi_a);
    if (b1 > a1) visible_range(p, u.n, u.len, a1, b1, &lo_b, &hi_b);
    r.lo = lo_a;  // rows grow, so A sees the first key of the unit and B the last
    r.hi = b1 > a1 ? hi_b : hi_a;
    const int t0 = r.lo / kKeys, t1 = r.hi > r.lo ? (r.hi + kKeys - 1) / kKeys : t0;
    const int per = (t1 - t0 + tp.splits - 1) / tp.splits;
    const int s0 = t0 + split * per;
    const int s1 = s0 + per < t1 ? s0 + per : t1;
    const int ta = hi_a > lo_a ? (hi_a + kKeys - 1) / kKeys : t0;
    r.first = s0;
    r.nb = b1 > a1 && s1 > s0 && hi_b > 0 ? s1 - s0 : 0;
    const int ea = ta < s1 ? ta : s1;
    r.na = ea > s0 ? ea - s0 : 0;
    return r;
}

// What the TMA warp tells the other roles about the CTA's next unit.
struct alignas(16) Job {
    Range rg;
    int n, len, pair, hk, tok;     // tok: first token of the sequence in the call
    int part;                      // unit * splits + split
    int valid;
};

// Cluster launch control: take over a block of the grid that has not started.
__device__ __forceinline__ void clc_try_cancel(uint32_t response, uint64_t* bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(response),
                 "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ bool clc_taken(uint32_t response, uint32_t* block) {
    uint32_t ok, x;
    asm volatile(
        "{\n .reg .b128 r;\n .reg .pred p;\n ld.shared.b128 r, [%2];\n mov.u32 %1, 0;\n"
        " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n selp.u32 %0, 1, 0, p;\n"
        " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}"
        : "=r"(ok), "=r"(x)
        : "r"(response)
        : "memory");
    *block = x;
    return ok != 0;
}

// Shared memory: Q tiles, the ring, the jobs, the barriers.
template <int DP, bool ONE>
struct Shared {
    using S = Shape<DP, ONE>;
    static constexpr int R = S::kRing;
    uint8_t* qs;    // [2][halves][128 rows][128 B]
    uint8_t* ring;  // [R][halves][128 rows][128 B], or (ONE) [R][16][halves][8 rows][128 B]
    uint8_t* stage; // [8 softmax warps][32 rows][128 B]
    Job* jobs;      // [2]
    uint8_t* response;
    uint64_t *kv_full, *kv_empty;                   // [R]
    uint64_t *q_full, *q_empty, *s_full;            // [2] per row tile, as those below
    uint64_t* p_full;                               // one arrival per softmax warp
    uint64_t *o_full, *o_free;
    uint64_t *job_full, *job_empty;                 // [2] per slot
    uint64_t *kv_ready, *clc_bar, *done;            // kv_ready [kReady] by step
    __device__ __forceinline__ explicit Shared(uint8_t* smem) {
        qs = smem;
        ring = smem + 2 * S::kTile;
        stage = ring + R * S::kTile;
        jobs = reinterpret_cast<Job*>(stage + kSoftWarps * kStageBytes);
        response = reinterpret_cast<uint8_t*>(jobs + 2);
        kv_full = reinterpret_cast<uint64_t*>(response + 16);
        kv_empty = kv_full + R;
        q_full = kv_empty + R;
        q_empty = q_full + 2;
        s_full = q_empty + 2;
        p_full = s_full + 2;
        o_full = p_full + 2;
        o_free = o_full + 2;
        job_full = o_free + 2;
        job_empty = job_full + 2;
        kv_ready = job_empty + 2;
        clc_bar = kv_ready + kReady;
        done = clc_bar + 1;
        static_assert(2 * sizeof(Job) + 16 + (2 * R + 18 + kReady) * 8 + 8 <= kBarBytes, "barriers fit");
    }
};

// Rows [z0, z1) of key tile j hold visible keys.
__device__ __forceinline__ bool zero_range(const Range& rg, int j, int* z0, int* z1) {
    const int kb = (rg.first + j) * kKeys;
    *z0 = rg.lo > kb ? rg.lo - kb : 0;
    *z1 = rg.hi - kb < kKeys ? rg.hi - kb : kKeys;
    return *z0 > 0 || *z1 < kKeys;
}

// The thread that issues all MMAs; false when a wait ran out.
template <int DT, int DP, bool ONE>
__device__ __forceinline__ bool mma_role(const Shared<DP, ONE>& sh, const AttnParams& p, const TcParams& tp, uint32_t tmem) {
    using S = Shape<DP, ONE>;
    constexpr int R = S::kRing;
    constexpr uint64_t kTileStep = S::kTile >> 4;
    // (under a negative scale Q is negated, so that the softmax knows positive ones alone)
    const uint32_t id_s = tc::idesc_f16(DT == kBF16, kRows, kKeys) | (uint32_t)tp.negate << 13;
    const uint32_t id_o = tc::idesc_f16(DT == kBF16, kRows, DP) | (1u << 16);  // B is MN-major
    const uint64_t q_desc = tc::sdesc_sw128(smem_u32(sh.qs)), k_desc = sdesc_k_sw128(smem_u32(sh.ring), S::kGroup);
    const uint64_t v_desc = sdesc_mn_sw128(smem_u32(sh.ring), S::kGroup, S::kHalf);
    // as long as the tries of the other roles (or the call's own limit, when it is shortened)
    const uint32_t limit = p.wait_limit == kWaitTries ? kWaitPolls : p.wait_limit;
    auto issue_s = [&](int x, int slot) {  // S_x = Q_x . K
        const uint64_t a = q_desc + (uint64_t)x * kTileStep, b = k_desc + (uint64_t)slot * kTileStep;
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) {
            const uint64_t off_q = (uint64_t)(((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4);
            const uint64_t off_k = (uint64_t)(((kk >> 2) * S::kHalf + (kk & 3) * 32) >> 4);
            mma_ss(tmem + (uint32_t)(x * 128), a + off_q, b + off_k, id_s, kk > 0 ? 1u : 0u);
        }
    };
    auto issue_o = [&](int x, int slot, bool first) {  // O_x += P_x . V
        const uint64_t b = v_desc + (uint64_t)slot * kTileStep;
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
            tc::mma_ta(tmem + 256u + (uint32_t)(x * 128), tmem + (uint32_t)(x * 128 + kk * 8), b + (uint64_t)(kk * (2 * S::kGroup >> 4)), id_o,
                       (!first || kk > 0) ? 1u : 0u);
    };
    int slot = 0;  // next ring entry, and the parity of its phase
    uint32_t phase = 0, seen = 0;  // (seen: steps of all units so far)
    uint32_t cnt_a = 0, cnt_b = 0, units_a = 0, units_b = 0;  // key tiles, and units with any, so far
    for (uint32_t k = 0;; ++k) {
        const Job* job = &sh.jobs[k & 1];
        if (!spin_for(&sh.job_full[k & 1], (k >> 1) & 1u, limit)) return false;
        if (!job->valid) return true;
        const Range rg = job->rg;
        mbar_arrive(&sh.job_empty[k & 1]);
        const int steps = rg.na > rg.nb ? rg.na : rg.nb;
        if (steps == 0) continue;
        int sv = 0, sk = slot;
        if (!spin_for(&sh.kv_full[slot], phase, limit)) return false;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int nx = x ? rg.nb : rg.na;
            if (nx == 0) continue;
            if (!spin_for(&sh.q_full[x], (x ? units_b : units_a) & 1u, limit)) return false;
            tc::fence_after();
            issue_s(x, sk);
            tc::commit(&sh.s_full[x]);
            if (nx == 1) tc::commit(&sh.q_empty[x]);
        }
        tc::commit(&sh.kv_empty[sk]);
        for (int j = 0; j < steps; ++j) {
            // V of this step and K of the next: warp 10 watches for them
            if (++slot == R) {
                slot = 0;
                phase ^= 1u;
            }
            sv = slot;
            if (++slot == R) {
                slot = 0;
                phase ^= 1u;
            }
            sk = slot;
            if (!spin_for(&sh.kv_ready[seen & (kReady - 1)], (seen / kReady) & 1u, limit)) return false;
            ++seen;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int nx = x ? rg.nb : rg.na;
                uint32_t& cnt = x ? cnt_b : cnt_a;
                if (j < nx) {
                    const uint32_t un = x ? units_b : units_a;
                    if (j == 0 && un > 0 && !spin_for(&sh.o_free[x], (un - 1) & 1u, limit)) return false;
                    if (!spin_for(&sh.p_full[x], cnt & 1u, limit)) return false;
                    tc::fence_after();
                    issue_o(x, sv, j == 0);
                    ++cnt;
                    if (j + 1 < nx) {
                        issue_s(x, sk);
                        tc::commit(&sh.s_full[x]);
                        if (j + 2 == nx) tc::commit(&sh.q_empty[x]);
                    } else {
                        tc::commit(&sh.o_full[x]);
                    }
                }
            }
            tc::commit(&sh.kv_empty[sv]);
            if (j + 1 < steps) tc::commit(&sh.kv_empty[sk]);
        }
        // (slot is one past the last V: the first K of the next unit)
        units_a += rg.na > 0;
        units_b += rg.nb > 0;
    }
}

template <int DT, int DP, bool ONE>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const AttnParams p, const TcParams tp,
                                                              const __grid_constant__ CUtensorMap qmap,
                                                              const __grid_constant__ CUtensorMap kmap,
                                                              const __grid_constant__ CUtensorMap vmap) {
    using S = Shape<DP, ONE>;
    constexpr int R = S::kRing;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const Shared<DP, ONE> sh(smem);
    uint8_t* const qs = sh.qs;
    uint8_t* const ring = sh.ring;
    Job* const jobs = sh.jobs;
    uint8_t* const response = sh.response;
    uint64_t *const kv_full = sh.kv_full, *const kv_empty = sh.kv_empty, *const q_full = sh.q_full, *const q_empty = sh.q_empty;
    uint64_t *const s_full = sh.s_full, *const p_full = sh.p_full, *const o_full = sh.o_full;
    uint64_t *const o_free = sh.o_free, *const job_full = sh.job_full, *const job_empty = sh.job_empty;
    uint64_t *const kv_ready = sh.kv_ready, *const clc_bar = sh.clc_bar, *const done = sh.done;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sh.done + 1);
    int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < R; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&q_full[x], 1);
            mbar_init(&q_empty[x], 1);
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[x], 4);
            mbar_init(&o_full[x], 1);
            mbar_init(&o_free[x], 4);
            mbar_init(&job_full[x], 1);
            mbar_init(&job_empty[x], kSoftWarps + 2);
        }
        for (int i = 0; i < kReady; ++i) mbar_init(&kv_ready[i], 1);
        mbar_init(clc_bar, 1);
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) tc::alloc(tmem_slot, 512);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;  // S_A | S_B | O_A | O_B, 128 columns each
    volatile int* abort_v = abort_flag;
    griddep_wait();
    griddep_launch_dependents();

    const int box_log = __ffs(tp.box_rows) - 1;
    if (warp >= kSoftWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtlRegs));
        if (warp == kTmaWarp) {
            const uint32_t q_bytes = (uint32_t)(tp.tokens * p.group * 128 * S::kHalves);
            const int boxes = kKeys >> box_log, ps_mask = (1 << p.page_shift) - 1;
            // a lane's box of the tile (at most 16, or 16 of each half): its page is read a tile ahead
            const int box = ONE ? lane : lane / S::kHalves, half = ONE ? 0 : lane % S::kHalves;
            int i = 0, q_used[2] = {0, 0};  // ring entries, and Q tiles of each kind, issued so far
            int k = 0, asked = 0;           // jobs told, blocks asked for
            bool ok = true, more = true;
            uint32_t block = blockIdx.x, unit = 0, split = 0;
            while (ok) {
                Unit u{};
                if (more) {  // ask for the next block before working on this one
                    if (lane == 0) {
                        fence_proxy_async_smem();  // the last response has been read
                        mbar_arrive_expect_tx(clc_bar, 16);
                        clc_try_cancel(smem_u32(response), clc_bar);
                    }
                    __syncwarp();
                    ++asked;
                    // a range of all units before the next range: units that share keys read them at one time
                    unit = block % (unsigned)tp.units, split = block / (unsigned)tp.units;
                    u = find_unit(p, tp.tokens, unit, blockIdx.x == 0 && k == 0);
                }
                Range rg{};
                if (u.ok || !more) {  // (a block past the last unit only gives way to the next one)
                    if (u.ok) rg = unit_range(p, tp, u, (int)split);
                    const int slot = k & 1;
                    ok = k < 2 || __all_sync(~0u, wait_for(&job_empty[slot], (uint32_t)((k >> 1) - 1) & 1u, abort_v, p));
                    if (!ok) break;
                    if (lane == 0) {
                        Job& job = jobs[slot];
                        job.rg = rg;
                        job.n = u.n;
                        job.len = u.len;
                        job.pair = u.pair;
                        job.hk = u.hk;
                        job.tok = u.tok;
                        job.part = (int)(unit * (unsigned)tp.splits + split);
                        job.valid = u.ok ? 1 : 0;
                        mbar_arrive(&job_full[slot]);
                    }
                    __syncwarp();
                    ++k;
                    if (!more) break;
                }
                const int steps = rg.na > rg.nb ? rg.na : rg.nb;
                const int32_t* table = p.tables + (int64_t)u.b * p.table_stride;
                auto page_of = [&](int j) -> int {
                    const int key = (rg.first + j) * kKeys + (box << box_log), col = key >> p.page_shift;
                    if (j >= steps || box >= boxes || key >= rg.hi || key + tp.box_rows <= rg.lo) return -1;
                    return col < p.table_stride ? __ldg(table + col) : -1;
                };
                int page = page_of(0);
                for (int j = 0; j < steps && ok; ++j) {
                    const int next = page_of(j + 1);
                    const int kb = (rg.first + j) * kKeys;
                    const int lo = rg.lo > kb ? (rg.lo - kb) >> box_log : 0;
                    const int hi = rg.hi - kb < kKeys ? (rg.hi - kb + tp.box_rows - 1) >> box_log : boxes;
                    const bool mine = box >= lo && box < hi;
                    if (mine && (unsigned)page >= (unsigned)p.num_pages) {
                        set_status(p.status, MNB_ERR_INVALID_ARG);
                        page = p.num_pages;  // past the last page: the box is filled with zeros
                    }
                    const uint32_t bytes = (uint32_t)(((hi - lo) << box_log) * 128 * S::kHalves);
                    const uint32_t dst = smem_u32(ring) + (uint32_t)(half * S::kHalf + (box << box_log) * (S::kGroup / 8));
                    const int row = (kb + (box << box_log)) & ps_mask;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {  // K, then V
                        const int slot = i % R;
                        ok = __all_sync(~0u, wait_for(&kv_empty[slot], (uint32_t)((i / R) & 1) ^ 1u, abort_v, p));
                        if (!ok) break;
                        if (lane == 0) mbar_arrive_expect_tx(&kv_full[slot], bytes);
                        __syncwarp();
                        if (mine) {
                            const CUtensorMap* map = kv ? &vmap : &kmap;
                            const uint32_t to = dst + (uint32_t)(slot * S::kTile);
                            if constexpr (ONE) {
                                tma_load_5d(to, map, 0, 0, u.hk * tp.head_halves, row >> 3, (int)(page * tp.page_step + u.hk * tp.head_step), &kv_full[slot]);
                            } else {
                                tma_load_4d(to, map, half * 64, row, u.hk, page, &kv_full[slot]);
                            }
                        }
                        ++i;
                        if (j > 0 || kv > 0) continue;
                        // the unit's Q behind its first K: its buffers come free with the last S of the unit before
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            if ((x ? rg.nb : rg.na) == 0) continue;
                            if (q_used[x] > 0) ok = ok && __all_sync(~0u, wait_for(&q_empty[x], (uint32_t)(q_used[x] - 1) & 1u, abort_v, p));
                            if (!ok) break;
                            if (lane == 0) {
                                mbar_arrive_expect_tx(&q_full[x], q_bytes);
                                for (int h = 0; h < S::kHalves; ++h)
                                    tma_load_4d(smem_u32(qs + x * S::kTile + h * kHalfBytes), &qmap, h * 64, 0, u.hk,
                                                u.tok + (u.pair * 2 + x) * tp.tokens, &q_full[x]);
                            }
                            __syncwarp();
                            ++q_used[x];
                        }
                        if (!ok) break;
                    }
                    page = next;
                }
                if (!ok) break;
                ok = __all_sync(~0u, wait_for(clc_bar, (uint32_t)(asked - 1) & 1u, abort_v, p));
                if (!ok) break;
                more = clc_taken(smem_u32(response), &block);
                __syncwarp();
            }
            if (!ok) {
                give_up(abort_v, p);
                __syncwarp();
                tc::drain_wait(clc_bar, (uint32_t)(asked - 1) & 1u);
            }
            // every copy has landed before the CTA ends (at once, unless a role gave up)
            for (int x = 0; x < 2; ++x)
                if (q_used[x]) tc::drain_wait(&q_full[x], (uint32_t)(q_used[x] - 1) & 1u);
            for (int e = i - R < 0 ? 0 : i - R; e < i; ++e) tc::drain_wait(&kv_full[e % R], (uint32_t)((e / R) & 1));
        } else if (warp == kMmaWarp) {
            if (elect_one() && !mma_role<DT, DP, ONE>(sh, p, tp, tmem)) {
                give_up(abort_v, p);
                tc::commit(sh.done);
                tc::drain_wait(sh.done, 0);
            }
        } else if (warp == kRingWarp) {
            // Watches the ring for the MMA thread (V of a step, K of the next), and clears the V rows before and past the
            // visible keys: their pages may hold anything, and 0 * NaN is NaN.
            int e = 0;           // ring entries so far
            uint32_t told = 0;   // steps so far
            bool ok = true;
            auto full = [&](int i) { return __all_sync(~0u, wait_for(&kv_full[i % R], (uint32_t)((i / R) & 1), abort_v, p)); };
            for (int k = 0; ok; ++k) {
                const Job* job = &jobs[k & 1];
                ok = __all_sync(~0u, wait_for(&job_full[k & 1], (uint32_t)((k >> 1) & 1), abort_v, p));
                if (!ok || !job->valid) break;
                const Range rg = job->rg;
                __syncwarp();
                if (lane == 0) mbar_arrive(&job_empty[k & 1]);
                const int steps = rg.na > rg.nb ? rg.na : rg.nb;
                for (int j = 0; j < steps; ++j) {
                    const int iv = e + 2 * j + 1;
                    ok = full(iv);
                    if (!ok) break;
                    int z0, z1;
                    if (zero_range(rg, j, &z0, &z1)) {
                        uint8_t* v = ring + (iv % R) * S::kTile;
                        for (int c = lane; c < kKeys * 8; c += 32) {
                            const int r = c >> 3;
                            if (r < z0 || r >= z1) {
#pragma unroll
                                for (int h = 0; h < S::kHalves; ++h)
                                    *reinterpret_cast<uint4*>(v + h * S::kHalf + (r >> 3) * S::kGroup + (c & 63) * 16) = make_uint4(0, 0, 0, 0);
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    ok = j + 1 == steps || full(iv + 1);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive(&kv_ready[told & (kReady - 1)]);
                    ++told;
                }
                e += 2 * steps;
            }
            if (!ok) give_up(abort_v, p);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int x = warp >> 2;                 // row tile
        const int r = (warp & 3) * 32 + lane;    // row of the tile = TMEM lane
        const int r_tok = r / p.group, r_head = r - r_tok * p.group;
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + (uint32_t)(x * 128) + lane_addr, to = tmem + 256u + (uint32_t)(x * 128) + lane_addr;
        uint32_t cnt = 0, units_of = 0;          // steps, and units with any, before this one
        bool ok = true;
        for (int k = 0;; ++k) {
            // The job stays in shared memory until its epilogue is done: the key loop needs the registers.
            const Job* job = &jobs[k & 1];
            ok = __all_sync(~0u, wait_for(&job_full[k & 1], (uint32_t)((k >> 1) & 1), abort_v, p));
            if (!ok || !job->valid) break;
            const int nx = x ? job->rg.nb : job->rg.na;
            const int i0 = (job->pair * 2 + x) * tp.tokens;
            int row_lo = 0, row_hi = 0, full_lo = 0, full_hi = 0, unused;
            if (i0 < job->n) {
                const int i1 = i0 + tp.tokens < job->n ? i0 + tp.tokens : job->n;
                if (r_tok < tp.tokens && i0 + r_tok < i1) visible_range(p, job->n, job->len, i0 + r_tok, i0 + r_tok + 1, &row_lo, &row_hi);
                // keys that every row of the tile sees
                visible_range(p, job->n, job->len, i0, i0 + 1, &unused, &full_hi);
                visible_range(p, job->n, job->len, i1 - 1, i1, &full_lo, &unused);
            }
            const int kb0 = job->rg.first * kKeys;
            float m = -INFINITY;
            uint64_t l2a = pack2(0.f, 0.f), l2b = l2a;
            for (int j = 0; j < nx; ++j) {
                ok = __all_sync(~0u, wait_for(&s_full[x], (cnt + (uint32_t)j) & 1u, abort_v, p));
                if (!ok) break;
                tc::fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tc::ld_32x32b<32>(ts + (uint32_t)(c * 32), s[c]);
                tc::wait_ld();
                const int kb = kb0 + j * kKeys;
                if (kb < full_lo || kb + kKeys > full_hi) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const int key = kb + c * 32 + e;
                            if (key < row_lo || key >= row_hi) s[c][e] = 0xFF800000u;
                        }
                }
                float t[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) t[c] = largest32(s[c]);
                const float top = max3(t[0], t[1], fmaxf(t[2], t[3])) * p.scale_log2;
                if (__any_sync(~0u, top > m + 8.f)) {
                    const float mn = fmaxf(m, top);
                    const float f = mn == -INFINITY ? 1.f : ex2(m - mn);
                    m = mn;
                    const uint64_t f2 = pack2(f, f);
                    l2a = ffma2(l2a, f2, pack2(0.f, 0.f));
                    l2b = ffma2(l2b, f2, pack2(0.f, 0.f));
                    if (j > 0) {
#pragma unroll
                        for (int c = 0; c < DP / 32; ++c) {
                            uint32_t v[32];
                            tc::ld_32x32b<32>(to + (uint32_t)(c * 32), v);
                            tc::wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
                            tc::st_32x32b_x32(to + (uint32_t)(c * 32), v);
                        }
                    }
                }
                const float nb = m == -INFINITY ? 0.f : -m;
                const uint64_t sc2 = pack2(p.scale_log2, p.scale_log2), nb2 = pack2(nb, nb);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    // 32 columns at a time, one kind of operation after the other: independent
                    // instructions lie next to each other, so their latencies overlap
                    float e[32];
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        const float2 a = unpack2(ffma2(pack2u(s[c][2 * q], s[c][2 * q + 1]), sc2, nb2));
                        e[2 * q] = a.x;
                        e[2 * q + 1] = a.y;
                    }
#pragma unroll
                    for (int q = 0; q < 32; ++q) e[q] = ex2(e[q]);
                    uint32_t pk[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q) pk[q] = pack16<DT>(e[2 * q], e[2 * q + 1]);
                    tc::st_32x32b_x16(ts + (uint32_t)(c * 16), pk);
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        if (q & 1) l2a = fadd2(l2a, pack2(e[2 * q], e[2 * q + 1]));
                        else l2b = fadd2(l2b, pack2(e[2 * q], e[2 * q + 1]));
                    }
                }
                tc::wait_st();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[x]);
            }
            if (!ok) break;
            if (nx > 0) {
                ok = __all_sync(~0u, wait_for(&o_full[x], units_of & 1u, abort_v, p));
                if (!ok) break;
                tc::fence_after();
            }
            const float2 la = unpack2(l2a), lb = unpack2(l2b);
            const float l = (la.x + la.y) + (lb.x + lb.y);
            const int i = i0 + r_tok;
            const bool row_ok = r_tok < tp.tokens && i < job->n;
            const int64_t tk = (int64_t)job->tok + i;
            const int h = job->hk * p.group + r_head;
            const int64_t part = (int64_t)job->part * 256 + x * 128 + r;
            const float inv = 1.f / l;
            // O leaves through shared memory, 128 bytes of the warp's 32 rows at a time, so that eight lanes store a row's
            // whole lines.  (A thread storing its own row touches 32 lines an instruction: 7000 cycles a unit for bf16,
            // 14000 for the f32 partial results, with the tensor pipe idle.)
            const bool whole = tp.splits == 1;
            uint8_t* const row = whole ? reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(p.o) + tk * p.o_ts + h * p.o_hs)
                                       : reinterpret_cast<uint8_t*>(tp.part_o + part * DP);
            const uint32_t rows_ok = __ballot_sync(~0u, row_ok && (whole || nx > 0));
            uint8_t* const stage = sh.stage + warp * kStageBytes;
            const int depths = whole ? 64 : 32;  // in 128 bytes
            for (int c = 0; c < DP; c += depths) {
                uint32_t v[32];
                if (nx > 0) {
                    tc::ld_32x32b<32>(to + (uint32_t)c, v);
                    tc::wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0u;
                }
                if (whole) {
                    uint32_t w[32];
                    if (nx > 0) {
                        tc::ld_32x32b<32>(to + (uint32_t)c + 32u, w);
                        tc::wait_ld();
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) w[e] = 0u;
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        v[e] = pack16<DT>(__uint_as_float(v[2 * e]) * inv, __uint_as_float(v[2 * e + 1]) * inv);
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[16 + e] = pack16<DT>(__uint_as_float(w[2 * e]) * inv, __uint_as_float(w[2 * e + 1]) * inv);
                }
                if (l == 0.f) {  // without a key O may be 0 * NaN
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0u;
                }
                if (c + depths >= DP && nx > 0) {  // O may be written by the next unit
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&o_free[x]);
                }
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    *reinterpret_cast<uint4*>(stage + lane * 128 + ((q ^ (lane & 7)) << 4)) = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                __syncwarp();
                const int q = lane & 7;
#pragma unroll
                for (int it = 0; it < 8; ++it) {
                    const int rr = it * 4 + (lane >> 3);
                    const uint4 u = *reinterpret_cast<const uint4*>(stage + rr * 128 + ((q ^ (rr & 7)) << 4));
                    uint8_t* const to_row = reinterpret_cast<uint8_t*>(__shfl_sync(~0u, reinterpret_cast<unsigned long long>(row), rr));
                    if ((rows_ok >> rr & 1u) && (!whole || c + q * 8 < p.D))
                        *reinterpret_cast<uint4*>(to_row + c * (whole ? 2 : 4) + q * 16) = u;
                }
                __syncwarp();
            }
            if (row_ok) {
                if (tp.splits > 1) tp.part_ml[part] = make_float2(m, l);
                else if (p.lse) p.lse[tk * p.q_heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            }
            cnt += (uint32_t)nx;
            units_of += nx > 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(&job_empty[k & 1]);
        }
        if (!ok) give_up(abort_v, p);
    }
    tc::fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after();
        tc::dealloc(tmem, 512);
    }
}

// Joins the splits of a unit: a warp per row, eight rows a block.
template <int DT, int DP>
__global__ void __launch_bounds__(256) attn_tc_join_kernel(const AttnParams p, const TcParams tp) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t idx = blockIdx.x / 32u;
    const int row = (int)(blockIdx.x % 32u) * 8 + (int)(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const Unit u = find_unit(p, tp.tokens, idx, false);
    if (!u.ok) return;
    const int x = row >> 7, r = row & 127;
    const int i = (u.pair * 2 + x) * tp.tokens + r / p.group;
    if (r >= tp.tokens * p.group || i >= u.n) return;
    const int64_t base = idx * tp.splits * 256 + row;
    // a lane's (m, l) of split lane (at most 64: two rounds), then the splits in order
    float top = -INFINITY;
    for (int s = lane; s < tp.splits; s += 32) top = fmaxf(top, tp.part_ml[base + s * 256].x);
#pragma unroll
    for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, k));
    // (-inf: no range has a visible key, or those that have hold NaN scores alone, which a maximum passes over)
    const float ref = top == -INFINITY ? 0.f : top;
    constexpr int PER = DP / 32;
    float acc[PER] = {}, l = 0.f;
    for (int s0 = 0; s0 < tp.splits; s0 += 32) {
        const float2 ml = s0 + lane < tp.splits ? tp.part_ml[base + (s0 + lane) * 256] : make_float2(-INFINITY, 0.f);
        const float w = exp2f(ml.x - ref), wl = ml.y * w;
        const int cnt = tp.splits - s0 < 32 ? tp.splits - s0 : 32;
#pragma unroll 4
        for (int s = 0; s < cnt; ++s) {
            const float ws = __shfl_sync(~0u, w, s);
            l += __shfl_sync(~0u, wl, s);
            const float* o = tp.part_o + (base + (s0 + s) * 256) * DP + lane * PER;
            float v[PER] = {};
            if (__shfl_sync(~0u, ml.y, s) != 0.f) {  // (a range without a visible key leaves its O unwritten)
                if constexpr (PER == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(o);
                else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(o);
            }
#pragma unroll
            for (int k = 0; k < PER; ++k) acc[k] = fmaf(v[k], ws, acc[k]);
        }
    }
    const int64_t tk = (int64_t)p.q_start[u.b] + i;
    const int h = u.hk * p.group + r % p.group;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t* o = static_cast<uint16_t*>(p.o) + tk * p.o_ts + h * p.o_hs + lane * PER;
    if (lane * PER < p.D) {
        if constexpr (PER == 4) *reinterpret_cast<uint2*>(o) = make_uint2(pack16<DT>(acc[0] * inv, acc[1] * inv), pack16<DT>(acc[2] * inv, acc[3] * inv));
        else *reinterpret_cast<uint32_t*>(o) = pack16<DT>(acc[0] * inv, acc[1] * inv);
    }
    if (lane == 0 && p.lse) p.lse[tk * p.q_heads + h] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
}

}  // namespace tca
}  // namespace attn
}  // namespace mnb
