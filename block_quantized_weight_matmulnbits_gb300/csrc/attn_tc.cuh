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
// boxes (a box is the part of a page that lies in the tile).
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
//   warp 8       TMEM; one thread issues all MMAs
//   warp 9       TMA
//   warp 10      zeroes V rows past the visible keys, whose pages may hold
//                anything (0 * NaN is NaN); warp 11 completes the warpgroup
// Few units (a short chunk over a long context) are cut into ranges of key
// tiles; attn_tc_join adds their (m, l, O) in order.
#pragma once

#include "attention.h"
#include "tc_ptx.cuh"

namespace mnb {
namespace attn {
namespace tca {

constexpr int kRows = 128, kKeys = 128;
constexpr int kSoftWarps = 8, kMmaWarp = 8, kTmaWarp = 9, kZeroWarp = 10, kThreads = 384;
// Registers: 384 threads start with 168 each (64512); the third warpgroup (MMA, TMA, two idle warps) gives
// 88 of each of its threads back, the softmax warpgroups take 40 more: 256 * 208 + 128 * 80 = 63488.
constexpr int kSoftRegs = 208, kCtlRegs = 80;
constexpr int kHalfBytes = 128 * 128;  // 128 rows of 64 values: one swizzled half of a Q, K or V tile

template <int DP> struct Shape {
    static constexpr int kHalves = DP / 64;
    static constexpr int kTile = kHalves * kHalfBytes;
    static constexpr int kRing = DP == 128 ? 5 : 8;
    static constexpr int kSmem = 1024 + 2 * kTile + kRing * kTile + 256;
};

struct TcParams {
    int tokens;      // new tokens of a row tile: 128 / group
    int units;       // bound on the units (grid = units * splits)
    int splits;
    float* part_o;   // [units][splits][256][DP]
    float2* part_ml; // [units][splits][256]
    int box_rows;    // rows of a K / V box: the part of a page in a tile
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}

// D[tmem] (+)= A[smem] . B[smem]^T, kind::f16, cta_group::1.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// MN-major, 128-byte swizzle: 64 values of the M / N dimension by 8 of K are a
// 1024-byte atom; atoms follow each other along K every 1024 bytes (stride
// byte offset), blocks of 64 along N every kHalfBytes (leading byte offset).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(kHalfBytes >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Bounded wait on an mbarrier phase: false when it ran out, or when another
// role of the CTA gave up.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort, const AttnParams& p) {
    if (mbar_try_wait(bar, parity)) return true;
    for (uint32_t i = 1; i < p.wait_limit; ++i) {
        const bool ok = p.wait_hint_ns == kWaitPoll ? mbar_test_wait(bar, parity)
                        : p.wait_hint_ns         ? mbar_try_wait_sleep(bar, parity, p.wait_hint_ns)
                                                 : mbar_try_wait(bar, parity);
        if (ok) return true;
        if (*abort) return false;
    }
    set_status(p.status, MNB_ERR_TIMEOUT);
    return false;
}
template <int DT>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    uint32_t d;
    if constexpr (DT == kBF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Unit `idx`: sequence, row-tile pair and key head.  The pairs of a sequence
// come last first, so that the longest ranges start first.  By one whole warp.
struct Unit {
    int b, n, len, pair, hk;
    bool ok;
};
__device__ __forceinline__ Unit find_unit(const AttnParams& p, int tokens, int64_t idx, bool tell) {
    const int lane = threadIdx.x & 31;
    Unit u{};
    int64_t base = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
        const int b = b0 + lane;
        int n = 0, len = 0;
        if (b < p.batch) {
            const int q0 = p.q_start[b], q1 = p.q_start[b + 1];
            n = q1 - q0;
            len = p.kv_lens[b];
            if (n < 0 || n > p.max_q || len < 0 || len > p.max_kv || q0 < 0 || q1 > p.T) {
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

template <int DT, int DP>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const AttnParams p, const TcParams tp,
                                                              const __grid_constant__ CUtensorMap qmap,
                                                              const __grid_constant__ CUtensorMap kmap,
                                                              const __grid_constant__ CUtensorMap vmap) {
    using S = Shape<DP>;
    constexpr int R = S::kRing;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* qs = smem;                  // [2][halves][128 rows][128 B]
    uint8_t* ring = smem + 2 * S::kTile; // [R][halves][128 rows][128 B]
    uint64_t* bars = reinterpret_cast<uint64_t*>(ring + R * S::kTile);
    uint64_t* kv_full = bars;
    uint64_t* kv_empty = bars + R;
    uint64_t* q_full = bars + 2 * R;     // [2]
    uint64_t* s_full = q_full + 2;       // [2]
    uint64_t* p_ready = s_full + 2;      // [2] one arrival per softmax warp
    uint64_t* o_full = p_ready + 2;      // [2]
    uint64_t* v_edge = o_full + 2;
    uint64_t* v_zeroed = v_edge + 1;
    uint64_t* done = v_zeroed + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
    static_assert((2 * R + 11) * 8 + 8 <= 256, "barriers fit");

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < R; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&q_full[x], 1);
            mbar_init(&s_full[x], 1);
            mbar_init(&p_ready[x], 4);
            mbar_init(&o_full[x], 1);
        }
        mbar_init(v_edge, 1);
        mbar_init(v_zeroed, 1);
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    griddep_wait();
    griddep_launch_dependents();
    const int64_t idx = blockIdx.x / (unsigned)tp.splits;
    const int split = (int)(blockIdx.x % (unsigned)tp.splits);
    const Unit u = find_unit(p, tp.tokens, idx, blockIdx.x == 0);
    if (!u.ok) return;  // the same for the block
    if (warp == kMmaWarp) tc::alloc(tmem_slot, 512);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;  // S_A | S_B | O_A | O_B, 128 columns each
    volatile int* abort_v = abort_flag;
    const Range rg = unit_range(p, tp, u, split);
    const int steps = rg.na > rg.nb ? rg.na : rg.nb;

    const int box_log = __ffs(tp.box_rows) - 1;
    // rows [z0, z1) of key tile j hold visible keys or lie in a box that was loaded for one
    auto zero_range = [&](int j, int* z0, int* z1) {
        const int kb = (rg.first + j) * kKeys;
        *z0 = rg.lo > kb ? ((rg.lo - kb) >> box_log) << box_log : 0;
        *z1 = rg.hi - kb < kKeys ? rg.hi - kb : kKeys;
        return *z0 > 0 || *z1 < kKeys;
    };
    if (warp >= kSoftWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtlRegs));
        if (warp == kTmaWarp) {
            int issued = 0;
            if (steps > 0) {
                const uint32_t q_bytes = (uint32_t)(tp.tokens * p.group * 128 * S::kHalves);
                const int tok = p.q_start[u.b] + u.pair * 2 * tp.tokens;
                if (lane == 0) {
                    for (int x = 0; x < 2; ++x) {
                        if ((x ? rg.nb : rg.na) == 0) continue;
                        mbar_arrive_expect_tx(&q_full[x], q_bytes);
                        for (int h = 0; h < S::kHalves; ++h)
                            tma_load_4d(smem_u32(qs + x * S::kTile + h * kHalfBytes), &qmap, h * 64, 0, u.hk, tok + x * tp.tokens, &q_full[x]);
                    }
                }
                const int32_t* table = p.tables + (int64_t)u.b * p.table_stride;
                const int boxes = kKeys >> box_log;
                // a lane's box of the tile (at most 16 boxes): its page is read a tile ahead
                const int box = lane / S::kHalves, half = lane % S::kHalves;
                const int ps_mask = (1 << p.page_shift) - 1;
                auto page_of = [&](int j) -> int {
                    const int key = (rg.first + j) * kKeys + (box << box_log), col = key >> p.page_shift;
                    if (j >= steps || box >= boxes || key >= rg.hi || key + tp.box_rows <= rg.lo) return -1;
                    return col < p.table_stride ? __ldg(table + col) : -1;
                };
                bool ok = true;
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
                    const uint32_t dst = smem_u32(ring) + (uint32_t)(half * kHalfBytes + (box << box_log) * 128);
                    const int row = (kb + (box << box_log)) & ps_mask;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {  // K, then V
                        const int i = 2 * j + kv, slot = i % R;
                        ok = ok && wait_for(&kv_empty[slot], (uint32_t)((i / R) & 1) ^ 1u, abort_v, p);
                        ok = __all_sync(~0u, ok);
                        if (!ok) break;
                        if (lane == 0) mbar_arrive_expect_tx(&kv_full[slot], bytes);
                        __syncwarp();
                        if (mine) tma_load_4d(dst + (uint32_t)(slot * S::kTile), kv ? &vmap : &kmap, half * 64, row, u.hk, page, &kv_full[slot]);
                        issued = i + 1;
                    }
                    page = next;
                }
                if (!ok) {
                    *abort_v = 1;
                    __syncwarp();
                    if (rg.na) tc::drain_wait(&q_full[0], 0);
                    if (rg.nb) tc::drain_wait(&q_full[1], 0);
                    for (int i = issued - R < 0 ? 0 : issued - R; i < issued; ++i)
                        tc::drain_wait(&kv_full[i % R], (uint32_t)((i / R) & 1));
                }
            }
        } else if (warp == kMmaWarp) {
            if (lane == 0 && steps > 0) {
                const uint32_t id_s = tc::idesc_f16(DT == kBF16, kRows, kKeys);
                const uint32_t id_o = tc::idesc_f16(DT == kBF16, kRows, DP) | (1u << 16);  // B is MN-major
                const uint64_t q_desc = tc::sdesc_sw128(smem_u32(qs)), k_desc = tc::sdesc_sw128(smem_u32(ring));
                const uint64_t v_desc = sdesc_mn_sw128(smem_u32(ring));
                bool ok = true;
                auto wait = [&](uint64_t* bar, uint32_t ph) {
                    ok = ok && wait_for(bar, ph, abort_v, p);
                    return ok;
                };
                auto issue_s = [&](int x, int slot) {  // S_x = Q_x . K
                    const uint64_t a = q_desc + (uint64_t)(x * (S::kTile >> 4)), b = k_desc + (uint64_t)(slot * (S::kTile >> 4));
#pragma unroll
                    for (int kk = 0; kk < DP / 16; ++kk) {
                        const uint64_t off = (uint64_t)(((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4);
                        mma_ss(tmem + (uint32_t)(x * 128), a + off, b + off, id_s, kk > 0 ? 1u : 0u);
                    }
                };
                auto issue_o = [&](int x, int slot, int step) {  // O_x += P_x . V
                    const uint64_t b = v_desc + (uint64_t)(slot * (S::kTile >> 4));
#pragma unroll
                    for (int kk = 0; kk < kKeys / 16; ++kk)
                        tc::mma_ta(tmem + 256u + (uint32_t)(x * 128), tmem + (uint32_t)(x * 128 + kk * 8), b + (uint64_t)(kk * (2048 >> 4)),
                                   id_o, (step > 0 || kk > 0) ? 1u : 0u);
                };
                wait(&kv_full[0], 0);
                for (int x = 0; x < 2 && ok; ++x) {
                    if ((x ? rg.nb : rg.na) == 0 || !wait(&q_full[x], 0)) continue;
                    tc::fence_after();
                    issue_s(x, 0);
                    tc::commit(&s_full[x]);
                }
                if (ok) tc::commit(&kv_empty[0]);
                uint32_t edges = 0;
                for (int j = 0; j < steps && ok; ++j) {
                    const int iv = 2 * j + 1, ik = iv + 1;
                    const int sv = iv % R, sk = ik % R;
                    int z0, z1;
                    if (!wait(&kv_full[sv], (uint32_t)((iv / R) & 1))) break;
                    if (zero_range(j, &z0, &z1)) {  // warp 10 clears the V rows that no row of the unit sees
                        mbar_arrive(v_edge);
                        if (!wait(v_zeroed, edges++ & 1)) break;
                    }
                    if (j + 1 < steps && !wait(&kv_full[sk], (uint32_t)((ik / R) & 1))) break;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int nx = x ? rg.nb : rg.na;
                        if (j >= nx || !wait(&p_ready[x], (uint32_t)(j & 1))) continue;
                        tc::fence_after();
                        issue_o(x, sv, j);
                        if (j + 1 < nx) {
                            issue_s(x, sk);
                            tc::commit(&s_full[x]);
                        } else {
                            tc::commit(&o_full[x]);
                        }
                    }
                    if (!ok) break;
                    tc::commit(&kv_empty[sv]);
                    if (j + 1 < steps) tc::commit(&kv_empty[sk]);
                }
                if (!ok) {
                    *abort_v = 1;
                    tc::commit(done);
                    tc::drain_wait(done, 0);
                }
            }
        } else if (warp == kZeroWarp) {
            // Rows of V past the visible keys: their pages may hold anything, and 0 * NaN is NaN.
            // The MMA thread asks for it once the tile has arrived.
            uint32_t edges = 0;
            for (int j = 0; j < steps; ++j) {
                int z0, z1;
                if (!zero_range(j, &z0, &z1)) continue;
                const int iv = 2 * j + 1;
                const bool ok = wait_for(v_edge, edges++ & 1, abort_v, p);
                if (!__all_sync(~0u, ok)) break;
                uint8_t* v = ring + (iv % R) * S::kTile;
                for (int c = lane; c < kKeys * 8; c += 32) {
                    const int r = c >> 3;
                    if (r < z0 || r >= z1) {
#pragma unroll
                        for (int h = 0; h < S::kHalves; ++h)
                            *reinterpret_cast<uint4*>(v + h * kHalfBytes + c * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(v_zeroed);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int x = warp >> 2;                 // row tile
        const int r = (warp & 3) * 32 + lane;    // row of the tile = TMEM lane
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + (uint32_t)(x * 128) + lane_addr, to = tmem + 256u + (uint32_t)(x * 128) + lane_addr;
        const int nx = x ? rg.nb : rg.na;
        const int i0 = (u.pair * 2 + x) * tp.tokens, i = i0 + r / p.group;
        const bool row_ok = r < tp.tokens * p.group && i < u.n;
        int row_lo = 0, row_hi = 0;
        if (row_ok) visible_range(p, u.n, u.len, i, i + 1, &row_lo, &row_hi);
        int full_lo, full_hi, unused;  // keys that every row of the tile sees
        {
            const int i1 = i0 + tp.tokens < u.n ? i0 + tp.tokens : u.n;
            visible_range(p, u.n, u.len, i0, i0 + 1, &unused, &full_hi);
            visible_range(p, u.n, u.len, i1 - 1, i1, &full_lo, &unused);
        }
        float m = -INFINITY;
        uint64_t l2a = pack2(0.f, 0.f), l2b = l2a;
        bool ok = true;
        for (int j = 0; j < nx; ++j) {
            ok = __all_sync(~0u, wait_for(&s_full[x], (uint32_t)(j & 1), abort_v, p));
            if (!ok) break;
            tc::fence_after();
            uint32_t s[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tc::ld_32x32b<32>(ts + (uint32_t)(c * 32), s[c]);
            tc::wait_ld();
            const int kb = (rg.first + j) * kKeys;
            if (kb < full_lo || kb + kKeys > full_hi) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const int key = kb + c * 32 + k;
                        if (key < row_lo || key >= row_hi) s[c][k] = p.scale_log2 < 0.f ? 0x7F800000u : 0xFF800000u;
                    }
            }
            // the largest of scale * s: the largest or (negative scale) smallest s
            float t[4];
            if (p.scale_log2 >= 0.f) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    t[c] = __uint_as_float(s[c][0]);
#pragma unroll
                    for (int k = 1; k < 32; ++k) t[c] = fmaxf(t[c], __uint_as_float(s[c][k]));
                }
                t[0] = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    t[c] = __uint_as_float(s[c][0]);
#pragma unroll
                    for (int k = 1; k < 32; ++k) t[c] = fminf(t[c], __uint_as_float(s[c][k]));
                }
                t[0] = fminf(fminf(t[0], t[1]), fminf(t[2], t[3]));
            }
            const float top = t[0] * p.scale_log2;
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
                        for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * f);
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
                for (int k = 0; k < 16; ++k) {
                    const float2 a = unpack2(ffma2(pack2u(s[c][2 * k], s[c][2 * k + 1]), sc2, nb2));
                    e[2 * k] = a.x;
                    e[2 * k + 1] = a.y;
                }
#pragma unroll
                for (int k = 0; k < 32; ++k) e[k] = ex2(e[k]);
                uint32_t pk[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) pk[k] = pack16<DT>(e[2 * k], e[2 * k + 1]);
                tc::st_32x32b_x16(ts + (uint32_t)(c * 16), pk);
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    if (k & 1) l2a = fadd2(l2a, pack2(e[2 * k], e[2 * k + 1]));
                    else l2b = fadd2(l2b, pack2(e[2 * k], e[2 * k + 1]));
                }
            }
            tc::wait_st();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready[x]);
        }
        const float2 la = unpack2(l2a), lb = unpack2(l2b);
        const float l = (la.x + la.y) + (lb.x + lb.y);
        bool fine = ok;
        if (fine && nx > 0) fine = wait_for(&o_full[x], 0, abort_v, p);
        fine = __all_sync(~0u, fine);
        if (!fine) *abort_v = 1;
        tc::fence_after();
        if (fine && i0 < u.n) {
            const int64_t tk = (int64_t)p.q_start[u.b] + i;
            const int h = u.hk * p.group + r % p.group;
            const int64_t part = (idx * tp.splits + split) * 256 + x * 128 + r;
            const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) {
                uint32_t v[32];
                if (nx > 0) {
                    tc::ld_32x32b<32>(to + (uint32_t)(c * 32), v);
                    tc::wait_ld();
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = 0u;
                }
                if (!row_ok) continue;
                if (tp.splits == 1) {
                    uint16_t* o = static_cast<uint16_t*>(p.o) + tk * p.o_ts + h * p.o_hs + c * 32;
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        if (c * 32 + k < p.D) {
                            uint4 w;
                            w.x = pack16<DT>(__uint_as_float(v[k]) * inv, __uint_as_float(v[k + 1]) * inv);
                            w.y = pack16<DT>(__uint_as_float(v[k + 2]) * inv, __uint_as_float(v[k + 3]) * inv);
                            w.z = pack16<DT>(__uint_as_float(v[k + 4]) * inv, __uint_as_float(v[k + 5]) * inv);
                            w.w = pack16<DT>(__uint_as_float(v[k + 6]) * inv, __uint_as_float(v[k + 7]) * inv);
                            *reinterpret_cast<uint4*>(o + k) = l > 0.f ? w : make_uint4(0, 0, 0, 0);
                        }
                    }
                } else if (nx > 0) {
                    uint4* o = reinterpret_cast<uint4*>(tp.part_o + part * DP + c * 32);
#pragma unroll
                    for (int k = 0; k < 8; ++k) o[k] = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                }
            }
            if (row_ok) {
                if (tp.splits > 1) tp.part_ml[part] = make_float2(m, l);
                else if (p.lse) p.lse[tk * p.q_heads + h] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
            }
        }
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
    float top = -INFINITY;
    for (int s = 0; s < tp.splits; ++s) top = fmaxf(top, tp.part_ml[base + s * 256].x);
    constexpr int PER = DP / 32;
    float acc[PER] = {}, l = 0.f;
    if (top > -INFINITY) {
        for (int s = 0; s < tp.splits; ++s) {
            const float2 ml = tp.part_ml[base + s * 256];
            if (ml.x == -INFINITY) continue;  // no key of the range is visible: its O may not be written
            const float w = exp2f(ml.x - top);
            l = fmaf(ml.y, w, l);
            const float* o = tp.part_o + (base + s * 256) * DP + lane * PER;
            float v[PER];
            if constexpr (PER == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(o);
            else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(o);
#pragma unroll
            for (int k = 0; k < PER; ++k) acc[k] = fmaf(v[k], w, acc[k]);
        }
    }
    const int64_t tk = (int64_t)p.q_start[u.b] + i;
    const int h = u.hk * p.group + r % p.group;
    const float inv = l > 0.f ? 1.f / l : 0.f;
    uint16_t* o = static_cast<uint16_t*>(p.o) + tk * p.o_ts + h * p.o_hs + lane * PER;
    if (lane * PER < p.D) {
        if constexpr (PER == 4) *reinterpret_cast<uint2*>(o) = make_uint2(pack16<DT>(acc[0] * inv, acc[1] * inv), pack16<DT>(acc[2] * inv, acc[3] * inv));
        else *reinterpret_cast<uint32_t*>(o) = pack16<DT>(acc[0] * inv, acc[1] * inv);
    }
    if (lane == 0 && p.lse) p.lse[tk * p.q_heads + h] = l > 0.f ? (top + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace tca
}  // namespace attn
}  // namespace mnb
