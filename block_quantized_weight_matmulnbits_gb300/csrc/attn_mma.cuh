// Paged attention for few rows (decode, and any head_dim up to 256) in bf16 /
// f16: warp-level MMA with the context divided evenly over the GPU.
//
// One query row of a key head does 4 D flops for the 4 D bytes of a key and
// its value, and a group of up to 16 heads shares them, so the bound is the
// bytes of the cache and everything here serves to keep its loads in flight.
//   - A row tile is the 16 rows of one m16n8k16 MMA: new tokens x the query
//     heads of one key head, so a cached value is read once for the group.
//   - Each of a CTA's 4 warps walks its own 16 keys of every 64-key tile with
//     its own ring of cp.async stages, its own online softmax and its own O
//     accumulator: no barrier inside the walk.  The four (m, l, O) are joined
//     through shared memory when the CTA leaves a unit.
//   - 2 CTAs per SM with 3 stages of 8 KB a warp (D = 128) hold 128 KB of loads
//     in flight per SM while a third of the ring is computed on.
//   - Page numbers are read one stage ahead of the loads that need them, and a
//     unit's first loads are issued before the unit before it is joined.
// Measured on a GB300 (6800 GB/s copy): 64 sequences of 684 to 8192 keys, 8 key
// heads x 128, 4 queries each, bf16: 130 us, 6070 GB/s (the even cut; 5 us of it
// the join); 256 of 49 to 600 keys: 54 us, 4520 GB/s (63 us without the overlap
// of units); one of 131001 keys, f16: 92 us, 5860 GB/s; one of 777 keys on
// clusters of 8: 7.7 us.  Bound by DRAM in the long ones, by the chain of
// dependent loads (length, page number, keys) in the last.
// The maximum a row is scaled by follows the true one only when it falls more
// than 8 (log2) behind, so O is rarely rescaled; p then stays below 2^8, exact
// in the f32 sums and rounded once to the MMA's type for the product with V.
#pragma once

#include "attn_split.cuh"

namespace mnb {
namespace attn {
namespace mma {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kRows = 16, kKeys = kWarps * 16;

// With 64 depths a cluster's CTAs are small enough for four on an SM at half the stages: twice the clusters' width, and
// shorter walks (16 sequences of 8 tokens under a window of 1024, 4 key heads: 13.6 -> 11.7 us).  The even cut keeps two
// with deep rings (64 sequences of up to 16000 keys: 76 us, 92 with four).
template <int DP, bool CL> struct Shape {
    static constexpr int kStages = DP == 64 && !CL ? 6 : 3;
    static constexpr int kCtasPerSm = DP == 256 ? 1 : DP == 64 && CL ? 4 : 2;
    static constexpr int kHalf = 16 * DP * 2;              // K or V of a stage, bytes
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kRing = kStages * kStage;         // of one warp
    static constexpr int kRed = kRows * DP * 4;            // a CTA's joined O, for the cluster form
    static constexpr int kSmem = kWarps * kRing + kRows * DP * 2 + (kWarps + 1) * kRows * 8 + kRed;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <int DT>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (DT == kBF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int DT>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    uint32_t d;
    if constexpr (DT == kBF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16-byte chunk c of row r in a [rows][DP] 16-bit tile: the chunk index is
// xored with the row so that eight rows' equal chunks lie in eight banks groups.
template <int DP>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) { return (uint32_t)(r * DP * 2 + ((c ^ (r & 7)) << 4)); }

__device__ __forceinline__ float2 ld_peer2(const void* local, uint32_t rank) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(local)), "r"(rank));
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(remote) : "memory");
    return v;
}

// CL: few units of a moderate context.  A cluster of 2, 4 or 8 CTAs takes one
// unit, each CTA an equal range of its keys, and joins the partial results
// through distributed shared memory: no division to work out, no second kernel.
template <int DT, int DP, bool CL>
__global__ void __launch_bounds__(kThreads, Shape<DP, CL>::kCtasPerSm) attn_mma_kernel(const AttnParams p, const SplitParams sp) {
    using S = Shape<DP, CL>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* qs = smem + kWarps * S::kRing;
    float2* ml_s = reinterpret_cast<float2*>(qs + kRows * DP * 2);
    float2* ml_c = ml_s + kWarps * kRows;         // the CTA's own (m, l) and O of a row, for its cluster
    float* o_c = reinterpret_cast<float*>(ml_c + kRows);
    // A warp's O [row][DP], for the others, lies in the stage of its ring that held the unit's last tile.
    static_assert(kRows * DP * 4 == S::kStage, "a warp's partial results take a stage");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    griddep_wait();
    griddep_launch_dependents();
    Division dv{};
    int64_t x0 = blockIdx.x, x1 = 0;
    int rank = 0, peers = 1;
    if constexpr (CL) {
        rank = (int)cluster_ctarank();
        asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(peers));
        x0 = blockIdx.x / (unsigned)peers;
        x1 = x0 + 1;
        dv.whole = true;
    } else {
        dv = divide<kRows, kKeys, kThreads>(p, sp, blockIdx.x == 0);
        x0 = dv.begin(blockIdx.x);
        x1 = dv.begin((int64_t)blockIdx.x + 1);
        if (threadIdx.x == 0) sp.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
        if (x0 >= x1) return;
    }
    Place pl = locate<kRows, kKeys, kThreads>(p, dv.whole, x0, CL && x0 == 0);
    if (CL && pl.b < 0) return;  // past the last unit: the whole cluster
    if (!dv.whole && x1 <= pl.unit_begin) return;  // a range inside what a unit is counted longer

    const uint32_t ring = smem_u32(smem) + warp * S::kRing, qa = smem_u32(qs);
    const uint16_t* kp = static_cast<const uint16_t*>(p.k);
    const uint16_t* vp = static_cast<const uint16_t*>(p.v);
    const int ps_mask = (1 << p.page_shift) - 1;
    constexpr int kChunks = DP / 8;              // 16-byte chunks of a row
    constexpr int kLanes = kChunks < 32 ? kChunks : 32;
    constexpr int kRpi = 32 / kLanes;            // rows a warp-wide copy covers
    const int lrow = lane / kLanes, lchunk = lane % kLanes;
    const bool col_ok = lchunk * 8 < p.D;

    // the unit at hand
    int rt, hk, t0, t1, rows, i0, i1, lo, hi, key_w;
    int64_t tok0, head_off;
    const int32_t* table;
    int c0 = 0;  // the stage of its first tile
    auto begin_unit = [&]() {
        rt = pl.unit / p.kv_heads;
        hk = pl.unit - rt * p.kv_heads;
        t0 = CL ? (int)((int64_t)pl.s.tiles * rank / peers) : pl.tile;
        const int64_t end = x1 - pl.unit_begin;
        t1 = CL ? (int)((int64_t)pl.s.tiles * (rank + 1) / peers) : dv.whole || end >= pl.s.tiles ? pl.s.tiles : (int)end;
        rows = pl.s.n * p.group - rt * kRows < kRows ? pl.s.n * p.group - rt * kRows : kRows;
        tok0 = p.q_start[pl.b];
        i0 = rt * kRows / p.group;
        i1 = (rt * kRows + rows - 1) / p.group + 1;
        visible_range(p, pl.s.n, pl.s.len, i0, i1, &lo, &hi);  // keys that a row of the tile sees
        table = p.tables + (int64_t)pl.b * p.table_stride;
        key_w = pl.s.lo + warp * 16;
        head_off = (int64_t)hk * p.head_stride;
    };
    auto stage = [&](int t) { return ring + (uint32_t)(((c0 + t - t0) % S::kStages) * S::kStage); };

    // page numbers of the 16 keys from key0 on: rows 0-7 in lane 0, 8-15 in lane 1 (and so on)
    auto pages_at = [&](int t) -> int {
        const int key = key_w + t * kKeys + (lane & 1) * 8;
        if (t >= t1 || key >= hi || key + 8 <= lo) return -1;
        const int col = key >> p.page_shift;
        int page = col < p.table_stride ? __ldg(table + col) : -1;
        if ((unsigned)page >= (unsigned)p.num_pages) {
            set_status(p.status, MNB_ERR_INVALID_ARG);
            page = -1;
        }
        return page;
    };
    auto load = [&](int t, int pages) {
        const int key0 = key_w + t * kKeys;
        if (t < t1 && key0 < hi && key0 + 16 > lo) {
            const int pa = __shfl_sync(~0u, pages, 0), pb = __shfl_sync(~0u, pages, 1);
            const int64_t offa = pa * p.page_stride + head_off + (key0 & ps_mask) * p.token_stride + lchunk * 8;
            const int64_t offb = pb * p.page_stride + head_off + ((key0 + 8) & ps_mask) * p.token_stride + lchunk * 8;
            const uint32_t dst = stage(t);
#pragma unroll
            for (int i = 0; i < 16 / kRpi; ++i) {
                const int r = i * kRpi + lrow;
                const bool b = r >= 8;
                // (zeros for keys that no row of the tile sees: 0 * NaN is NaN)
                const bool ok = (b ? pb : pa) >= 0 && key0 + r >= lo && key0 + r < hi && col_ok;
                const int64_t off = ok ? (b ? offb : offa) + (r & 7) * p.token_stride : 0;
                const uint32_t to = dst + chunk_at<DP>(r, lchunk);
                cp16(to, kp + off, ok);
                cp16(to + S::kHalf, vp + off, ok);
            }
        }
        cp_commit();
    };

    int pg;
    auto first_loads = [&]() {
        pg = pages_at(t0);
#pragma unroll
        for (int s = 0; s < S::kStages - 1; ++s) {
            const int nx = pages_at(t0 + s + 1);
            load(t0 + s, pg);
            pg = nx;
        }
    };
    // the unit's rows of Q (past the last row or depth: zero), through registers
    constexpr int kQ = kRows * kChunks / kThreads;
    static_assert(kQ * kThreads == kRows * kChunks, "Q divides among the threads");
    uint4 qv[kQ];
    auto load_q = [&]() {
#pragma unroll
        for (int i = 0; i < kQ; ++i) {
            const int c = tid + i * kThreads, r = c / kChunks, ch = c % kChunks;
            qv[i] = make_uint4(0, 0, 0, 0);
            if (r < rows && ch * 8 < p.D) {
                const int g = rt * kRows + r;
                const int64_t t = tok0 + g / p.group;
                const int h = hk * p.group + g % p.group;
                qv[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + t * p.q_ts + h * p.q_hs + ch * 8);
            }
        }
    };
    begin_unit();
    first_loads();
    load_q();

    for (bool first = true;; first = false) {
#pragma unroll
        for (int i = 0; i < kQ; ++i) {
            const int c = tid + i * kThreads;
            *reinterpret_cast<uint4*>(qs + chunk_at<DP>(c / kChunks, c % kChunks)) = qv[i];
        }
        __syncthreads();
        const int mi = lane >> 3;
        const uint32_t q_lane = (mi & 1) * 8 + (lane & 7);
        constexpr int KK = DP / 16;
        constexpr bool kQRegs = DP <= 128;
        uint32_t qf[kQRegs ? KK : 1][4];
        if constexpr (kQRegs) {
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) ldsm4(qf[kk], qa + chunk_at<DP>(q_lane, kk * 2 + (mi >> 1)));
        }
        // visible keys of this thread's rows, lane / 4 and lane / 4 + 8
        int row_lo[2], row_hi[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int g = rt * kRows + (lane >> 2) + 8 * j;
            visible_range(p, pl.s.n, pl.s.len, g / p.group, g / p.group + 1, &row_lo[j], &row_hi[j]);
        }
        // every row sees all keys of [full_lo, full_hi)
        int full_lo, full_hi, dummy;
        visible_range(p, pl.s.n, pl.s.len, i0, i0 + 1, &dummy, &full_hi);
        visible_range(p, pl.s.n, pl.s.len, i1 - 1, i1, &full_lo, &dummy);

        float o[DP / 8][4] = {};
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        for (int t = t0; t < t1; ++t) {
            const int nx = pages_at(t + S::kStages);
            load(t + S::kStages - 1, pg);
            pg = nx;
            cp_wait<S::kStages - 1>();
            __syncwarp();
            const int key0 = key_w + t * kKeys;
            if (key0 < hi && key0 + 16 > lo) {
                const uint32_t ka = stage(t), va = ka + S::kHalf;
                float s[2][4] = {};
                const uint32_t k_row = (mi >> 1) * 8 + (lane & 7);
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    uint32_t b[4];
                    ldsm4(b, ka + chunk_at<DP>(k_row, kk * 2 + (mi & 1)));
                    if constexpr (kQRegs) {
                        mma16816<DT>(s[0], qf[kk], b[0], b[1]);
                        mma16816<DT>(s[1], qf[kk], b[2], b[3]);
                    } else {
                        uint32_t a[4];
                        ldsm4(a, qa + chunk_at<DP>(q_lane, kk * 2 + (mi >> 1)));
                        mma16816<DT>(s[0], a, b[0], b[1]);
                        mma16816<DT>(s[1], a, b[2], b[3]);
                    }
                }
                const bool edge = key0 < full_lo || key0 + 16 > full_hi;
                float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v = s[n][e] * p.scale_log2;
                        const int j = e >> 1;
                        if (edge) {
                            const int key = key0 + n * 8 + (lane & 3) * 2 + (e & 1);
                            if (key < row_lo[j] || key >= row_hi[j]) v = -INFINITY;
                        }
                        s[n][e] = v;
                        top[j] = fmaxf(top[j], v);
                    }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    top[j] = fmaxf(top[j], __shfl_xor_sync(~0u, top[j], 1));
                    top[j] = fmaxf(top[j], __shfl_xor_sync(~0u, top[j], 2));
                }
                if (__any_sync(~0u, top[0] > m[0] + 8.f || top[1] > m[1] + 8.f)) {
                    float f[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float mn = fmaxf(m[j], top[j]);
                        f[j] = mn == -INFINITY ? 1.f : ex2(m[j] - mn);
                        m[j] = mn;
                        l[j] *= f[j];
                    }
#pragma unroll
                    for (int n = 0; n < DP / 8; ++n) {
                        o[n][0] *= f[0];
                        o[n][1] *= f[0];
                        o[n][2] *= f[1];
                        o[n][3] *= f[1];
                    }
                }
                const float base[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
                float e[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        e[n][c] = ex2(s[n][c] - base[c >> 1]);
                        l[c >> 1] += e[n][c];
                    }
                const uint32_t pa[4] = {pack16<DT>(e[0][0], e[0][1]), pack16<DT>(e[0][2], e[0][3]),
                                        pack16<DT>(e[1][0], e[1][1]), pack16<DT>(e[1][2], e[1][3])};
                const uint32_t v_row = (mi & 1) * 8 + (lane & 7);
#pragma unroll
                for (int n = 0; n < DP / 16; ++n) {
                    uint32_t b[4];
                    ldsm4t(b, va + chunk_at<DP>(v_row, n * 2 + (mi >> 1)));
                    mma16816<DT>(o[2 * n], pa, b[0], b[1]);
                    mma16816<DT>(o[2 * n + 1], pa, b[2], b[3]);
                }
            }
            __syncwarp();  // the stage is free for the next load
        }
        // (the range may be empty: any stage then, all loads have landed)
        const int n_tiles = t1 > t0 ? t1 - t0 : 0;
        if (n_tiles == 0) cp_wait<0>();
        const int last = (c0 + (n_tiles ? n_tiles - 1 : S::kStages - 1)) % S::kStages;
        auto o_of = [&](int w) { return reinterpret_cast<float*>(smem + w * S::kRing + last * S::kStage); };
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            l[j] += __shfl_xor_sync(~0u, l[j], 1);
            l[j] += __shfl_xor_sync(~0u, l[j], 2);
            const int r = (lane >> 2) + 8 * j;
            if ((lane & 3) == 0) ml_s[warp * kRows + r] = make_float2(m[j], l[j]);
            float* row = o_of(warp) + r * DP + (lane & 3) * 2;
#pragma unroll
            for (int n = 0; n < DP / 8; ++n) *reinterpret_cast<float2*>(row + ((n ^ (r & 7)) * 8)) = make_float2(o[n][2 * j], o[n][2 * j + 1]);
        }
        const bool done = dv.whole || (t0 == 0 && t1 == pl.s.tiles);
        const int e_rt = rt, e_hk = hk, e_rows = rows;
        const int64_t e_tok0 = tok0;
        bool more = false;
        if constexpr (!CL) {
            if (tid == 0 && !dv.whole && t1 < pl.s.tiles && x0 <= pl.unit_begin) {
                // this range's end is the first cut of the unit; its pieces end with the last CTA that begins before its end
                const int64_t end = ((pl.unit_begin + pl.s.tiles) * dv.ctas - 1) / dv.total;
                sp.cut[blockIdx.x] = make_int4((int)tok0, rt * kRows, hk | rows << 16,
                                               (int)(end - blockIdx.x + 1) * 2 + (first ? 0 : 1));
            }
            // the next unit's first loads are on their way while this one is joined and written
            more = !dv.whole && x1 > pl.unit_begin + pl.s.tiles;
            if (more) {
                next_unit<kRows, kKeys>(p, pl);
                more = x1 > pl.unit_begin;
            }
            if (more) {
                c0 = (last + 1) % S::kStages;
                begin_unit();
                first_loads();
                load_q();
            }
        }
        __syncthreads();
        {
            const int r = tid >> 3, q8 = tid & 7;  // 8 threads a row, groups of 8 columns each
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml_s[w * kRows + r].x);
            const float base = top == -INFINITY ? 0.f : top;
            float wt[kWarps], sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 v = ml_s[w * kRows + r];
                wt[w] = ex2(v.x - base);
                sum = fmaf(v.y, wt[w], sum);
            }
            if (CL || r < e_rows) {
                const int g = e_rt * kRows + r;
                const int64_t tk = e_tok0 + g / p.group;
                const int h = e_hk * p.group + g % p.group;
                const int slot = first ? 0 : 1;
                const int64_t at = ((int64_t)blockIdx.x * 2 + slot) * kRows + r;
                const float inv = 1.f / sum;
                for (int c = q8; c < DP / 8; c += 8) {
                    float a[8] = {};
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float4* src = reinterpret_cast<const float4*>(o_of(w) + r * DP + ((c ^ (r & 7)) * 8));
                        const float4 u = src[0], v = src[1];
                        a[0] = fmaf(u.x, wt[w], a[0]); a[1] = fmaf(u.y, wt[w], a[1]);
                        a[2] = fmaf(u.z, wt[w], a[2]); a[3] = fmaf(u.w, wt[w], a[3]);
                        a[4] = fmaf(v.x, wt[w], a[4]); a[5] = fmaf(v.y, wt[w], a[5]);
                        a[6] = fmaf(v.z, wt[w], a[6]); a[7] = fmaf(v.w, wt[w], a[7]);
                    }
                    if (CL) {
                        float4* dst = reinterpret_cast<float4*>(o_c + r * DP + c * 8);
                        dst[0] = make_float4(a[0], a[1], a[2], a[3]);
                        dst[1] = make_float4(a[4], a[5], a[6], a[7]);
                    } else if (done) {
                        if (c * 8 < p.D) {
                            uint4 out = make_uint4(0, 0, 0, 0);  // without a key: its a may be 0 * NaN
                            if (sum != 0.f) {
                                out.x = pack16<DT>(a[0] * inv, a[1] * inv);
                                out.y = pack16<DT>(a[2] * inv, a[3] * inv);
                                out.z = pack16<DT>(a[4] * inv, a[5] * inv);
                                out.w = pack16<DT>(a[6] * inv, a[7] * inv);
                            }
                            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + tk * p.o_ts + h * p.o_hs + c * 8) = out;
                        }
                    } else {
                        float4* dst = reinterpret_cast<float4*>(sp.part_o + at * DP + c * 8);
                        dst[0] = make_float4(a[0], a[1], a[2], a[3]);
                        dst[1] = make_float4(a[4], a[5], a[6], a[7]);
                    }
                }
                if (q8 == 0) {
                    if (CL) ml_c[r] = make_float2(top, sum);
                    else if (!done) sp.part_ml[at] = make_float2(top, sum);
                    else if (p.lse) p.lse[tk * p.q_heads + h] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * kLn2;
                }
            }
        }
        if constexpr (CL) {
            cluster_sync();
            // CTA `rank` joins rows rank, rank + peers, ..., a warp a row
            for (int r = rank + warp * peers; r < e_rows; r += peers * kWarps) {
                float top = -INFINITY;
                for (int c = 0; c < peers; ++c) top = fmaxf(top, ld_peer2(ml_c + r, (uint32_t)c).x);
                const float base = top == -INFINITY ? 0.f : top;
                float sum = 0.f, a[DP / 32] = {};
                for (int c = 0; c < peers; ++c) {
                    const float2 v = ld_peer2(ml_c + r, (uint32_t)c);
                    const float w = ex2(v.x - base);
                    sum = fmaf(v.y, w, sum);
#pragma unroll
                    for (int d = 0; d < DP / 64; ++d) {
                        const float2 u = ld_peer2(o_c + r * DP + d * 64 + lane * 2, (uint32_t)c);
                        a[2 * d] = fmaf(u.x, w, a[2 * d]);
                        a[2 * d + 1] = fmaf(u.y, w, a[2 * d + 1]);
                    }
                }
                const int g = e_rt * kRows + r;
                const int64_t tk = e_tok0 + g / p.group;
                const int h = e_hk * p.group + g % p.group;
                const float inv = 1.f / sum;
                uint16_t* dst = static_cast<uint16_t*>(p.o) + tk * p.o_ts + h * p.o_hs;
#pragma unroll
                for (int d = 0; d < DP / 64; ++d)
                    if (d * 64 + lane * 2 < p.D)
                        *reinterpret_cast<uint32_t*>(dst + d * 64 + lane * 2) = sum == 0.f ? 0u : pack16<DT>(a[2 * d] * inv, a[2 * d + 1] * inv);
                if (lane == 0 && p.lse) p.lse[tk * p.q_heads + h] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * kLn2;
            }
            cluster_sync();  // nobody leaves while its shared memory is read
            return;
        }
        if (!more) break;
        // (the barrier behind the next Q keeps the exchange's stage and ml_s until all have read them)
    }
}

}  // namespace mma
}  // namespace attn
}  // namespace mnb
