// The two kernels of mnb_moe:
//
//   gate_up:  h[t, s, :] = w[t, s] * act(gate_e x_t) * (up_e x_t),   e = ids[t, s]
//   down:     y[t, :]    = sum_s down_e h[t, s, :]
//
// The active experts' weights are read once and everything else is small, so
// their bytes bound both.  What a warp does for 512 bytes of packed 4-bit
// codes (a tile of 16 rows x 64 depths): 4 k-steps of an unpack (7 shifts and
// ands, 4 exact packed subtractions of the zero point) and one m16n8k16 MMA per
// 8 columns.
//
// The work unit of a warp is an item: two row tiles that multiply the same
// columns (gate and up of one row tile; two neighbouring row tiles of down), 128
// depths.  Its weights go straight from global memory into registers, its
// scales and zero points too (a lane those of one of the 32 rows; as float and
// subtraction constant they then pass through a table of the warp in shared
// memory), and its columns through asynchronous copies into a slot of the warp
// in shared memory, DEPTH items ahead.  Warps wait for no other warp while they
// stream; sharing the columns between two row tiles halves what their fragments
// cost in shared-memory cycles, which otherwise bound the loop before the
// weights' bytes do.
//
// The columns of an item are the tokens of its expert: its pairs (t, s), in
// ascending order, at most 8 NG of them a segment (down: 4 NG, each as a high
// and a low bf16 part, so that h keeps 16 bits and no f16 can overflow; the two
// columns are added before they leave).  An expert with more pairs has more
// segments, whose weights come from L2.
//
// gate_up: teams of 1, 2, 4 or 8 warps take row tiles; a team's warps split the
// depths and one of them adds the partial sums, in order.  down: a cluster of
// CTAs owns 32 rows of y and its warps split the depths of all experts, each an
// equal range; partial sums of tokens are added over the warps, then over the
// cluster through distributed shared memory, in order.  So results repeat.
//
// Both are launched as programmatic dependents.  down begins while gate_up
// runs: it needs the experts only (from the logits, or from a routing kernel
// that was complete before gate_up began), and has its first items' weights in
// flight when gate_up ends.
#pragma once

#include "decoder.h"
#include "gemv_mma.cuh"
#include "moe_route.cuh"

namespace mnb {
namespace moe {

using gmma::mma16816;
using gmma::Unpack;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kDepth = 128;                // depths of an item
constexpr int kSlotRow = kDepth * 2 + 16;  // bytes of a column in a slot: padded, ldmatrix rows meet no bank twice

struct Seg {
    int e, first, cnt;  // expert, place of its first pair in the sorted list, pairs
};

// Shared memory after the streaming buffers: the routing of the call.
struct Lists {
    int* nseg;
    float* w;      // weight of pair p
    int* ids;      // expert of pair p
    int* sorted;   // pairs by expert, ascending
    Seg* seg;
    int* cnt;      // pairs of each expert, then its first place
    __device__ __forceinline__ Lists(uint8_t* at, int P) {
        nseg = reinterpret_cast<int*>(at);
        w = reinterpret_cast<float*>(at + 16);
        ids = reinterpret_cast<int*>(w + P);
        sorted = ids + P;
        seg = reinterpret_cast<Seg*>(sorted + P);
        cnt = reinterpret_cast<int*>(seg + P);
    }
    static size_t bytes(int P, int E) { return 16 + (size_t)P * 24 + (size_t)E * 4; }
};

// Routes (or reads the routing) and sorts the pairs by expert, in segments of at most `cap` pairs.  All threads call it.
__device__ __forceinline__ void make_lists(const Params& p, const Lists& L, int cap) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = p.r.S, P = p.r.T * S, E = p.r.E;
    for (int i = tid; i < E; i += kThreads) L.cnt[i] = 0;
    if (p.ids_in) {
        for (int i = tid; i < P; i += kThreads) {
            L.ids[i] = p.ids_in[i];
            L.w[i] = p.w_in[i];
        }
    } else if (warp < p.r.T) {
        int e;
        float w;
        route_any(p.r, warp, e, w);
        if (lane < S) {
            L.ids[warp * S + lane] = e;
            L.w[warp * S + lane] = w;
            if (p.ids_out && blockIdx.x == 0) p.ids_out[warp * S + lane] = e;
            if (p.w_out && blockIdx.x == 0) p.w_out[warp * S + lane] = w;
        }
    }
    __syncthreads();
    if (warp == 0) {
        // rank of each pair among its expert's: a match over 32 pairs, after those of the chunks before
        for (int i0 = 0; i0 < P; i0 += 32) {
            const int i = i0 + lane;
            const int e = i < P ? L.ids[i] : -1 - lane;
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
            const int rank = __popc(same & ((1u << lane) - 1u));
            const int before = i < P ? L.cnt[e] : 0;
            __syncwarp();
            if (i < P) {
                L.sorted[i] = before + rank;  // for now
                if (rank == 0) L.cnt[e] = before + __popc(same);
            }
            __syncwarp();
        }
        int first = 0, segs = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane, c = e < E ? L.cnt[e] : 0, n = (c + cap - 1) / cap;
            int fs = c, ss = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(0xFFFFFFFFu, fs, o), b = __shfl_up_sync(0xFFFFFFFFu, ss, o);
                if (lane >= o) {
                    fs += a;
                    ss += b;
                }
            }
            const int f = first + fs - c, s = segs + ss - n;
            for (int k = 0; k < n; ++k) L.seg[s + k] = Seg{e, f + k * cap, min(cap, c - k * cap)};
            if (e < E) L.cnt[e] = f;
            first += __shfl_sync(0xFFFFFFFFu, fs, 31);
            segs += __shfl_sync(0xFFFFFFFFu, ss, 31);
        }
        if (lane == 0) *L.nseg = segs;
    }
    __syncthreads();
    int rank[kMaxPairs / kThreads];
#pragma unroll
    for (int k = 0; k < kMaxPairs / kThreads; ++k) {
        const int i = tid + k * kThreads;
        rank[k] = i < P ? L.sorted[i] + L.cnt[L.ids[i]] : 0;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMaxPairs / kThreads; ++k) {
        const int i = tid + k * kThreads;
        if (i < P) L.sorted[rank[k]] = i;
    }
    __syncthreads();
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

// SUB: k-steps that one scale covers in the loop (2: blocks of 32 depths and more; 1: blocks of 16).
template <int BITS, bool BF, int SUB, int NG>
struct Item {
    static constexpr int TPI = BITS / 2;   // packed tiles of 128 depths
    static constexpr int SPT = 16 / BITS;  // k-steps of a packed tile
    static constexpr int NSUB = 8 / SUB;   // scales of a row
    // items in flight: what 128 registers hold (8-bit weights take 32 a buffer)
    static constexpr int DEPTH = BITS == 8 || SUB == 1 || NG == 2 ? 2 : 3;
    static constexpr int kSlotBytes = 8 * NG * kSlotRow;
    static constexpr int kTabBytes = 2 * NSUB * 16 * 8;
    using U = Unpack<BITS, BF>;

    uint4 w[2][TPI];
    uint32_t s[NSUB], z[NSUB];  // raw scales and zero points of the lane's row

    // w0, w1: the lane's 16 bytes of the row tiles' first packed tile; srow, zrow: the lane's row (zrow null: none)
    __device__ __forceinline__ void load(const Params& p, const uint8_t* w0, const uint8_t* w1, const uint8_t* srow,
                                         const uint8_t* zrow, int c) {
        const int kt = (int)p.a.k_tiles;
#pragma unroll
        for (int j = 0; j < TPI; ++j) {
            // past the last tile the columns are zero: any codes do
            const int64_t at = (int64_t)min(c * TPI + j, kt - 1) * kTileBytes;
            w[0][j] = ldg_stream(w0 + at);
            w[1][j] = ldg_stream(w1 + at);
        }
        if (p.s_vec) {
            if constexpr (SUB == 2) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(srow) + c);
                s[0] = v.x;
                s[1] = v.y;
            } else {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(srow) + c);
                s[0] = v.x;
                s[1] = v.y;
                s[2] = v.z;
                s[3] = v.w;
            }
        } else {
            const int every = max(1 << p.bs_shift >> (SUB == 2 ? 5 : 4), 1) - 1;
#pragma unroll
            for (int j = 0; j < NSUB; ++j) {
                const int b = (c * kDepth + j * 16 * SUB) >> p.bs_shift;
                if (j == 0 || (j & every) == 0) {
                    s[j] = 0u;  // depths past the last block: scale 0
                    if (b < p.a.KB)
                        s[j] = p.sdt == kF32 ? __ldg(reinterpret_cast<const uint32_t*>(srow) + b)
                                             : (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(srow) + b);
                }
            }
        }
        if (zrow != nullptr) {
            if (p.z_vec) {
                constexpr int ZB = NSUB * BITS / 8;  // bytes of an item
                if constexpr (ZB == 1) z[0] = __ldg(zrow + c);
                else if constexpr (ZB == 2) z[0] = __ldg(reinterpret_cast<const uint16_t*>(zrow) + c);
                else if constexpr (ZB == 4) z[0] = __ldg(reinterpret_cast<const uint32_t*>(zrow) + c);
                else {
                    const uint2 v = __ldg(reinterpret_cast<const uint2*>(zrow) + c);
                    z[0] = v.x;
                    z[1] = v.y;
                }
            } else {
                const int every = max(1 << p.bs_shift >> (SUB == 2 ? 5 : 4), 1) - 1;
#pragma unroll
                for (int j = 0; j < NSUB; ++j) {
                    const int b = min((c * kDepth + j * 16 * SUB) >> p.bs_shift, p.a.KB - 1);
                    if (j == 0 || (j & every) == 0) z[j] = (uint32_t)__ldg(zrow + ((b * BITS) >> 3)) >> ((b * BITS) & 7);
                }
            }
        }
    }

    static __device__ __forceinline__ float widen(uint32_t raw, int dt) {
        if (dt == kF32) return __uint_as_float(raw);
        return dt == kBF16 ? __uint_as_float(raw << 16) : __half2float(__ushort_as_half((unsigned short)raw));
    }

    // The lane's row into the warp's table: entry [row tile][j][row] = (scale, subtraction constant).
    __device__ __forceinline__ void table(const Params& p, uint2* tab, bool has_z) const {
        const int lane = threadIdx.x & 31;
        uint2* dst = tab + (lane >> 4) * NSUB * 16 + (lane & 15);
        const int every = max(1 << p.bs_shift >> (SUB == 2 ? 5 : 4), 1) - 1;
        uint32_t sr = 0, zr = 0;
#pragma unroll
        for (int j = 0; j < NSUB; ++j) {
            const bool own = j == 0 || (j & every) == 0;
            if (p.s_vec) sr = (j & 1) ? s[j >> 1] >> 16 : s[j >> 1] & 0xFFFFu;
            else if (own) sr = s[j];
            if (p.z_vec) {
                constexpr int per = 32 / BITS;
                zr = z[j / per] >> ((j % per) * BITS);
            } else if (own) {
                zr = z[j];
            }
            const uint32_t zp = has_z ? zr & (uint32_t)((1 << BITS) - 1) : 1u << (BITS - 1);
            dst[j * 16] = make_uint2(__float_as_uint(widen(sr, p.sdt)), U::zconst(zp));
        }
    }

    // y[m][ng] += row tile m times column group ng.  slot: the warp's columns; tab: its table.
    __device__ __forceinline__ void compute(uint32_t slot, const uint2* tab, float (&y)[2][NG][4]) const {
        const int lane = threadIdx.x & 31, g = lane >> 2;
        const float zero4[4] = {0.f, 0.f, 0.f, 0.f};
        const uint32_t at = slot + (uint32_t)((lane & 7) * kSlotRow + (lane >> 3) * 16);
        float acc[2][NG][4];
        uint32_t x[NG][4];
        uint2 lo[2], hi[2];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k % SUB == 0) {
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    lo[m] = tab[(m * NSUB + k / SUB) * 16 + g];
                    hi[m] = tab[(m * NSUB + k / SUB) * 16 + g + 8];
                }
            }
            if ((k & 1) == 0) {
#pragma unroll
                for (int n = 0; n < NG; ++n) ldmatrix4(x[n], at + (uint32_t)(n * 8 * kSlotRow + k * 32));
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                uint32_t a[4];
                U::kstep(w[m][k / SPT], k % SPT, lo[m].y, hi[m].y, a);
#pragma unroll
                for (int n = 0; n < NG; ++n) {
                    const uint32_t b0 = x[n][2 * (k & 1)], b1 = x[n][2 * (k & 1) + 1];
                    if (k % SUB == 0) mma16816<BF>(acc[m][n], a, b0, b1, zero4);
                    else mma16816<BF>(acc[m][n], a, b0, b1, acc[m][n]);
                    if (k % SUB == SUB - 1) {
                        const float sl = __uint_as_float(lo[m].x), sh = __uint_as_float(hi[m].x);
                        y[m][n][0] = fmaf(sl, acc[m][n][0], y[m][n][0]);
                        y[m][n][1] = fmaf(sl, acc[m][n][1], y[m][n][1]);
                        y[m][n][2] = fmaf(sh, acc[m][n][2], y[m][n][2]);
                        y[m][n][3] = fmaf(sh, acc[m][n][3], y[m][n][3]);
                    }
                }
            }
        }
    }
};

// Addresses of two row tiles of an expert for one lane (lanes 0-15: the first tile's rows, 16-31 the second's).
struct RowTiles {
    const uint8_t *w0, *w1, *srow, *zrow;
    __device__ __forceinline__ void set(const Params& p, int e, int64_t rt0, int64_t rt1) {
        const int lane = threadIdx.x & 31;
        const Weights& q = lane < 16 ? p.a : p.b;
        const int n = min((int)(lane < 16 ? rt0 : rt1) * 16 + (lane & 15), q.N - 1);
        w0 = p.a.packed + (size_t)e * p.a.expert_bytes + kHeaderBytes + (size_t)rt0 * p.a.k_tiles * kTileBytes + lane * 16;
        w1 = p.b.packed + (size_t)e * p.b.expert_bytes + kHeaderBytes + (size_t)rt1 * p.b.k_tiles * kTileBytes + lane * 16;
        srow = q.scales + (size_t)e * q.scale_bytes + (size_t)n * q.KB * (p.sdt == kF32 ? 4 : 2);
        zrow = q.zp ? q.zp + (size_t)e * q.zp_bytes + (size_t)n * q.zp_row : nullptr;
    }
};

__device__ __forceinline__ void check_headers(const Params& p, const Weights& q, int e, int BITS) {
    Layout L;
    L.init(q.N, q.K, BITS, 1 << p.bs_shift);
    verify_header(q.packed + (size_t)e * q.expert_bytes, L, p.status);
}

__device__ __forceinline__ float activate(float g, int act) {
    if (act == MNB_ACT_SILU) return g / (1.f + expf(-g));
    const float u = 0.7978845608028654f * (g + 0.044715f * g * g * g);  // sqrt(2 / pi)
    return 0.5f * g * (1.f + tanhf(u));
}

__device__ __forceinline__ void team_barrier(int team, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(threads) : "memory");
}

template <int BITS, bool BF, int SUB, int NG>
__global__ void __launch_bounds__(kThreads, 2) gate_up_kernel(const __grid_constant__ Params p) {
    using It = Item<BITS, BF, SUB, NG>;
    constexpr int DEPTH = It::DEPTH;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t slots = smem_u32(smem) + (uint32_t)(warp * DEPTH * It::kSlotBytes);
    uint8_t* at = smem + kWarps * DEPTH * It::kSlotBytes;
    uint2* tab = reinterpret_cast<uint2*>(at + warp * It::kTabBytes);
    at += kWarps * It::kTabBytes;
    float4* red = reinterpret_cast<float4*>(at);  // [warp][2 NG][lane]
    at += kWarps * 2 * NG * 32 * 16;
    const Lists L(at, p.r.T * p.r.S);

    griddep_wait();
    griddep_launch_dependents();
    make_lists(p, L, 8 * NG);

    const int KC = (p.a.K + kDepth - 1) / kDepth, NT = (int)p.a.row_tiles;
    const int units = *L.nseg * NT;
    // warps a row tile: the fewest items in a row for any warp, then the fewest warps
    int wpu = 1, cost = 0x7FFFFFFF;
    for (int w = 1; w <= kWarps && w <= KC; w *= 2) {
        const int teams = (int)gridDim.x * (kWarps / w);
        const int c = ((units + teams - 1) / teams) * ((KC + w - 1) / w);
        if (c < cost) {
            cost = c;
            wpu = w;
        }
    }
    const int team = warp / wpu, wit = warp % wpu;
    const int stride = (int)gridDim.x * (kWarps / wpu);

    // a warp's items: chunks wit, wit + wpu, ... of the team's row tiles
    struct Cursor {
        int u, c;
    };
    auto advance = [&](Cursor& i) {
        i.c += wpu;
        if (i.c >= KC) {
            i.c = wit;
            i.u += stride;
        }
    };
    Cursor cur{(int)blockIdx.x + team * (int)gridDim.x, wit}, ahead = cur;
    RowTiles rows;
    Seg ls{0, 0, 0};
    int lu = -1;
    auto load = [&](It& b, uint32_t slot) {
        if (ahead.u < units) {
            if (ahead.u != lu) {
                lu = ahead.u;
                const int sg = lu / NT, rt = lu - sg * NT;
                ls = L.seg[sg];
                rows.set(p, ls.e, rt, rt);
            }
            b.load(p, rows.w0, rows.w1, rows.srow, rows.zrow, ahead.c);
            const int piece = lane & 15, k = ahead.c * kDepth + piece * 8, left = p.a.K - k;
#pragma unroll 1
            for (int col = lane >> 4; col < ls.cnt; col += 2) {
                const int64_t row = (int64_t)(L.sorted[ls.first + col] / p.r.S) * p.x_stride;
                const uint16_t* x = static_cast<const uint16_t*>(p.x) + row;
                const uint32_t dst = slot + (uint32_t)(col * kSlotRow + piece * 16);
                if (p.x_wide) {
                    cp_async16(dst, left > 0 ? x + k : x, max(0, min(left * 2, 16)));
                } else {
                    uint32_t v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t lo = 2 * j < left ? x[k + 2 * j] : 0u, hi = 2 * j + 1 < left ? x[k + 2 * j + 1] : 0u;
                        v[j] = lo | (hi << 16);
                    }
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                                 : "memory");
                }
            }
            advance(ahead);
        }
        cp_commit();
    };

    float y[2][NG][4];
    auto clear = [&] {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
#pragma unroll
            for (int n = 0; n < NG; ++n) {
#pragma unroll
                for (int j = 0; j < 4; ++j) y[m][n][j] = 0.f;
            }
        }
    };
    clear();
    // the row tile's sums are complete (in wpu warps): h of its rows
    int turn = 0;
    auto finish = [&](int u) {
        const int sg = u / NT, rt = u - sg * NT;
        if (wpu > 1) {
            team_barrier(team, wpu * 32);  // the partials of the row tile before are read
#pragma unroll
            for (int m = 0; m < 2; ++m) {
#pragma unroll
                for (int n = 0; n < NG; ++n)
                    red[(warp * 2 * NG + m * NG + n) * 32 + lane] = make_float4(y[m][n][0], y[m][n][1], y[m][n][2], y[m][n][3]);
            }
            team_barrier(team, wpu * 32);
        }
        if (wit == turn) {
            if (wpu > 1) {
                clear();
                for (int w = 0; w < wpu; ++w) {
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
#pragma unroll
                        for (int n = 0; n < NG; ++n) {
                            const float4 v = red[((team * wpu + w) * 2 * NG + m * NG + n) * 32 + lane];
                            y[m][n][0] += v.x;
                            y[m][n][1] += v.y;
                            y[m][n][2] += v.z;
                            y[m][n][3] += v.w;
                        }
                    }
                }
            }
            const Seg sgm = L.seg[sg];
#pragma unroll
            for (int n = 0; n < NG; ++n) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int col = n * 8 + 2 * (lane & 3) + (j & 1), row = rt * 16 + (lane >> 2) + 8 * (j >> 1);
                    if (col < sgm.cnt) {
                        const int pair = L.sorted[sgm.first + col];
                        const float v = row < p.a.N ? activate(y[0][n][j], p.act) * y[1][n][j] * L.w[pair] : 0.f;
                        const __nv_bfloat16 hi = __float2bfloat16_rn(v);
                        const float rest = v - __bfloat162float(hi);  // exact; NaN beside an infinity
                        uint16_t* dst = p.h + (int64_t)pair * 2 * p.inner + row;
                        dst[0] = __bfloat16_as_ushort(hi);
                        dst[p.inner] = isinf(__bfloat162float(hi)) ? 0 : __bfloat16_as_ushort(__float2bfloat16_rn(rest));
                    }
                }
            }
        }
        if (++turn == wpu) turn = 0;
        clear();
    };

    It buf[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(buf[d], slots + d * It::kSlotBytes);
    const bool has_z = (lane < 16 ? p.a.zp : p.b.zp) != nullptr;
    auto step = [&](It& b, uint32_t slot) {
        if (cur.u >= units) return false;
        cp_wait<DEPTH - 1>();
        b.table(p, tab, has_z);
        __syncwarp();
        b.compute(slot, tab, y);
        __syncwarp();
        load(b, slot);
        const int u = cur.u;
        advance(cur);
        if (cur.u != u) finish(u);
        return true;
    };
    bool more = true;
    while (more) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            if (more) more = step(buf[d], slots + d * It::kSlotBytes);
    }
    cp_wait<0>();
    if (blockIdx.x == 0)
        for (int i = tid; i < *L.nseg; i += kThreads) {
            check_headers(p, p.a, L.seg[i].e, BITS);
            check_headers(p, p.b, L.seg[i].e, BITS);
        }
}

template <int BITS, int SUB, int NG>
__global__ void __launch_bounds__(kThreads, 2) down_kernel(const __grid_constant__ Params p) {
    using It = Item<BITS, true, SUB, NG>;
    constexpr int DEPTH = It::DEPTH;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t slots = smem_u32(smem) + (uint32_t)(warp * DEPTH * It::kSlotBytes);
    uint8_t* at = smem + kWarps * DEPTH * It::kSlotBytes;
    uint2* tab = reinterpret_cast<uint2*>(at + warp * It::kTabBytes);
    at += kWarps * It::kTabBytes;
    const int T = p.r.T;
    float* sums = reinterpret_cast<float*>(at);  // [warp][token][32 rows]
    at += (size_t)kWarps * T * 32 * 4;
    const Lists L(at, T * p.r.S);
    const int C = p.cluster;
    const int rank = C > 1 ? (int)cluster_ctarank() : 0;
    const int group = (int)blockIdx.x / C;

    for (int i = tid; i < kWarps * T * 32; i += kThreads) sums[i] = 0.f;
    // The routing's inputs were complete before the kernel that this one follows began: no wait.
    make_lists(p, L, 4 * NG);

    const int IC = ((int)p.inner + kDepth - 1) / kDepth, items = *L.nseg * IC;
    const int W = C * kWarps, me = rank * kWarps + warp;
    const int i0 = (int)((int64_t)items * me / W), i1 = (int)((int64_t)items * (me + 1) / W);
    const int64_t rt0 = 2 * group, rt1 = min(rt0 + 1, p.a.row_tiles - 1);
    RowTiles rows;
    Seg ls{0, 0, 0};
    int lsg = -1, ahead = i0;
    auto place = [&](int i) {  // the segment and chunk of item i, and the segment's addresses
        const int sg = i / IC;
        if (sg != lsg) {
            lsg = sg;
            ls = L.seg[sg];
            rows.set(p, ls.e, rt0, rt1);
        }
        return i - sg * IC;
    };
    auto columns = [&](int i, int c, const Seg& sg, uint32_t slot) {
        const int piece = lane & 15, k = c * kDepth + piece * 8, left = (int)p.inner - k;
#pragma unroll 1
        for (int r = lane >> 4; r < 2 * sg.cnt; r += 2) {  // token r / 2, its high or low part
            const int j = r >> 1, col = (j & 3) + 4 * (r & 1) + 8 * (j >> 2);
            const uint16_t* h = p.h + ((int64_t)L.sorted[sg.first + j] * 2 + (r & 1)) * p.inner;
            cp_async16(slot + (uint32_t)(col * kSlotRow + piece * 16), left > 0 ? h + k : h, max(0, min(left * 2, 16)));
        }
        (void)i;
    };
    auto load = [&](It& b, uint32_t slot) {
        if (ahead < i1) {
            const int c = place(ahead);
            b.load(p, rows.w0, rows.w1, rows.srow, rows.zrow, c);
            columns(ahead, c, ls, slot);
            ++ahead;
        }
        cp_commit();
    };

    It buf[DEPTH];
    // the first items' weights before the wait for h, their columns after it
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        if (i0 + d < i1) {
            const int c = place(i0 + d);
            buf[d].load(p, rows.w0, rows.w1, rows.srow, rows.zrow, c);
        }
    griddep_wait();
    griddep_launch_dependents();
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
        if (ahead < i1) {
            const int c = place(ahead);
            columns(ahead, c, ls, slots + d * It::kSlotBytes);
            ++ahead;
        }
        cp_commit();
    }

    float y[2][NG][4];
    auto clear = [&] {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
#pragma unroll
            for (int n = 0; n < NG; ++n) {
#pragma unroll
                for (int j = 0; j < 4; ++j) y[m][n][j] = 0.f;
            }
        }
    };
    clear();
    float* mine = sums + warp * T * 32;
    // a segment ends: its columns' high and low parts are added and go to their tokens' sums
    auto flush = [&](int sg) {
        const Seg s = L.seg[sg];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
#pragma unroll
            for (int n = 0; n < NG; ++n) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float v = y[m][n][j] + __shfl_xor_sync(0xFFFFFFFFu, y[m][n][j], 2);
                    const int col = n * 4 + 2 * (lane & 3) + (j & 1);
                    if ((lane & 3) < 2 && col < s.cnt)
                        mine[L.sorted[s.first + col] / p.r.S * 32 + m * 16 + (lane >> 2) + 8 * (j >> 1)] += v;
                }
            }
        }
        clear();
        __syncwarp();
    };
    const bool has_z = p.a.zp != nullptr;
    int cur = i0;
    auto step = [&](It& b, uint32_t slot) {
        if (cur >= i1) return false;
        cp_wait<DEPTH - 1>();
        b.table(p, tab, has_z);
        __syncwarp();
        b.compute(slot, tab, y);
        __syncwarp();
        load(b, slot);
        const int sg = cur / IC;
        ++cur;
        if (cur == i1 || cur / IC != sg) flush(sg);
        return true;
    };
    bool more = true;
    while (more) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            if (more) more = step(buf[d], slots + d * It::kSlotBytes);
    }
    cp_wait<0>();
    __syncthreads();
    for (int i = tid; i < T * 32; i += kThreads) {
        float v = sums[i];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v += sums[w * T * 32 + i];
        sums[i] = v;
    }
    if (C > 1) cluster_sync();
    else __syncthreads();
    // the cluster's CTAs take equal parts of the tokens x 32 values
    for (int i = rank * kThreads + tid; i < T * 32; i += C * kThreads) {
        float v = sums[i];
        if (C > 1) {
            v = 0.f;
            for (int r = 0; r < C; ++r) v += ld_dsmem_f32(sums + i, (uint32_t)r);
        }
        const int64_t n = (int64_t)group * 32 + (i & 31);
        if (n < p.a.N) store_f32(p.y, (int64_t)(i >> 5) * p.y_stride + n, v, p.y_dt);
    }
    if (C > 1) cluster_sync();  // until the others have read
    if (blockIdx.x == 0)
        for (int i = tid; i < *L.nseg; i += kThreads) check_headers(p, p.a, L.seg[i].e, BITS);
}

template <int BITS, bool BF, int SUB, int NG>
cudaError_t launch_gate_up(const Params& p, cudaStream_t s) {
    using It = Item<BITS, BF, SUB, NG>;
    auto kern = gate_up_kernel<BITS, BF, SUB, NG>;
    const int P = p.r.T * p.r.S;
    const size_t smem = (size_t)kWarps * (It::DEPTH * It::kSlotBytes + It::kTabBytes + 2 * NG * 32 * 16) + Lists::bytes(P, p.r.E);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    // two CTAs an SM; no more than the row tiles of the most experts that can be active
    const int64_t most = (int64_t)(P < p.r.E ? P : p.r.E) * p.a.row_tiles;
    const int grid = (int)(most < 2 * dec::kSms ? most : 2 * dec::kSms);
    return dec::launch_pdl(kern, dim3(grid), dim3(kThreads), smem, s, 1, p);
}

template <int BITS, int SUB, int NG>
cudaError_t launch_down(const Params& p, cudaStream_t s) {
    using It = Item<BITS, true, SUB, NG>;
    auto kern = down_kernel<BITS, SUB, NG>;
    const size_t smem = (size_t)kWarps * (It::DEPTH * It::kSlotBytes + It::kTabBytes + p.r.T * 32 * 4) +
                        Lists::bytes(p.r.T * p.r.S, p.r.E);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int64_t groups = (p.a.row_tiles + 1) / 2;
    // as many CTAs a group of 32 rows as two an SM hold, up to a portable cluster
    Params q = p;
    q.cluster = 1;
    while (q.cluster < 8 && groups * q.cluster * 2 <= 2 * dec::kSms) q.cluster *= 2;
    return dec::launch_pdl(kern, dim3((unsigned)(groups * q.cluster)), dim3(kThreads), smem, s, q.cluster, q);
}

template <int BITS, int SUB>
cudaError_t launch_sub(const Params& g, const Params& d, int bf, cudaStream_t s) {
    // columns: one group of 8 (4 tokens in two parts) where no expert can have more pairs
    const bool two = g.r.T > 8;
    cudaError_t e;
    if (bf) e = two ? launch_gate_up<BITS, true, SUB, 2>(g, s) : launch_gate_up<BITS, true, SUB, 1>(g, s);
    else e = two ? launch_gate_up<BITS, false, SUB, 2>(g, s) : launch_gate_up<BITS, false, SUB, 1>(g, s);
    if (e != cudaSuccess) return e;
    return d.r.T > 4 ? launch_down<BITS, SUB, 2>(d, s) : launch_down<BITS, SUB, 1>(d, s);
}

template <int BITS>
cudaError_t launch_bits(const Params& g, const Params& d, int bf, cudaStream_t s) {
    return g.bs_shift == 4 ? launch_sub<BITS, 1>(g, d, bf, s) : launch_sub<BITS, 2>(g, d, bf, s);
}

}  // namespace moe
}  // namespace mnb
