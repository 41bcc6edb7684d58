// The two kernels of mnb_moe:
//
//   gate_up:  h[t, s, :] = w[t, s] * act(gate_e x_t) * (up_e x_t),   e = ids[t, s]
//   down:     y[t, :]    = sum_s down_e h[t, s, :]
//
// The active experts' weights are read once and everything else is small, so
// their bytes bound both, and the issue of instructions is the next bound.
//
// Arithmetic.  A code q in the low bits of a 16-bit lane is, read as an f16 or
// bf16 number, q times the type's smallest subnormal (in bits 4 to 7, 16 q
// times it; in bf16 the lowest exponent bit continues the scale up to 255).
// Packed subtraction and the MMA take subnormal operands exactly, so an A
// fragment of 4-bit codes is a shift, four ands and four subtractions of the
// zero point, with no conversion; rows 8 to 15 come out 16 times as large, and
// the sums are scaled at the end.  Columns of bf16 are scaled by 2^60 (h where
// it is written, x in the loop), so that the products are normal numbers.
//
// A warp-level m16n8k16 takes 8 cycles of a quarter of an SM, 2 of the SM: the 16
// of an item's 2 KB take 32 cycles, its bytes from memory about 90.  So the MMAs
// are not the bound, but the instructions around them come close to it.
//
// The work of a warp comes in items: two row tiles that multiply the same
// columns (gate and up of one row tile; two neighbouring row tiles of down), 128
// depths (8-bit codes: 64).  Weights and columns go through a ring of the warp
// in shared memory by asynchronous copies, two to four items ahead: a lane
// copies the 16 bytes of a packed tile that it alone reads, and warps wait for
// no other warp while they stream (bulk copies with barriers took a quarter more
// instructions and 10% more time).  Two row tiles share the fragments of the
// columns, which halves what those cost in shared-memory cycles.  Scales and
// zero points (a lane loads those of one of the 32 rows, one item ahead) pass
// through a table of the warp as floats.  One copy of the loop, indexed by the
// ring's slot, keeps the code in the instruction cache.
//
// The columns of an item are the tokens of its expert: its pairs (t, s), in
// ascending order, at most 8 of them a segment (down: 4, each as a high and a
// low bf16 part, so that h keeps 16 bits and no f16 can overflow; a lane adds
// the two columns before they leave).  An expert with more pairs has more
// segments, whose weights come from L2.
//
// gate_up: a CTA takes consecutive row tiles and its warps equal runs of their
// items.  A row tile inside a warp's run is finished there; the others' partial
// sums are added in order after the runs.  down: a cluster of CTAs owns 32 rows
// of y and its warps equal runs of the items of all experts; partial sums of
// tokens are added over the warps, then over the cluster through distributed
// shared memory, in order.  So results repeat.
//
// Both are launched as programmatic dependents.  down begins while gate_up
// runs: it needs the experts only (from the logits, or from a routing kernel
// that was complete before gate_up began), and has its first items' weights in
// flight when gate_up ends.
//
// Measured (int4, f16 or bf16 scales, both kernels): 4 tokens x 2 of 8 experts of
// 4096 x 14336 in 147 us (3470 GB/s, half a copy's rate; 24 us of it are MMAs,
// issue slots 61% full in gate_up and 51% in down, by 16 warps an SM), 16 tokens x
// 8 of 64 experts of 2048 x 1408 in 78, one token x 8 of 64 of 2048 x 1024 in 20.9,
// of which about 8 stream weights and the rest is the start, routing and the joins
// of two kernels.
#pragma once

#include "decoder.h"
#include "gemv_mma.cuh"
#include "moe_route.cuh"

namespace mnb {
namespace moe {

using gmma::mma16816;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kRingBytes = 9216;         // of a warp: two CTAs fit an SM beside 40 KB of L1 (for the scales); two to four slots
constexpr float kColumnScale = 0x1p60f;  // of bf16 columns

// Shared memory after the streaming buffers: the routing of the call.
struct Lists {
    int *nseg, *most;  // segments; pairs of the largest
    float* w;          // weight of pair p
    int* sorted;       // pairs by expert, ascending
    int* token;        // their tokens
    Seg* seg;
    int* ids;          // expert of pair p; whether it begins a segment (scratch of make_lists)
    int* head;
    __device__ __forceinline__ Lists(uint8_t* at, int P) {
        nseg = reinterpret_cast<int*>(at);
        most = nseg + 1;
        w = reinterpret_cast<float*>(at + 16);
        sorted = reinterpret_cast<int*>(w + P);
        token = sorted + P;
        seg = reinterpret_cast<Seg*>(token + P);
        ids = reinterpret_cast<int*>(seg + P);
        head = ids + P;
    }
    static size_t bytes(int P) { return 16 + (size_t)P * 32; }
};

// The lists of a call, with segments of at most `cap` pairs: from a routing kernel's, or (few tokens and experts) from the
// logits.  All threads call it.  scratch: shared memory for T * E scores and T * E keys.
__device__ __forceinline__ void make_lists(const Params& p, const Lists& L, int cap, uint32_t* scratch) {
    const int tid = threadIdx.x;
    const int S = p.r.S, T = p.r.T, P = T * S, E = p.r.E;
    if (p.plan) {
        const Plan& g = *p.plan;
        const PlanSegs& from = cap == 8 ? g.by8 : g.by4;
        const int n = from.n;
        for (int i = tid; i < P; i += kThreads) {
            L.w[i] = g.w[i];
            L.sorted[i] = g.sorted[i];
            L.token[i] = g.sorted[i] / S;
        }
        for (int i = tid; i < n; i += kThreads) L.seg[i] = from.seg[i];
        if (tid == 0) {
            *L.nseg = n;
            *L.most = from.most;
        }
        __syncthreads();
        return;
    }
    // The rank of a score among its token's is its place: a thread a score, no rounds that wait for each other.
    float* score = reinterpret_cast<float*>(scratch + T * E);
    for (int i = tid; i < T * E; i += kThreads) {
        const int t = i / E, e = i - t * E;
        const float l = load_f32(p.r.logits, t * p.r.stride + e, p.r.dt);
        score[i] = l;
        scratch[i] = route_key(p.r, l, e);
    }
    if (tid == 0) *L.most = 0;
    __syncthreads();
    for (int i = tid; i < T * E; i += kThreads) {
        const int t = i / E, e = i - t * E;
        const uint32_t mine = scratch[i], *all = scratch + t * E;
        int rank = 0;
#pragma unroll 8
        for (int f = 0; f < E; ++f) rank += all[f] > mine || (all[f] == mine && f < e) ? 1 : 0;
        if (rank < S) L.ids[t * S + rank] = e;
    }
    __syncthreads();
    int e = 0, less = 0, before = 0, same = 0;
    bool head = false;
    if (tid < P) {
        // a thread a pair: its weight, and the pairs before it in the order of (expert, pair)
        const int t = tid / S;
        e = L.ids[tid];
        const float w = route_weight(p.r, score + t * E, L.ids + t * S, tid - t * S);
        L.w[tid] = w;
        if (blockIdx.x == 0 && p.ids_out) p.ids_out[tid] = e;
        if (blockIdx.x == 0 && p.w_out) p.w_out[tid] = w;
#pragma unroll 8
        for (int q = 0; q < P; ++q) {
            const int f = L.ids[q];
            less += f < e ? 1 : 0;
            same += f == e ? 1 : 0;
            before += f == e && q < tid ? 1 : 0;
        }
        head = before % cap == 0;
        L.sorted[less + before] = tid;
        L.token[less + before] = t;
        L.head[tid] = head;
    }
    const int heads = __syncthreads_count(head);
    if (head) {
        int at = 0;
#pragma unroll 8
        for (int q = 0; q < P; ++q) at += L.head[q] && (L.ids[q] < e || (L.ids[q] == e && q < tid)) ? 1 : 0;
        const int cnt = min(cap, same - before);
        L.seg[at] = Seg{e, less + before, cnt};
        atomicMax(L.most, cnt);
    }
    if (tid == 0) *L.nseg = heads;
    __syncthreads();
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// `bytes` of 16, the rest zeros (columns: through L1, where a CTA's warps meet)
__device__ __forceinline__ void cp_async16_part(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// The oldest of `depth` groups is complete.
__device__ __forceinline__ void cp_wait_oldest(int depth) {
    if (depth == 2) cp_wait<1>();
    else if (depth == 3) cp_wait<2>();
    else cp_wait<3>();
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

// Read-only loads of scales and zero points: a miss brings 256 bytes of the row into L2, those of the items to come.
template <class T>
__device__ __forceinline__ T ldg_ahead(const T* p) {
    T v;
    if constexpr (sizeof(T) == 16) {
        asm volatile("ld.global.nc.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    } else if constexpr (sizeof(T) == 8) {
        asm volatile("ld.global.nc.L2::256B.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    } else if constexpr (sizeof(T) == 4) {
        asm volatile("ld.global.nc.L2::256B.u32 %0, [%1];" : "=r"(v) : "l"(p));
    } else if constexpr (sizeof(T) == 2) {
        asm volatile("ld.global.nc.L2::256B.u16 %0, [%1];" : "=h"(v) : "l"(p));
    } else {
        uint32_t u;
        asm volatile("ld.global.nc.L2::256B.u8 %0, [%1];" : "=r"(u) : "l"(p));
        v = (T)u;
    }
    return v;
}

// Addresses of two row tiles of an expert for one lane (lanes 0-15: the first tile's rows, 16-31 the second's).
struct RowTiles {
    const uint8_t *w0, *w1;
    __device__ __forceinline__ void set(const Params& p, int e, int rt0, int rt1) {
        const int lane = threadIdx.x & 31;
        const int64_t bytes = p.a.k_tiles * kTileBytes;
        w0 = p.a.packed + (size_t)e * p.a.expert_bytes + kHeaderBytes + rt0 * bytes + lane * 16;
        w1 = p.b.packed + (size_t)e * p.b.expert_bytes + kHeaderBytes + rt1 * bytes + lane * 16;
    }
};
struct RowScales {
    const uint8_t *s, *z;  // z null: no zero points
    __device__ __forceinline__ void set(const Params& p, int e, int rt0, int rt1) {
        const int lane = threadIdx.x & 31;
        const Weights& q = lane < 16 ? p.a : p.b;
        const int n = min((lane < 16 ? rt0 : rt1) * 16 + (lane & 15), q.N - 1);
        s = q.scales + (size_t)e * q.scale_bytes + (size_t)n * q.KB * (p.sdt == kF32 ? 4 : 2);
        z = q.zp ? q.zp + (size_t)e * q.zp_bytes + (size_t)n * q.zp_row : nullptr;
    }
};

// BSL: log2 of the block's k-steps, at most an item's (a longer block spans items).  LIFT: the columns are bf16 values
// that the loop scales.
template <int BITS, bool BF, int BSL, bool LIFT>
struct Item {
    static constexpr int KST = BITS == 8 ? 4 : 8;                // k-steps
    static constexpr int kDepth = 16 * KST;
    static constexpr int SPT = 16 / BITS;                        // k-steps of a packed tile
    static constexpr int TPI = KST / SPT;                        // packed tiles of a row tile
    static constexpr int SUB = (1 << BSL) < KST ? 1 << BSL : KST;  // k-steps of a scale
    static constexpr int NB = KST / SUB;                         // scales of a row
    static constexpr int PC = 2 * KST;                           // 16-byte pieces of a column
    static constexpr int kColBytes = 16 * PC, kColStride = kColBytes + 16;  // (padded: ldmatrix rows meet no bank twice)
    static constexpr int kWBytes = 2 * TPI * kTileBytes;
    static constexpr int kTabBytes = 2 * NB * 16 * 8;
    static constexpr int kLift8 = BITS == 4 ? 16 : BITS == 2 ? 4 : 1;  // rows 8 to 15 of a tile: their codes stand higher
    static constexpr float kUnscale = BF ? 0x1p73f : 0x1p24f;          // of y in rows 0 to 7: 2^133 / kColumnScale, 2^24
    static_assert(NB * BITS <= 32, "an item's zero points of a row are one word");
    // Bytes of a slot: the weights, and as many columns as a segment of the call has.
    static __device__ __forceinline__ int slot_bytes(int cols) { return kWBytes + cols * kColStride; }
    static_assert(2 * (kWBytes + 8 * kColStride) <= kRingBytes, "two slots of 8 columns");

    // Copies of the item's weights into a slot (w0, w1: the lane's 16 bytes of its first packed tiles; `tiles` of them
    // are there).
    static __device__ __forceinline__ void weights(const uint8_t* w0, const uint8_t* w1, int tiles, uint32_t slot) {
        const uint32_t at = slot + (threadIdx.x & 31) * 16;
        if (tiles >= TPI) {
#pragma unroll
            for (int j = 0; j < TPI; ++j) {
                cp_async16(at + j * kTileBytes, w0 + j * kTileBytes);
                cp_async16(at + (TPI + j) * kTileBytes, w1 + j * kTileBytes);
            }
        } else {  // past the last tile the columns are zero: any codes do
#pragma unroll
            for (int j = 0; j < TPI; ++j) {
                cp_async16(at + j * kTileBytes, w0 + min(j, tiles - 1) * kTileBytes);
                cp_async16(at + (TPI + j) * kTileBytes, w1 + min(j, tiles - 1) * kTileBytes);
            }
        }
    }

    // A fragment of k-step s of a lane's 16 packed bytes: q - zp as subnormal numbers, rows 8 to 15 times kLift8.
    static __device__ __forceinline__ void fragment(const uint4& wv, int s, uint32_t zg, uint32_t zg8, uint32_t (&a)[4]) {
        const uint32_t w[4] = {wv.x, wv.y, wv.z, wv.w};
        if constexpr (BITS == 4) {
            const uint32_t v = w[s], u = v >> 8;
            a[0] = v & 0x000F000Fu;
            a[1] = v & 0x00F000F0u;
            a[2] = u & 0x000F000Fu;
            a[3] = u & 0x00F000F0u;
        } else if constexpr (BITS == 2) {
            const uint32_t v = w[s >> 1] >> ((s & 1) * 8), u = v >> 4;
            a[0] = v & 0x00030003u;
            a[1] = v & 0x000C000Cu;
            a[2] = u & 0x00030003u;
            a[3] = u & 0x000C000Cu;
        } else {
            a[0] = prmt(w[2 * s], 0u, 0x4140u);
            a[1] = prmt(w[2 * s], 0u, 0x4342u);
            a[2] = prmt(w[2 * s + 1], 0u, 0x4140u);
            a[3] = prmt(w[2 * s + 1], 0u, 0x4342u);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) a[r] = BF ? gmma::hsub2_bf16(a[r], (r & 1) ? zg8 : zg) : gmma::hsub2_f16(a[r], (r & 1) ? zg8 : zg);
    }

    // Raw scales (two a word, f32: one) and zero points of the lane's row.
    struct Raw {
        uint32_t s[NB], z;
    };
    static __device__ __forceinline__ void raw(const Params& p, const RowScales& r, int c, Raw& v) {
        if (p.s_vec) {
            if constexpr (NB == 8) {
                const uint4 a = ldg_ahead(reinterpret_cast<const uint4*>(r.s) + c);
                v.s[0] = a.x;
                v.s[1] = a.y;
                v.s[2] = a.z;
                v.s[3] = a.w;
            } else if constexpr (NB == 4) {
                const uint2 a = ldg_ahead(reinterpret_cast<const uint2*>(r.s) + c);
                v.s[0] = a.x;
                v.s[1] = a.y;
            } else if constexpr (NB == 2) {
                v.s[0] = ldg_ahead(reinterpret_cast<const uint32_t*>(r.s) + c);
            } else {
                v.s[0] = ldg_ahead(reinterpret_cast<const uint16_t*>(r.s) + ((c * kDepth) >> p.bs_shift));
            }
        } else {
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const int b = (c * kDepth + j * 16 * SUB) >> p.bs_shift;
                uint32_t u = 0u;  // depths past the last block: scale 0
                if (b < p.a.KB) u = p.sdt == kF32 ? ldg_ahead(reinterpret_cast<const uint32_t*>(r.s) + b) : ldg_ahead(reinterpret_cast<const uint16_t*>(r.s) + b);
                if (p.sdt == kF32) v.s[j] = u;
                else v.s[j >> 1] = (j & 1) ? v.s[j >> 1] | (u << 16) : u;
            }
        }
        constexpr int ZBITS = NB * BITS;
        if (r.z == nullptr) {
            v.z = BITS == 2 ? 0xAAAAAAAAu : BITS == 4 ? 0x88888888u : 0x80808080u;  // 2^(bits - 1) in every field
        } else if (ZBITS >= 8 && p.z_vec) {
            if constexpr (ZBITS == 32) v.z = ldg_ahead(reinterpret_cast<const uint32_t*>(r.z) + c);
            else if constexpr (ZBITS == 16) v.z = ldg_ahead(reinterpret_cast<const uint16_t*>(r.z) + c);
            else v.z = ldg_ahead(r.z + c);
        } else {
            v.z = 0u;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const int b = min((c * kDepth + j * 16 * SUB) >> p.bs_shift, p.a.KB - 1) * BITS;
                v.z |= (((uint32_t)ldg_ahead(r.z + (b >> 3)) >> (b & 7)) & (uint32_t)((1 << BITS) - 1)) << (j * BITS);
            }
        }
    }

    // The lane's row into the warp's table: entry [row tile][j][g] = (scale, zero point as the codes' numbers) of rows g and g + 8.
    static __device__ __forceinline__ void table(int sdt, const Raw& v, uint2* tab) {
        const int lane = threadIdx.x & 31;
        uint2* dst = tab + (lane >> 4) * NB * 16 + (lane & 7) * 2 + ((lane >> 3) & 1);
        const uint32_t lift = ((lane & 8) ? kLift8 : 1) * 0x00010001u;
        auto put = [&](int j, float s) {
            dst[j * 16] = make_uint2(__float_as_uint(s), ((v.z >> (j * BITS)) & (uint32_t)((1 << BITS) - 1)) * lift);
        };
        if (sdt == kF16) {
#pragma unroll
            for (int j = 0; j < NB; ++j) put(j, __half2float(__ushort_as_half((unsigned short)((j & 1) ? v.s[j >> 1] >> 16 : v.s[j >> 1]))));
        } else if (sdt == kBF16) {
#pragma unroll
            for (int j = 0; j < NB; ++j) put(j, __uint_as_float((j & 1) ? v.s[j >> 1] & 0xFFFF0000u : v.s[j >> 1] << 16));
        } else {
#pragma unroll
            for (int j = 0; j < NB; ++j) put(j, __uint_as_float(v.s[j]));
        }
    }

    // Where piece `piece` of column `col` lies in a slot.
    static __device__ __forceinline__ uint32_t piece_at(int col, int piece) { return (uint32_t)(kWBytes + col * kColStride + piece * 16); }

    // y[m] += row tile m times the columns, in units of the codes' (times kColumnScale).  (Columns past the segment's hold
    // anything: their sums are not used.)
    static __device__ __forceinline__ void compute(uint32_t slot, const uint2* tab, float (&y)[2][4]) {
        constexpr int KG = BITS == 2 ? 8 : 4;  // k-steps of a turn: with all 8 unrolled the loads of a whole item come first and spill
        constexpr int TPG = KG / SPT;
        const int lane = threadIdx.x & 31;
        const float zero4[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t cols = slot + kWBytes + (lane & 7) * kColStride + (lane >> 3) * 16, mine = slot + lane * 16;
        const uint4* row = reinterpret_cast<const uint4*>(tab) + (lane >> 2);
        float acc[2][4];
        uint4 e[2];  // of the block: scale and zero point of rows g and g + 8
        if constexpr (SUB > KG) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                e[m] = row[m * NB * 8];
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[m][j] = 0.f;
            }
        }
        auto scale = [&] {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                y[m][0] = fmaf(__uint_as_float(e[m].x), acc[m][0], y[m][0]);
                y[m][1] = fmaf(__uint_as_float(e[m].x), acc[m][1], y[m][1]);
                y[m][2] = fmaf(__uint_as_float(e[m].z), acc[m][2], y[m][2]);
                y[m][3] = fmaf(__uint_as_float(e[m].z), acc[m][3], y[m][3]);
            }
        };
#pragma unroll 1
        for (int k0 = 0; k0 < KST; k0 += KG) {
            uint32_t x[KG / 2][4];
            uint4 w[2][TPG];
#pragma unroll
            for (int t = 0; t < TPG; ++t) {
                w[0][t] = lds16(mine + t * kTileBytes);
                w[1][t] = lds16(mine + (TPI + t) * kTileBytes);
            }
#pragma unroll
            for (int k = 0; k < KG; k += 2) ldmatrix4(x[k / 2], cols + k * 32);
            if constexpr (LIFT) {
#pragma unroll
                for (int k = 0; k < KG / 2; ++k) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(x[k][j]) : "r"(0x5D805D80u));  // 2^60
                }
            }
#pragma unroll
            for (int k = 0; k < KG; ++k) {
                if (SUB <= KG && k % SUB == 0) {
                    e[0] = row[k / SUB * 8];
                    e[1] = row[(NB + k / SUB) * 8];
                }
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    uint32_t a[4];
                    fragment(w[m][k / SPT], k % SPT, e[m].y, e[m].w, a);
                    const uint32_t b0 = x[k / 2][2 * (k & 1)], b1 = x[k / 2][2 * (k & 1) + 1];
                    if (SUB <= KG && k % SUB == 0) mma16816<BF>(acc[m], a, b0, b1, zero4);
                    else mma16816<BF>(acc[m], a, b0, b1, acc[m]);
                }
                if (SUB <= KG && k % SUB == SUB - 1) scale();
            }
            mine += TPG * kTileBytes;
            cols += KG * 32;
            if constexpr (SUB <= KG) row += KG / SUB * 8;
        }
        if constexpr (SUB > KG) scale();
    }

    // The sums as they are.
    static __device__ __forceinline__ void unscale(float (&y)[2][4]) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[m][j] *= j < 2 ? kUnscale : kUnscale / kLift8;
        }
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

// Start of part i of n things in `parts` parts that differ by at most one.
__device__ __forceinline__ int part_start(int n, int i, int parts) {
    const int q = n / parts;
    return q * i + min(i, n - q * parts);
}

// An item of a warp's run: its number, its unit and the unit's chunk.
struct Cursor {
    int i, u, c;
    __device__ __forceinline__ void next(int chunks) {
        ++i;
        if (++c == chunks) {
            c = 0;
            ++u;
        }
    }
};

template <int BITS, bool BF, int BSL>
__global__ void __launch_bounds__(kThreads, 2) gate_up_kernel(const __grid_constant__ Params p) {
    using It = Item<BITS, BF, BSL, BF>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kRingBytes);
    uint8_t* at = smem + kWarps * kRingBytes;
    uint2* tab = reinterpret_cast<uint2*>(at + warp * It::kTabBytes);
    at += kWarps * It::kTabBytes;
    float4* heads = reinterpret_cast<float4*>(at);  // [warp][gate, up][lane]: sums of the row tile that a run ends but did not begin
    at += kWarps * 2 * 32 * 16;
    const Lists L(at, p.r.T * p.r.S);

    griddep_wait();
    griddep_launch_dependents();
    make_lists(p, L, 8, reinterpret_cast<uint32_t*>(smem));
    const int slot_bytes = It::slot_bytes(*L.most), depth = min(4, kRingBytes / slot_bytes);

    const int KC = (p.a.K + It::kDepth - 1) / It::kDepth, NT = (int)p.a.row_tiles;
    const int units = *L.nseg * NT;
    const int u0 = part_start(units, blockIdx.x, gridDim.x), items = (part_start(units, blockIdx.x + 1, gridDim.x) - u0) * KC;
    const int i0 = part_start(items, warp, kWarps), i1 = part_start(items, warp + 1, kWarps);
    Cursor cur{i0, u0 + i0 / KC, i0 % KC};
    Cursor ahead = cur, next = cur;

    const int piece = lane % It::PC, col0 = lane / It::PC;
    const uint32_t to0 = It::piece_at(col0, piece);
    RowTiles tiles;
    Seg ls{0, 0, 0};
    const uint16_t* x0 = nullptr;
    int tiles_u = -1, scales_u = -1;
    // item `ahead` into a slot
    auto load = [&](uint32_t slot) {
        if (ahead.i < i1) {
            if (ahead.u != tiles_u) {
                tiles_u = ahead.u;
                const int sg = tiles_u / NT, rt = tiles_u - sg * NT;
                ls = L.seg[sg];
                tiles.set(p, ls.e, rt, rt);
                tiles.w0 += (int64_t)ahead.c * (It::TPI * kTileBytes);
                tiles.w1 += (int64_t)ahead.c * (It::TPI * kTileBytes);
                x0 = static_cast<const uint16_t*>(p.x) + L.token[ls.first + min(col0, ls.cnt - 1)] * p.x_stride;
            }
            It::weights(tiles.w0, tiles.w1, (int)p.a.k_tiles - ahead.c * It::TPI, slot);
            tiles.w0 += It::TPI * kTileBytes;
            tiles.w1 += It::TPI * kTileBytes;
            const int k = ahead.c * It::kDepth + piece * 8, left = p.a.K - k;
            if (p.x_wide) {
                const int bytes = left > 0 ? 16 : 0, from = left > 0 ? k : 0;  // (rows end on a whole vector)
                if (col0 < ls.cnt) cp_async16_part(slot + to0, x0 + from, bytes);
#pragma unroll 1
                for (int col = col0 + 32 / It::PC; col < ls.cnt; col += 32 / It::PC)
                    cp_async16_part(slot + It::piece_at(col, piece),
                                    static_cast<const uint16_t*>(p.x) + L.token[ls.first + col] * p.x_stride + from, bytes);
            } else {
#pragma unroll 1
                for (int col = col0; col < ls.cnt; col += 32 / It::PC) {
                    const uint16_t* x = static_cast<const uint16_t*>(p.x) + L.token[ls.first + col] * p.x_stride;
                    uint32_t v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t a = 2 * j < left ? x[k + 2 * j] : 0u, b = 2 * j + 1 < left ? x[k + 2 * j + 1] : 0u;
                        v[j] = a | (b << 16);
                    }
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(slot + It::piece_at(col, piece)), "r"(v[0]),
                                 "r"(v[1]), "r"(v[2]), "r"(v[3])
                                 : "memory");
                }
            }
            ahead.next(KC);
        }
        cp_commit();
    };
    RowScales rows;
    typename It::Raw raw;
    auto load_scales = [&] {
        if (next.i < i1) {
            if (next.u != scales_u) {
                scales_u = next.u;
                const int sg = scales_u / NT, rt = scales_u - sg * NT;
                rows.set(p, L.seg[sg].e, rt, rt);
            }
            It::raw(p, rows, next.c, raw);
            next.next(KC);
        }
    };

    float y[2][4];
    auto clear = [&] {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[m][j] = 0.f;
        }
    };
    auto put = [&](float4* to) {
#pragma unroll
        for (int m = 0; m < 2; ++m) to[m * 32 + lane] = make_float4(y[m][0], y[m][1], y[m][2], y[m][3]);
    };
    // a row tile's sums are complete: h of its rows
    auto finish = [&](int u) {
        const int sg = u / NT, rt = u - sg * NT;
        const Seg s = L.seg[sg];
        It::unscale(y);
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {  // (one at a time: four abreast need 30 registers more)
            const int col = 2 * (lane & 3) + (j & 1), row = rt * 16 + (lane >> 2) + 8 * (j >> 1);
            const float g = j == 0 ? y[0][0] : j == 1 ? y[0][1] : j == 2 ? y[0][2] : y[0][3];
            const float v0 = j == 0 ? y[1][0] : j == 1 ? y[1][1] : j == 2 ? y[1][2] : y[1][3];
            if (col < s.cnt) {
                const int pair = L.sorted[s.first + col];
                const float v = row < p.a.N ? activate(g, p.act) * v0 * L.w[pair] * kColumnScale : 0.f;
                const __nv_bfloat16 hi = __float2bfloat16_rn(v);
                const float rest = v - __bfloat162float(hi);  // exact; NaN beside an infinity
                uint16_t* dst = p.h + (int64_t)pair * 2 * p.inner + row;
                dst[0] = __bfloat16_as_ushort(hi);
                dst[p.inner] = isinf(__bfloat162float(hi)) ? 0 : __bfloat16_as_ushort(__float2bfloat16_rn(rest));
            }
        }
    };

    load_scales();
#pragma unroll 1
    for (int d = 0; d < depth; ++d) load(ring + d * slot_bytes);
    clear();
    const int first_u = cur.u, first_c = cur.c;
    const uint32_t last_slot = ring + (depth - 1) * slot_bytes;
    bool ends = false;  // the run ends a row tile that began in another
    uint32_t slot = ring;
#pragma unroll 1
    while (cur.i < i1) {
        cp_wait_oldest(depth);
        It::table(p.sdt, raw, tab);
        load_scales();
        __syncwarp();
        It::compute(slot, tab, y);
        __syncwarp();
        load(slot);
        slot = slot == last_slot ? ring : slot + slot_bytes;
        const int u = cur.u;
        cur.next(KC);
        if (cur.c == 0) {  // the row tile's last item
            if (u != first_u || first_c == 0) {
                finish(u);
            } else {
                put(heads + warp * 64);
                ends = true;
            }
            clear();
        }
    }
    cp_wait<0>();
    // the run that ends a row tile adds its parts in order
    auto rest = [&](int w) { return reinterpret_cast<float4*>(smem + w * kRingBytes); };  // of the row tile that a run leaves unended
    __syncwarp();
    if (i1 > i0 && cur.c != 0) put(rest(warp));
    __syncthreads();
    if (ends) {
        clear();
        const int start = (first_u - u0) * KC;  // the row tile's first item
        for (int w = 0; w <= warp; ++w) {
            const int w0 = part_start(items, w, kWarps), w1 = part_start(items, w + 1, kWarps);
            if (w1 <= start || w0 == w1) continue;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float4 v = (w < warp ? rest(w) : heads + warp * 64)[m * 32 + lane];
                y[m][0] += v.x;
                y[m][1] += v.y;
                y[m][2] += v.z;
                y[m][3] += v.w;
            }
        }
        finish(first_u);
    }
    if (blockIdx.x == 0)
        for (int i = tid; i < *L.nseg; i += kThreads) {
            check_headers(p, p.a, L.seg[i].e, BITS);
            check_headers(p, p.b, L.seg[i].e, BITS);
        }
}

template <int BITS, int BSL>
__global__ void __launch_bounds__(kThreads, 2) down_kernel(const __grid_constant__ Params p) {
    using It = Item<BITS, true, BSL, false>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kRingBytes);
    uint8_t* at = smem + kWarps * kRingBytes;
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
    make_lists(p, L, 4, reinterpret_cast<uint32_t*>(smem));
    const int slot_bytes = It::slot_bytes(2 * *L.most), depth = min(4, kRingBytes / slot_bytes);

    const int KC = ((int)p.inner + It::kDepth - 1) / It::kDepth;
    const int items = *L.nseg * KC, me = rank * kWarps + warp;
    const int i0 = part_start(items, me, C * kWarps), i1 = part_start(items, me + 1, C * kWarps);
    const int rt0 = 2 * group, rt1 = min(rt0 + 1, (int)p.a.row_tiles - 1);
    Cursor cur{i0, i0 / KC, i0 % KC};
    Cursor ahead = cur, next = cur, column = cur;
    RowTiles tiles;
    int tiles_u = -1, scales_u = -1, column_u = -1;
    auto load_weights = [&](uint32_t slot) {
        if (ahead.i < i1) {
            if (ahead.u != tiles_u) {
                tiles_u = ahead.u;
                tiles.set(p, L.seg[tiles_u].e, rt0, rt1);
                tiles.w0 += (int64_t)ahead.c * (It::TPI * kTileBytes);
                tiles.w1 += (int64_t)ahead.c * (It::TPI * kTileBytes);
            }
            It::weights(tiles.w0, tiles.w1, (int)p.a.k_tiles - ahead.c * It::TPI, slot);
            tiles.w0 += It::TPI * kTileBytes;
            tiles.w1 += It::TPI * kTileBytes;
            ahead.next(KC);
        }
    };
    // columns 2 j and 2 j + 1: the high and the low part of the segment's pair j
    const int piece = lane % It::PC, col0 = lane / It::PC;
    const uint32_t to0 = It::piece_at(col0, piece);
    const uint16_t* h0 = nullptr;
    Seg ls{0, 0, 0};
    auto load_columns = [&](uint32_t slot) {
        if (column.i < i1) {
            if (column.u != column_u) {
                column_u = column.u;
                ls = L.seg[column_u];
                h0 = p.h + ((int64_t)L.sorted[ls.first + min(col0 >> 1, ls.cnt - 1)] * 2 + (col0 & 1)) * p.inner;
            }
            const int k = column.c * It::kDepth + piece * 8, left = (int)p.inner - k;
            const int bytes = left > 0 ? 16 : 0, from = left > 0 ? k : 0;  // (rows of h are whole row tiles)
            if (col0 < 2 * ls.cnt) cp_async16_part(slot + to0, h0 + from, bytes);
#pragma unroll 1
            for (int col = col0 + 32 / It::PC; col < 2 * ls.cnt; col += 32 / It::PC)
                cp_async16_part(slot + It::piece_at(col, piece),
                                p.h + ((int64_t)L.sorted[ls.first + (col >> 1)] * 2 + (col & 1)) * p.inner + from, bytes);
            column.next(KC);
        }
    };
    RowScales rows;
    typename It::Raw raw;
    auto load_scales = [&] {
        if (next.i < i1) {
            if (next.u != scales_u) {
                scales_u = next.u;
                rows.set(p, L.seg[scales_u].e, rt0, rt1);
            }
            It::raw(p, rows, next.c, raw);
            next.next(KC);
        }
    };

    // the first items' weights before the wait for h (all in the first group), their columns after it
    load_scales();
#pragma unroll 1
    for (int d = 0; d < depth; ++d) load_weights(ring + d * slot_bytes);
    griddep_wait();
    griddep_launch_dependents();
#pragma unroll 1
    for (int d = 0; d < depth; ++d) {
        load_columns(ring + d * slot_bytes);
        cp_commit();
    }

    float y[2][4];
    auto clear = [&] {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[m][j] = 0.f;
        }
    };
    clear();
    float* mine = sums + warp * T * 32;
    const uint32_t last_slot = ring + (depth - 1) * slot_bytes;
    uint32_t slot = ring;
#pragma unroll 1
    while (cur.i < i1) {
        cp_wait_oldest(depth);
        It::table(p.sdt, raw, tab);
        load_scales();
        __syncwarp();
        It::compute(slot, tab, y);
        __syncwarp();
        load_weights(slot);
        load_columns(slot);
        cp_commit();
        slot = slot == last_slot ? ring : slot + slot_bytes;
        const int u = cur.u;
        cur.next(KC);
        if (cur.c == 0 || cur.i == i1) {
            // the segment ends: its pairs' high and low parts are added and go to their tokens' sums
            const Seg s = L.seg[u];
            It::unscale(y);
            if ((lane & 3) < s.cnt) {
                float* dst = mine + L.token[s.first + (lane & 3)] * 32 + (lane >> 2);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    dst[m * 16] += y[m][0] + y[m][1];
                    dst[m * 16 + 8] += y[m][2] + y[m][3];
                }
            }
            clear();
            __syncwarp();
        }
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

// The loads of an item's scales and zero points as one access, where a row's blocks come in whole items and aligned.
template <class It>
void set_vectors(Params& p, int bits) {
    auto all = [&](const void* a, const void* b, int n) { return dec::aligned_to(a, n) && dec::aligned_to(b, n); };
    const bool runs = It::NB == 1 || p.a.KB % It::NB == 0;
    p.s_vec = runs && p.sdt != kF32 && all(p.a.scales, p.b.scales, 2 * It::NB);
    p.z_vec = It::NB > 1 && runs && It::NB * bits >= 8 && all(p.a.zp, p.b.zp, It::NB * bits / 8);
}

template <int BITS, bool BF, int BSL>
cudaError_t launch_gate_up(Params p, cudaStream_t s) {
    using It = Item<BITS, BF, BSL, BF>;
    set_vectors<It>(p, BITS);
    auto kern = gate_up_kernel<BITS, BF, BSL>;
    const int P = p.r.T * p.r.S;
    const size_t smem = (size_t)kWarps * (kRingBytes + It::kTabBytes + 2 * 32 * 16) + Lists::bytes(P);
    const cudaError_t e = allow_shared(kern);
    if (e != cudaSuccess) return e;
    // two CTAs an SM; no more than the row tiles of the most experts that can be active
    const int64_t most = (int64_t)(P < p.r.E ? P : p.r.E) * p.a.row_tiles;
    const int grid = (int)(most < 2 * dec::kSms ? most : 2 * dec::kSms);
    return dec::launch_pdl(kern, dim3(grid), dim3(kThreads), smem, s, 1, p);
}

template <int BITS, int BSL>
cudaError_t launch_down(Params p, cudaStream_t s) {
    using It = Item<BITS, true, BSL, false>;
    set_vectors<It>(p, BITS);
    auto kern = down_kernel<BITS, BSL>;
    const size_t smem = (size_t)kWarps * (kRingBytes + It::kTabBytes + p.r.T * 32 * 4) + Lists::bytes(p.r.T * p.r.S);
    const cudaError_t e = allow_shared(kern);
    if (e != cudaSuccess) return e;
    const int64_t groups = (p.a.row_tiles + 1) / 2;
    // as many CTAs a group of 32 rows as two an SM hold, up to a portable cluster
    p.cluster = 1;
    while (p.cluster < 8 && groups * p.cluster * 2 <= 2 * dec::kSms) p.cluster *= 2;
    return dec::launch_pdl(kern, dim3((unsigned)(groups * p.cluster)), dim3(kThreads), smem, s, p.cluster, p);
}

template <int BITS, int BSL>
cudaError_t launch_block(const Params& g, const Params& d, int bf, cudaStream_t s) {
    const cudaError_t e = bf ? launch_gate_up<BITS, true, BSL>(g, s) : launch_gate_up<BITS, false, BSL>(g, s);
    return e == cudaSuccess ? launch_down<BITS, BSL>(d, s) : e;
}

// Blocks of 16, 32, 64, and 128 and more (8-bit codes: 64 and more, an item).
template <int BITS>
cudaError_t launch_bits(const Params& g, const Params& d, int bf, cudaStream_t s) {
    switch (g.bs_shift) {
        case 4: return launch_block<BITS, 0>(g, d, bf, s);
        case 5: return launch_block<BITS, 1>(g, d, bf, s);
        case 6: return launch_block<BITS, 2>(g, d, bf, s);
        default:
            if constexpr (BITS == 8) return launch_block<BITS, 2>(g, d, bf, s);
            else return launch_block<BITS, 3>(g, d, bf, s);
    }
}

}  // namespace moe
}  // namespace mnb
