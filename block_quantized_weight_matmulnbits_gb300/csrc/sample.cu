// mnb_sample: one token of each row of logits, by temperature, top-k, top-p and
// min-p from a given uniform number.
//
// With the tokens in descending order of their logits (equal ones by ascending
// index) and w_i = exp((x_i - max) / T), each cut keeps a start of that order,
// and the token drawn is the first whose sum of weights passes u times the sum
// of what is kept.  So a row needs sums of weights up to a place, not a sorted
// row.  A cluster of CTAs takes a row, each CTA a range of its tokens:
//
//   1. the range goes to shared memory (one pass over memory) with its maximum;
//   2. 2048 bins of equal width in max - x get the sums of their tokens' weights
//      (under top-k first their counts, which need no weights); the cluster adds
//      them and each CTA forms the prefix;
//   3. a place in the order (the k-th token, the share p, the draw) lies in one
//      bin: its tokens, or those of all bins up to it, if at most 1024, go to
//      the first CTA, which sorts them and takes their sums in order;
//   4. a bin with more of them is divided again, over the range of its values,
//      until it has few or one value, whose j-th token is counted out.
//
// A draw depends on sums of up to millions of weights next to a border, so the
// weights are integers: 2^-y, y = (max - x) / T * log2 e in two floats, from a
// table of 2^(-j / 1024) and a cubic of the rest (relative error below 2^-34).
// The unit goes by the bin: 2^-43 of the bin's octave (2^-(43 - extra) from 2^19
// tokens on), so a weight keeps its bits however small it is, and many equal ones
// do not lose them in one direction.  Sums inside a bin are exact, their prefix
// over the bins is kept in units of 2^-43 and a fraction of 32 bits and floored
// once; no order of atomics changes them.  So results repeat, and a sum up to a
// place is within 2^-33 of what is kept of its value: two roundings down of 2^-37
// at most, the weights' 2^-34, and 2^-36 for all weights past the last bin.
//
// Bound: the arithmetic of the weights and their bins (95 to 120 instructions a
// token), not the logits' bytes: 64 rows of 128000 f32 in 75 us (0.44 TB/s), 256 of
// 50257 f16 in 83, 16 of 200003 f32 in 41 (with one unit for all bins 70, 80 and
// 40: a third atomic addition for small weights).  Few rows: the barriers of a
// cluster, about 0.7 us each; one row of 128000 bf16 takes 15.9 us.
#include <algorithm>
#include <cmath>

#include "decoder.h"

namespace mnb {
namespace {

constexpr int kBins = 2048;
constexpr int kList = 1024;                            // tokens that the first CTA sorts
constexpr int kRankSort = 256;                         // up to so many by counting those before each
constexpr int kUnit = 43;                              // sums are in units of 2^-43 (2^extra times that) of the largest weight
constexpr int kTableUnit = 53;                         // the table's numbers in units of 2^-53
constexpr int kListUnit = 52;                          // weights of a list that spans bins: 1024 of them fit
constexpr int kAbreast = 4;                            // weights that a thread forms at a time
constexpr int kMaxVocab = 1 << 24;
constexpr int kGathers = 32;                           // of a row: 2 of nuclei, 3 of places with at most 4 divisions each

// 2^53 * 2^(-j / 1024), from the exponential series in double at compile time (good to 2^-50).
struct Table {
    unsigned long long v[1024];
    constexpr Table() : v() {
        for (int j = 0; j < 1024; ++j) {
            const double a = -0.693147180559945309417232121458 * j / 1024.0;
            double term = 1.0, sum = 1.0;
            for (int n = 1; n < 24; ++n) {
                term = term * a / n;
                sum += term;
            }
            v[j] = (unsigned long long)(sum * 9007199254740992.0 + 0.5);
        }
    }
};
__device__ const Table g_table = Table();

struct SampleParams {
    const void* logits;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    const float* u;
    int32_t* tokens;
    float* probs;
    int64_t stride;
    int V, C, seg, staged;
    int extra;  // sums lose this many bits, so that V weights fit 63
    int cut;    // octaves of the bins: weights below 2^-cut of the largest are left out
    int* status;
};

// ---- distributed shared memory ----
__device__ __forceinline__ uint32_t map_to(const void* p, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t ld_u32(const uint32_t* p, int rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_to(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ unsigned long long ld_u64(const unsigned long long* p, int rank) {
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(map_to(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_u32(uint32_t* p, int rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void st_u64(unsigned long long* p, int rank, unsigned long long v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(map_to(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t add_u32(uint32_t* p, int rank, uint32_t v) {
    uint32_t old;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(map_to(p, rank)), "r"(v) : "memory");
    return old;
}
__device__ __forceinline__ void min_u32(uint32_t* p, int rank, uint32_t v) {
    asm volatile("red.shared::cluster.min.u32 [%0], %1;" ::"r"(map_to(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void max_u32(uint32_t* p, int rank, uint32_t v) {
    asm volatile("red.shared::cluster.max.u32 [%0], %1;" ::"r"(map_to(p, rank)), "r"(v) : "memory");
}

// Floats in ascending order as unsigned integers (-0 as 0), and back.
__device__ __forceinline__ uint32_t key_of(float f) {
    const uint32_t u = __float_as_uint(f + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k); }

struct Scale {
    float top, c_hi, c_lo;  // maximum, log2 e / T in two floats
    float cut, per;         // largest max - x of a weight that counts, bins per unit of max - x
};

// 2^-y of a token, y = (top - x) c, in units of 2^-53 before a right shift.  (top is finite.)
__device__ __forceinline__ long long weight_parts(float x, const Scale& s, const unsigned long long* table, int& shift) {
    // d and its own rounding error (exact: d + e = top - x; top - x >= 0, so the larger of top and -x is so in magnitude)
    const float d = s.top - x;
    const float e = fminf(s.top, -x) - (d - fmaxf(s.top, -x));
    const float p = d * s.c_hi;
    const float rest = fmaf(e, s.c_hi, fmaf(d, s.c_lo, fmaf(d, s.c_hi, -p)));
    const float q = p + 12288.f;  // 1.5 * 2^13: p in units of 2^-10
    const int k = __float_as_int(q) - 0x46400000;
    const float z = (p - (q - 12288.f)) + rest;  // |z| <= 2^-11 and a little
    // 2^-z - 1 = -z ln 2 + (z ln 2)^2 / 2 - (z ln 2)^3 / 6, in units of 2^-42
    const float a = z * -0.69314718056f;
    const int f = __float2int_rn(fmaf(a * a, fmaf(a, 0.16666667f, 0.5f), a) * 4398046511104.f);
    const long long t = (long long)table[k & 1023];
    shift = k >> 10;
    return t + (((long long)(int)(t >> 23) * f) >> 19);  // (t / 2^53 in units of 2^-30) * f
}

// The weight of a token in a bin, in units of 2^-(52 - coarser), rounded.  (coarser may be negative where the shift makes up
// for it; a token in no bin gets anything.)
__device__ __forceinline__ unsigned long long weight_of(float x, const Scale& s, const unsigned long long* table, int coarser) {
    int shift;
    const unsigned long long t = (unsigned long long)weight_parts(x, s, table, shift);
    return ((t >> ((shift + coarser) & 63)) + 1ull) >> 1;
}

// v * 2^o, at most 2^63 - 1.
__device__ __forceinline__ unsigned long long shift_up(unsigned long long v, int o) {
    constexpr unsigned long long most = ~0ull >> 1;
    return v > most >> o ? most : v << o;
}

// 2^e for e from -126 to 127.
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((127 + e) << 23); }

// Bin of a token of max - x = d: equal widths, -1 for one that does not count (NaN too).
__device__ __forceinline__ int bin_of(float x, const Scale& s) {
    const float d = s.top - x;
    return d <= s.cut ? min(__float_as_int(fmaf(d, s.per, 8388608.f)) - 0x4B000000, kBins - 1) : -1;
}

// f * n for 0 <= f <= 1, exactly, rounded down (UP: up).  (Every thread forms it: in integers, as a few 64-bit floating
// point operations by all of them take microseconds on this part.)
template <bool UP>
__device__ __forceinline__ unsigned long long share_of(float f, unsigned long long n) {
    const uint32_t u = __float_as_uint(f) & 0x7FFFFFFFu, e = u >> 23;  // (-0 is 0)
    const unsigned long long m = e ? (u & 0x7FFFFFu) | 0x800000u : u & 0x7FFFFFu;
    const int s = 150 - (int)(e ? e : 1u);  // f = m / 2^s, s from 23 to 149
    const unsigned long long hi = __umul64hi(m, n), lo = m * n;
    unsigned long long q, rest;
    if (s < 64) {
        q = (hi << (64 - s)) | (lo >> s);
        rest = lo << (64 - s);
    } else {
        q = s < 128 ? hi >> (s - 64) : 0ull;
        rest = lo | (s < 128 ? hi & ((1ull << (s - 64)) - 1ull) : hi);
    }
    return UP && rest ? q + 1ull : q;
}

// Shared memory of a CTA, before its tokens.
struct Shared {
    unsigned long long table[1024];
    unsigned long long mw[kBins];  // the cluster's sums, then their prefix
    uint32_t mc[kBins];            // the cluster's counts, then their prefix
    union {
        struct {
            uint32_t cnt[kBins], lo[kBins], hi[kBins];  // this CTA's, while they are summed; lo: then the fractions of the cluster's
        };
        struct {
            unsigned long long list[kList];  // (order, index) of the cluster's gathered tokens (first CTA)
            unsigned long long sums[kList];  // this CTA's gathered tokens, then the prefix of the list's weights
        };
    };
    unsigned long long scan_w[32], scan_f[32];
    unsigned long long minp_w, res_w, found_w;
    uint32_t scan_c[32];
    uint32_t listed[kGathers];  // (first CTA) tokens of each gather
    uint32_t tops[8], ties[8];  // of each CTA: its largest key; its tokens of a value
    uint32_t mine, first_index, kmin, kmax, found, found2, res_token;
    float res_x;
    Scale scale;
};
// Other CTAs write the first one's list while it may still read the fractions in lo.
static_assert(sizeof(Shared::cnt) == sizeof(Shared::list), "the list must not reach lo");
static_assert(kBins == 2048, "octave() divides by it");

// The place of min-p among the bins: those before `lo` hold only weights above it, those after `hi` none.
struct MinP {
    float p;  // 0: none
    int lo, hi, oct;               // oct: octave of lo
    unsigned long long least;      // the smallest weight that is kept, in units of that octave
};

template <int DT, int THREADS>
struct Row {
    static constexpr int E = DT == kF32 ? 4 : 8;  // tokens of a 16-byte window
    const uint8_t* base;                           // first window (16-byte aligned)
    int windows, skip, n, first;                   // windows; tokens before the range in the first; tokens; index of the first token
    bool edges;                                    // the first and last windows hold other memory
    float mul, only;                               // what logits are multiplied by; 0: those equal to `only` count as 0, others as -inf

    __device__ __forceinline__ static void widen(const uint4& v, float (&x)[E]) {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == kF32) {
                x[i] = __uint_as_float(u[i]);
            } else if constexpr (DT == kBF16) {
                x[2 * i] = __uint_as_float(u[i] << 16);
                x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
            } else {
                const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
                x[2 * i] = h.x;
                x[2 * i + 1] = h.y;
            }
        }
    }
    // Window w, tokens outside the range as -inf.
    __device__ __forceinline__ uint4 raw(int w) const {
        if (!edges || (w * E >= skip && (w + 1) * E <= skip + n)) return *reinterpret_cast<const uint4*>(base + (size_t)w * 16);
        constexpr uint32_t none = DT == kF32 ? 0xFF800000u : DT == kBF16 ? 0xFF80u : 0xFC00u;
        uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const bool in = w * E + j >= skip && w * E + j < skip + n;
            if constexpr (DT == kF32) {
                u[j] = in ? reinterpret_cast<const uint32_t*>(base)[(size_t)w * E + j] : none;
            } else {
                const uint32_t h = in ? reinterpret_cast<const uint16_t*>(base)[(size_t)w * E + j] : none;
                u[j >> 1] |= h << (16 * (j & 1));
            }
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
    __device__ __forceinline__ void scale(float (&x)[E]) const {
        if (mul != 1.f) {
#pragma unroll
            for (int j = 0; j < E; ++j) x[j] = mul > 0.f ? x[j] * mul : x[j] == only ? 0.f : -INFINITY;
        }
    }
    __device__ __forceinline__ void values(int w, float (&x)[E]) const {
        widen(raw(w), x);
        scale(x);
    }
    // Every window of the thread, the next one loaded ahead (from L2 where the range is not in shared memory).
    template <class F>
    __device__ __forceinline__ void each_window(F&& f) const {
        int w = threadIdx.x;
        uint4 next = make_uint4(0, 0, 0, 0);
        if (w < windows) next = raw(w);
#pragma unroll 1
        while (w < windows) {
            const uint4 v = next;
            const int at = w;
            w += THREADS;
            if (w < windows) next = raw(w);
            float x[E];
            widen(v, x);
            scale(x);
            f(x, at * E);
        }
    }
    template <class F>
    __device__ __forceinline__ void each_few(F&& f) const {
        each_window([&](const float (&x)[E], int) {
#pragma unroll
            for (int j = 0; j < E; j += kAbreast) f(x + j);
        });
    }
    template <class F>
    __device__ __forceinline__ void each(F&& f) const {
        each_window([&](const float (&x)[E], int at) {
#pragma unroll
            for (int j = 0; j < E; ++j) f(x[j], at + j);
        });
    }
    __device__ __forceinline__ int index(int at) const { return first + at - skip; }
};

template <int DT, int THREADS>
struct Sampler {
    static constexpr int kWarps = THREADS / 32, kPer = kBins / THREADS;  // bins of a thread in the prefix
    Shared& S;
    const SampleParams& p;
    Row<DT, THREADS> row;
    Scale sc;
    int rank;
    int tid, lane, warp;
    MinP mp{};
    int gathers = 0;

    // The octave that the unit of a bin's weights goes by: no weight of the bin is below 2 octaves under it, none above it.
    __device__ __forceinline__ int octave(int b) const { return (max(b - 1, 0) * p.cut) >> 11; }
    __device__ __forceinline__ int coarser(int oct) const { return kListUnit - kUnit + p.extra - oct; }

    __device__ __forceinline__ void set_min_p(float min_p) {
        mp.p = 0.f;
        if (!(min_p > 0.f)) return;
        const float q = fminf(min_p, 1.f);
        // the bin of its place, or two where it is nearer to their border than the bins are exact (0.001)
        const float at = -log2f(q) * ((float)kBins / (float)p.cut);
        if (at > (float)kBins - 0.4f) return;  // all that counts is kept
        mp.p = q;
        mp.lo = max(__float2int_rn(at - 0.01f), 0);
        mp.hi = min(__float2int_rn(at + 0.01f), kBins - 1);
        mp.oct = octave(mp.lo);
        mp.least = share_of<true>(fminf(q * pow2f(mp.oct), 1.f), 1ull << (kUnit - p.extra));
    }
    // Whether min-p keeps a token in a bin.
    __device__ __forceinline__ bool keeps(float x) const {
        int shift;
        const unsigned long long t = (unsigned long long)weight_parts(x, sc, S.table, shift);
        const float least = mp.p * pow2f(shift);  // of t in units of 2^-53
        return least <= 2.f && t >= share_of<true>(0.5f * least, 2ull << kTableUnit);
    }

    __device__ __forceinline__ void sync() const {
        if (p.C > 1) cluster_sync();
        else __syncthreads();
    }

    // After the last gather: the others read the first CTA's counter, so its shared memory stays until they have.
    __device__ __forceinline__ void leave() const {
        __syncthreads();
        if (p.C > 1) cluster_sync();
    }

    // Bins' counts (CNT) and sums of weights (WGT) over the cluster, then their prefix in mc and mw.  bin(x) < 0: in none.
    // ALL: the bins by max - x, each summed in units of its octave, the prefix in those of octave 0; else bins of one
    // octave `oct`, whose units the prefix keeps.  MINP: minp_w gets the sum of what min-p keeps of the bins lo and hi.
    template <bool CNT, bool WGT, bool MINP, bool ALL, class B>
    __device__ __forceinline__ void histogram(B&& bin, int oct) {
        __syncthreads();
        for (int i = tid; i < kBins; i += THREADS) {
            S.cnt[i] = 0u;
            if (WGT) S.lo[i] = S.hi[i] = 0u;
        }
        if (MINP && tid == 0) S.minp_w = 0ull;
        __syncthreads();
        unsigned long long keep = 0ull;
        // Sums of weights: without counts and up to 65536 tokens a CTA as three sums of 16, 16 and the upper bits, which
        // nobody has to wait for; else of 32 bits with a carry.
        const bool three = !CNT && p.seg <= 65536;
        row.each_few([&](const float* x) {
            int b[kAbreast];
#pragma unroll
            for (int j = 0; j < kAbreast; ++j) {
                b[j] = bin(x[j]);
                if (CNT && b[j] >= 0) atomicAdd(&S.cnt[b[j]], 1u);
            }
            // weights abreast, without a branch: token by token would leave one chain of them at a time
            if constexpr (WGT) {
                unsigned long long w[kAbreast];
#pragma unroll
                for (int j = 0; j < kAbreast; ++j) w[j] = weight_of(x[j], sc, S.table, coarser(ALL ? octave(b[j]) : oct));
#pragma unroll
                for (int j = 0; j < kAbreast; ++j) {
                    if (b[j] < 0) continue;
                    if (MINP && b[j] >= mp.lo && b[j] <= mp.hi) {
                        const int finer = octave(b[j]) - mp.oct;
                        if (w[j] >= mp.least << finer) keep += w[j] >> finer;
                    }
                    const uint32_t lo = (uint32_t)w[j];
                    uint32_t hi = (uint32_t)(w[j] >> 32);
                    if (three) {
                        atomicAdd(&S.lo[b[j]], lo & 0xFFFFu);
                        atomicAdd(&S.cnt[b[j]], lo >> 16);
                    } else {
                        const uint32_t old = atomicAdd(&S.lo[b[j]], lo);
                        hi += old + lo < old ? 1u : 0u;
                    }
                    if (hi) atomicAdd(&S.hi[b[j]], hi);
                }
            }
        });
        if (MINP) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) keep += __shfl_xor_sync(0xFFFFFFFFu, keep, o);
            if (lane == 0) atomicAdd(&S.minp_w, keep);
        }
        if (p.C > 1) {
            cluster_sync();
            // each CTA adds a slice of the bins and hands it to all
            const int slice = kBins / p.C, b0 = rank * slice;
            for (int i = tid; i < slice; i += THREADS) {
                uint32_t c[8], lo[8], hi[8];  // (their loads are independent: a distributed one takes 0.3 us)
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    c[r] = (CNT || three) && r < p.C ? ld_u32(&S.cnt[b0 + i], r) : 0u;
                    lo[r] = WGT && r < p.C ? ld_u32(&S.lo[b0 + i], r) : 0u;
                    hi[r] = WGT && r < p.C ? ld_u32(&S.hi[b0 + i], r) : 0u;
                }
                uint32_t cs = 0;
                unsigned long long ws = 0;
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    if (CNT) cs += c[r];
                    ws += lo[r] + ((unsigned long long)(WGT && three ? c[r] : 0u) << 16) + ((unsigned long long)hi[r] << 32);
                }
                const int o = ALL ? octave(b0 + i) : 0;
                for (int r = 0; r < p.C; ++r) {
                    if (CNT) st_u32(&S.mc[b0 + i], r, cs);
                    if (WGT) st_u64(&S.mw[b0 + i], r, ws >> o);
                    if (WGT && ALL) st_u32(&S.lo[b0 + i], r, fraction(ws, o));  // (nobody else reads that bin's lo)
                }
            }
            unsigned long long all = 0;
            if (MINP && tid == 0) {
                for (int r = 0; r < p.C; ++r) all += ld_u64(&S.minp_w, r);
            }
            cluster_sync();
            if (MINP && tid == 0) S.minp_w = all;  // (every CTA has read the others' parts)
        } else {
            __syncthreads();
            for (int i = tid; i < kBins; i += THREADS) {
                if (CNT) S.mc[i] = S.cnt[i];
                if (WGT) {
                    const unsigned long long ws = S.lo[i] + ((unsigned long long)(three ? S.cnt[i] : 0u) << 16) + ((unsigned long long)S.hi[i] << 32);
                    const int o = ALL ? octave(i) : 0;
                    S.mw[i] = ws >> o;
                    if (ALL) S.lo[i] = fraction(ws, o);
                }
            }
            __syncthreads();
        }
        // inclusive prefix: kPer bins a thread
        constexpr bool FRAC = WGT && ALL;
        uint32_t c[kPer], cs = 0;
        unsigned long long w[kPer], ws = 0, f[kPer], fs = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (CNT) cs += S.mc[tid * kPer + i];
            c[i] = cs;
            if (WGT) ws += S.mw[tid * kPer + i];
            w[i] = ws;
            if (FRAC) fs += S.lo[tid * kPer + i];
            f[i] = fs;
        }
        uint32_t ci = cs;
        unsigned long long wi = ws, fi = fs;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t a = CNT ? __shfl_up_sync(0xFFFFFFFFu, ci, o) : 0u;
            const unsigned long long b = WGT ? __shfl_up_sync(0xFFFFFFFFu, wi, o) : 0ull;
            const unsigned long long d = FRAC ? __shfl_up_sync(0xFFFFFFFFu, fi, o) : 0ull;
            if (lane >= o) {
                ci += a;
                wi += b;
                fi += d;
            }
        }
        if (lane == 31) {
            S.scan_c[warp] = ci;
            S.scan_w[warp] = wi;
            S.scan_f[warp] = fi;
        }
        __syncthreads();
        uint32_t cb = ci - cs;
        unsigned long long wb = wi - ws, fb = fi - fs;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            if (CNT) cb += k < warp ? S.scan_c[k] : 0u;
            if (WGT) wb += k < warp ? S.scan_w[k] : 0ull;
            if (FRAC) fb += k < warp ? S.scan_f[k] : 0ull;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (CNT) S.mc[tid * kPer + i] = cb + c[i];
            if (WGT) S.mw[tid * kPer + i] = wb + w[i] + (FRAC ? (fb + f[i]) >> 32 : 0ull);
        }
        __syncthreads();
    }
    // What a sum in units of an octave has below the units of octave 0, in 32 bits.
    static __device__ __forceinline__ uint32_t fraction(unsigned long long w, int o) {
        return o ? (uint32_t)((w << (64 - o)) >> 32) : 0u;
    }

    // First bin whose prefix reaches `target` (-1: none does).
    template <bool COUNT>
    __device__ __forceinline__ int first_bin(unsigned long long target) {
        if (tid == 0) S.found = ~0u;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = tid * kPer + i;
            const unsigned long long upto = COUNT ? (unsigned long long)S.mc[b] : S.mw[b];
            const unsigned long long before = b == 0 ? 0ull : COUNT ? (unsigned long long)S.mc[b - 1] : S.mw[b - 1];
            if (upto >= target && before < target) S.found = (uint32_t)b;
        }
        __syncthreads();
        const int b = (int)S.found;
        __syncthreads();
        return b;
    }

    // About the most tokens that the bins up to b hold: each bin's sum over its least weight.  (gather() counts them.)
    __device__ __forceinline__ float most_tokens(int b) {
        float n = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int j = tid * kPer + i;
            // (a weight at the far edge, half a bin past its middle)
            const float w = (float)(S.mw[j] - (j ? S.mw[j - 1] : 0ull));
            if (j <= b) n += w * exp2f(((float)j + 0.5f) * ((float)p.cut / kBins) - (float)(kUnit - p.extra)) * 1.001f;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
        if (lane == 0) S.scan_w[warp] = __float_as_uint(n);
        __syncthreads();
        n = 0.f;
        for (int k = 0; k < kWarps; ++k) n += __uint_as_float((uint32_t)S.scan_w[k]);
        __syncthreads();
        return n;
    }

    // So many bins as a difference of max - x, and a little (bin b's values lie within half a bin of b / per; the last bin's
    // anywhere above).
    __device__ __forceinline__ float radius_of(int b, float bins) const { return b < kBins - 1 ? (bins + 0x1p-8f) / sc.per : INFINITY; }

    // The number of tokens with in(x); if it is at most kList, they are in the first CTA's list, sorted, with the prefix of
    // their weights (in units of 2^-(52 - coarser)).
    // Few windows have any: those without a token within `radius` of max - x = mid are passed over (in(x) implies that).
    template <class P>
    __device__ __forceinline__ int gather(P&& in, float mid, float radius, int coarser) {
        __syncthreads();
        if (tid == 0) S.mine = 0u;
        __syncthreads();
        uint32_t* const listed = &S.listed[min(gathers++, kGathers - 1)];
        row.each_window([&](const float (&x)[Row<DT, THREADS>::E], int at) {
            float near = INFINITY;
#pragma unroll
            for (int j = 0; j < Row<DT, THREADS>::E; ++j) near = fminf(near, fabsf((sc.top - x[j]) - mid));  // passes over NaN
            if (!(near <= radius)) return;
#pragma unroll
            for (int j = 0; j < Row<DT, THREADS>::E; ++j) {
                if (!in(x[j])) continue;
                // the lanes that found one take places together
                const uint32_t mask = __activemask();
                const int leader = __ffs(mask) - 1;
                uint32_t i = 0;
                if (lane == leader) i = atomicAdd(&S.mine, (uint32_t)__popc(mask));
                i = __shfl_sync(mask, i, leader) + __popc(mask & ((1u << lane) - 1u));
                if (i < kList) S.sums[i] = ((unsigned long long)(~key_of(x[j])) << 32) | (uint32_t)row.index(at + j);
            }
        });
        __syncthreads();
        const uint32_t mine = S.mine;
        if (p.C > 1) {
            if (tid == 0) S.found = mine ? add_u32(listed, 0, mine) : 0u;
            __syncthreads();
            const uint32_t at = S.found;
            for (uint32_t i = tid; i < mine && at + i < kList && i < kList; i += THREADS) st_u64(&S.list[at + i], 0, S.sums[i]);
            cluster_sync();
            if (tid == 0) S.found = ld_u32(listed, 0);
            __syncthreads();
        } else {
            for (uint32_t i = tid; i < mine && i < kList; i += THREADS) S.list[i] = S.sums[i];
            if (tid == 0) S.found = mine;
            __syncthreads();
        }
        const int n = (int)S.found;
        __syncthreads();
        if (n <= kList && rank == 0) sort(n, coarser);
        return n;
    }

    __device__ __forceinline__ void sort(int n, int coarser) {
        unsigned long long w[kList / THREADS], s = 0;
        if (n <= kRankSort) {
            // the place of a token is the number of those before it
            const unsigned long long v = tid < n ? S.list[tid] : ~0ull;
            int place = 0;
            if (tid < n) {
#pragma unroll 4
                for (int i = 0; i < n; ++i) place += S.list[i] < v ? 1 : 0;
            }
            __syncthreads();
            if (tid < n) S.list[place] = v;
            __syncthreads();
        } else {
            int size = 512;
            while (size < n) size *= 2;
            for (int i = n + tid; i < size; i += THREADS) S.list[i] = ~0ull;
            __syncthreads();
            for (int k = 2; k <= size; k *= 2) {
                for (int j = k / 2; j > 0; j /= 2) {
                    for (int t = tid; t < size / 2; t += THREADS) {
                        const int a = 2 * t - (t & (j - 1)), b = a + j;
                        const unsigned long long x = S.list[a], y = S.list[b];
                        if ((x > y) == ((a & k) == 0)) {
                            S.list[a] = y;
                            S.list[b] = x;
                        }
                    }
                    __syncthreads();
                }
            }
        }
        // the prefix of the weights: kList / THREADS tokens a thread
        constexpr int per = kList / THREADS;
#pragma unroll
        for (int i = 0; i < per; ++i) {
            const int at = per * tid + i;
            s += at < n ? weight_of(value_of(~(uint32_t)(S.list[at] >> 32)), sc, S.table, coarser) : 0ull;
            w[i] = s;
        }
        unsigned long long si = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long b = __shfl_up_sync(0xFFFFFFFFu, si, o);
            if (lane >= o) si += b;
        }
        if (lane == 31) S.scan_w[warp] = si;
        __syncthreads();
        unsigned long long before = si - s;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) before += k < warp ? S.scan_w[k] : 0ull;
#pragma unroll
        for (int i = 0; i < per; ++i) S.sums[per * tid + i] = before + w[i];
        __syncthreads();
    }

    // (first CTA) First place of the sorted list whose prefix reaches `target`; n - 1 if none does.
    __device__ __forceinline__ int first_listed(unsigned long long target, int n) {
        if (tid == 0) S.found2 = (uint32_t)(n - 1);
        __syncthreads();
        for (int at = tid; at < n; at += THREADS)
            if (S.sums[at] >= target && (at == 0 || S.sums[at - 1] < target)) S.found2 = (uint32_t)at;
        __syncthreads();
        const int at = (int)S.found2;
        __syncthreads();
        return at;
    }

    // (total: in units of 2^-unit)
    __device__ __forceinline__ void write(int64_t r, int token, float x, unsigned long long total, int unit) {
        if (tid != 0) return;
        p.tokens[r] = token;
        if (p.probs) {
            int shift;
            const double w = (double)weight_parts(x, sc, S.table, shift);
            p.probs[r] = (float)(w / (double)total * exp2i(unit - kTableUnit - shift));
        }
    }
    static __device__ __forceinline__ double exp2i(int e) { return __longlong_as_double((long long)(1023 + e) << 52); }

    // The token at a place of the order: the first whose prefix of counts (COUNT) or weights reaches `target`, which the
    // prefix in mc / mw of the bins by max - x does in bin `b`.  Every CTA gets the sum of weights up to it (found_w), the
    // first its index and logit.  True if the bins' prefixes were overwritten.  LAST: only the first CTA gets anything.
    template <bool COUNT, bool LAST>
    __device__ __forceinline__ bool resolve(int b, unsigned long long target) {
        b = max(b, 0);
        const int oct = octave(b);
        const unsigned long long base_w = b ? S.mw[b - 1] : 0ull;
        // what is left of the target inside the bin (weights in units of its octave), and the weights before what is looked into
        unsigned long long left = COUNT ? target - (b ? S.mc[b - 1] : 0u) : shift_up(target - base_w, oct), passed = 0ull;
        uint32_t kmin = 0u, kmax = ~0u;
        bool divided = false;
        __syncthreads();
        auto extent = [&](auto&& in) {  // lowest and highest key of the tokens in(x)
            if (tid == 0) {
                S.kmin = ~0u;
                S.kmax = 0u;
            }
            sync();
            uint32_t lo = ~0u, hi = 0u;
            row.each([&](float x, int) {
                if (!in(x)) return;
                lo = min(lo, key_of(x));
                hi = max(hi, key_of(x));
            });
            lo = __reduce_min_sync(0xFFFFFFFFu, lo);
            hi = __reduce_max_sync(0xFFFFFFFFu, hi);
            if (lane == 0) {
                for (int r = 0; r < p.C; ++r) {
                    if (p.C > 1) {
                        min_u32(&S.kmin, r, lo);
                        max_u32(&S.kmax, r, hi);
                    } else {
                        atomicMin(&S.kmin, lo);
                        atomicMax(&S.kmax, hi);
                    }
                }
            }
            sync();
            kmin = S.kmin;
            kmax = S.kmax;
            __syncthreads();
        };
        // (a NaN's key is above or below every number's, so x == x is asked)
        auto in = [&](float x) { return divided ? x == x && key_of(x) >= kmin && key_of(x) <= kmax : bin_of(x, sc) == b; };
        int m;
        while ((m = gather(in, divided ? 0.f : b / sc.per, divided ? INFINITY : radius_of(b, 0.5f), coarser(oct))) > kList) {
            if (!divided) extent(in);
            divided = true;
            if (kmin == kmax) break;
            const uint32_t k0 = kmin, k1 = kmax;
            const unsigned long long span = (unsigned long long)(k1 - k0) + 1ull;
            auto sub = [&](float x) {
                const uint32_t k = key_of(x);
                return x == x && k >= k0 && k <= k1 ? (int)((unsigned long long)(k1 - k) * kBins / span) : -1;
            };
            histogram<COUNT, true, false, false>(sub, oct);
            // (the prefix over the bins is floored, so what is left may be up to a unit more than the bin has: its last token)
            if (!COUNT) left = min(left, S.mw[kBins - 1]);
            const int f = max(first_bin<COUNT>(left), 0);  // (one always does)
            if (f) {
                left -= COUNT ? (unsigned long long)S.mc[f - 1] : S.mw[f - 1];
                passed += S.mw[f - 1];
            }
            extent([&](float x) { return sub(x) == f; });
        }
        if (m <= kList) {
            if (rank == 0) {
                const int at = COUNT ? min((int)left, m) - 1 : first_listed(left, m);
                if (tid == 0) {
                    S.res_w = base_w + ((passed + S.sums[at]) >> oct);
                    S.res_token = (uint32_t)S.list[at];
                    S.res_x = value_of(~(uint32_t)(S.list[at] >> 32));
                }
            }
        } else {
            // one value, more than fits the list: the j-th of its tokens
            const float x0 = value_of(kmin);
            const unsigned long long w = weight_of(x0, sc, S.table, coarser(oct));
            const unsigned long long j = COUNT ? left : min((left + w - 1) / w, (unsigned long long)m);  // from 1
            // a thread counts windows that follow each other
            const int per = (row.windows + THREADS - 1) / THREADS;
            const int w0 = min(tid * per, row.windows), w1 = min(w0 + per, row.windows);
            uint32_t c = 0;
            for (int i = w0; i < w1; ++i) {
                float x[Row<DT, THREADS>::E];
                row.values(i, x);
#pragma unroll
                for (int e = 0; e < Row<DT, THREADS>::E; ++e) c += in(x[e]) ? 1u : 0u;
            }
            uint32_t ci = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t a = __shfl_up_sync(0xFFFFFFFFu, ci, o);
                if (lane >= o) ci += a;
            }
            if (lane == 31) S.scan_c[warp] = ci;
            __syncthreads();
            uint32_t before = ci - c, all = 0;
            for (int k = 0; k < kWarps; ++k) {
                if (k < warp) before += S.scan_c[k];
                all += S.scan_c[k];
            }
            if (p.C > 1) {
                if (tid == 0)
                    for (int r = 0; r < p.C; ++r) st_u32(&S.ties[rank], r, all);
                cluster_sync();
                for (int r = 0; r < rank; ++r) before += S.ties[r];
            }
            if (j > before && j <= (unsigned long long)before + c) {
                uint32_t left = (uint32_t)(j - before);
                for (int i = w0; i < w1; ++i) {
                    float x[Row<DT, THREADS>::E];
                    row.values(i, x);
#pragma unroll
                    for (int e = 0; e < Row<DT, THREADS>::E; ++e)
                        if (in(x[e]) && --left == 0u) {
                            const uint32_t token = (uint32_t)row.index(i * Row<DT, THREADS>::E + e);
                            if (p.C > 1) st_u32(&S.res_token, 0, token);
                            else S.res_token = token;
                        }
                }
            }
            if (rank == 0 && tid == 0) {
                S.res_w = base_w + ((passed + j * w) >> oct);
                S.res_x = x0;
            }
        }
        if (LAST && m <= kList) {
            __syncthreads();
            return divided;
        }
        sync();
        if (LAST) return divided;
        if (tid == 0) S.found_w = p.C > 1 ? ld_u64(&S.res_w, 0) : S.res_w;
        sync();  // (the next resolve writes the first CTA's result)
        return divided;
    }
};

template <int DT, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) sample_kernel(const SampleParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared& S = *reinterpret_cast<Shared*>(smem);
    uint8_t* data = smem + (sizeof(Shared) + 15) / 16 * 16;
    constexpr int E = Row<DT, THREADS>::E, esize = 16 / E;
    const int tid = threadIdx.x;
    const int rank = p.C > 1 ? (int)cluster_ctarank() : 0;
    const int64_t r = blockIdx.x / p.C;
    for (int i = tid; i < 1024; i += THREADS) S.table[i] = g_table.v[i];
    if (tid < kGathers) S.listed[tid] = 0u;
    if (tid == 0) S.first_index = ~0u;
    if (p.C > 1) cluster_arrive();  // waited for before the first access to another CTA
    griddep_wait();
    griddep_launch_dependents();

    const float temperature = p.temperature ? p.temperature[r] : 1.f;
    const int top_k = p.top_k ? p.top_k[r] : 0;
    const float top_p = p.top_p ? p.top_p[r] : 1.f;
    const float min_p = p.min_p ? p.min_p[r] : 0.f;
    const float u = p.u[r];
    if (!(temperature >= 0.f) || !(top_p == top_p) || !(min_p == min_p) || !(u >= 0.f && u < 1.f)) {
        if (rank == 0 && tid == 0) {
            p.tokens[r] = -1;
            if (p.probs) p.probs[r] = 0.f;
            set_status(p.status, 1 /* MNB_ERR_INVALID_ARG */);
        }
        if (p.C > 1) cluster_wait();
        return;  // the whole cluster does
    }

    // Under a temperature near the ends of f32, differences of logits or log2 e / T would pass its range or be subnormal: both
    // are taken with a power of two.
    const float lift = temperature >= 0x1p64f ? 0x1p-64f : temperature < 0x1p-100f ? 0x1p64f : 1.f;
    if (tid == 0) {  // (64-bit floating point: by one thread, beside the loads)
        const double c = 1.4426950408889634 / ((double)temperature * (double)lift);
        S.scale.c_hi = (float)c;
        S.scale.c_lo = (float)(c - (double)S.scale.c_hi);
        S.scale.cut = fminf(__fdiv_rn((float)p.cut, S.scale.c_hi), 3.4e38f);
        S.scale.per = (float)kBins / S.scale.cut;
    }

    // ---- 1. the range, and the row's maximum ----
    Row<DT, THREADS> row;
    row.first = min(rank * p.seg, p.V);
    row.n = min(p.seg, p.V - row.first);
    const uint8_t* src = static_cast<const uint8_t*>(p.logits) + (size_t)(r * p.stride + row.first) * esize;
    row.base = reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(src) & ~uintptr_t(15));
    row.skip = (int)(src - row.base) / esize;
    row.windows = row.n > 0 ? (row.skip + row.n + E - 1) / E : 0;
    row.edges = true;
    row.mul = 1.f;
    row.only = 0.f;
    float top = -INFINITY;
    for (int w = tid; w < row.windows; w += THREADS) {
        const uint4 v = row.raw(w);
        if (p.staged) *reinterpret_cast<uint4*>(data + (size_t)w * 16) = v;
        float x[E];
        Row<DT, THREADS>::widen(v, x);
#pragma unroll
        for (int j = 0; j < E; ++j) top = fmaxf(top, x[j]);  // passes over NaN
    }
    if (p.staged) {
        row.base = data;
        row.edges = false;  // the ends hold -inf there
    }
    const uint32_t k = __reduce_max_sync(0xFFFFFFFFu, key_of(top));
    if ((tid & 31) == 0) S.scan_c[tid >> 5] = k;
    __syncthreads();
    if (tid < 32) {
        const uint32_t mine = __reduce_max_sync(0xFFFFFFFFu, tid < THREADS / 32 ? S.scan_c[tid] : 0u);
        if (p.C > 1) {
            cluster_wait();
            if (tid < p.C) st_u32(&S.tops[rank], tid, mine);
        } else if (tid == 0) {
            S.tops[0] = mine;
        }
    } else if (p.C > 1) {
        cluster_wait();
    }
    Sampler<DT, THREADS> q{S, p, row, {}, rank, tid, tid & 31, tid >> 5};
    q.sync();
    uint32_t best = S.tops[0];
    for (int c = 1; c < p.C; ++c) best = max(best, S.tops[c]);
    top = value_of(best);
    if (top == -INFINITY) {  // nothing can be drawn
        if (rank == 0 && tid == 0) {
            p.tokens[r] = -1;
            if (p.probs) p.probs[r] = 0.f;
        }
        return;
    }
    if (temperature == 0.f) {
        // the first token with the maximum
        uint32_t at = ~0u;
        row.each([&](float x, int i) {
            if (x == top) at = min(at, (uint32_t)row.index(i));
        });
        at = __reduce_min_sync(0xFFFFFFFFu, at);
        if ((tid & 31) == 0 && at != ~0u) {
            if (p.C > 1) min_u32(&S.first_index, 0, at);
            else atomicMin(&S.first_index, at);
        }
        q.sync();
        if (rank == 0 && tid == 0) {
            p.tokens[r] = (int32_t)S.first_index;
            if (p.probs) p.probs[r] = 1.f;
        }
        return;
    }
    q.sc = S.scale;
    q.sc.top = top * lift;
    q.row.mul = lift;
    if (isinf(q.sc.top)) {  // (of a finite maximum: nothing but its equals is near enough to weigh anything)
        q.row.mul = q.sc.top = 0.f;
        q.row.only = top;
    }

    // ---- 2. bins ----
    q.set_min_p(min_p);
    auto bin = [&](float x) { return bin_of(x, q.sc); };
    auto weigh = [&] {
        if (q.mp.p > 0.f) q.template histogram<false, true, true, true>(bin, 0);
        else q.template histogram<false, true, false, true>(bin, 0);
    };
    auto upto = [&](int last) {
        return [&, last](float x) { const int b = bin_of(x, q.sc); return b >= 0 && b <= last; };
    };
    bool by_k = top_k > 0 && top_k < p.V;
    int n = kList + 1;  // tokens of the list that holds all that can be kept
    unsigned long long total = 0ull, kept = 0ull, least = ~0ull;  // sums: of the top k, of what is kept; of what min-p keeps
    if (by_k) {
        q.template histogram<true, false, false, true>(bin, 0);
        const int b = q.template first_bin<true>((unsigned long long)top_k);
        if (b < 0) by_k = false;  // every token that counts is among the k
        else if (S.mc[b] <= (uint32_t)kList) n = q.gather(upto(b), 0.f, q.radius_of(b, b + 0.5f), 0);
    }
    if (n > kList) {
        weigh();
        if (q.mp.p > 0.f) least = (q.mp.lo ? S.mw[q.mp.lo - 1] : 0ull) + (S.minp_w >> q.mp.oct);
        total = S.mw[kBins - 1];
        bool whole = true;  // mw is that of the bins
        if (by_k) {
            whole = !q.template resolve<true, false>(q.template first_bin<true>((unsigned long long)top_k), (unsigned long long)top_k);
            total = S.found_w;
        }
        kept = total;
        if (top_p < 1.f) {
            const unsigned long long target = max(share_of<true>(fmaxf(top_p, 0.f), total), 1ull);
            if (!whole) weigh();
            whole = true;
            const int b = q.template first_bin<false>(target);
            // a nucleus that fits the list: all of it, and the draw from it
            if (q.most_tokens(b) <= (float)kList) n = q.gather(upto(b), 0.f, q.radius_of(b, b + 0.5f), 0);
            if (n > kList) {
                whole = !q.template resolve<false, false>(b, target);
                kept = S.found_w;
            }
        }
        if (n > kList) {
            kept = min(kept, least);
            const unsigned long long target = share_of<false>(u, kept) + 1ull;
            if (!whole) weigh();
            q.template resolve<false, true>(q.template first_bin<false>(target), target);
            if (rank == 0) q.write(r, (int)S.res_token, S.res_x, kept, kUnit - p.extra);
            q.leave();
            return;
        }
    }

    // ---- 3. all that can be kept is in the list ----
    if (rank == 0) {
        // (its weights are finer than the sums of the bins, which a nucleus that was found among those goes by)
        const bool all = total == 0ull;
        kept = S.sums[min(all ? top_k : n, n) - 1];
        if (top_p < 1.f) {
            const unsigned long long target = max(share_of<true>(fmaxf(top_p, 0.f), all ? kept : total), 1ull);
            kept = S.sums[q.first_listed(all ? target : shift_up(target, kListUnit - kUnit + p.extra), n)];
        }
        if (min_p > 0.f) {  // weights descend along the list: the sum before the first that is not kept
            q.mp.p = fminf(min_p, 1.f);
            if (tid == 0) S.mine = (uint32_t)n;
            __syncthreads();
            for (int at = tid; at < n; at += THREADS)
                if (!q.keeps(value_of(~(uint32_t)(S.list[at] >> 32)))) atomicMin(&S.mine, (uint32_t)at);
            __syncthreads();
            kept = min(kept, S.sums[max((int)S.mine, 1) - 1]);
        }
        const unsigned long long target = share_of<false>(u, kept) + 1ull;
        const int at = q.first_listed(target, n);
        q.write(r, (int)(uint32_t)S.list[at], value_of(~(uint32_t)(S.list[at] >> 32)), kept, kListUnit);
    }
    q.leave();
}

template <int DT, int THREADS>
cudaError_t launch_threads(SampleParams p, int64_t rows, cudaStream_t s) {
    constexpr int esize = DT == kF32 ? 4 : 2;
    const size_t fixed = (sizeof(Shared) + 15) / 16 * 16;
    size_t bytes = ((size_t)p.seg * esize + 15) / 16 * 16 + 16;
    // a range in shared memory where two CTAs of 512 threads (one of 1024) still fit an SM; else the passes read L2
    p.staged = fixed + bytes <= (THREADS == 512 ? device_info().smem_optin / 2 - 1024 : device_info().smem_optin);
    if (!p.staged) bytes = 0;
    auto kern = sample_kernel<DT, THREADS>;
    const cudaError_t e = allow_shared(kern);
    if (e != cudaSuccess) return e;
    return dec::launch_pdl(kern, dim3((unsigned)(rows * p.C)), dim3(THREADS), fixed + bytes, s, p.C, p);
}

template <int DT>
cudaError_t launch_sample(SampleParams p, int64_t rows, cudaStream_t s) {
    // CTAs a row: as many as the SMs hold at two an SM, up to a portable cluster, none with fewer than 2048 tokens
    p.C = 1;
    while (p.C < 8 && rows * p.C * 2 <= 2 * dec::kSms && p.V > p.C * 2048) p.C *= 2;
    p.seg = ((p.V + p.C - 1) / p.C + 7) / 8 * 8;
    // CTAs for at most half the SMs: 1024 threads each; more: 512, of which an SM holds two (both within 64 registers, with
    // about 270 bytes of spills).  Between a half and all of the SMs each has one CTA of 512.
    return rows * p.C <= dec::kSms / 2 ? launch_threads<DT, 1024>(p, rows, s) : launch_threads<DT, 512>(p, rows, s);
}

}  // namespace
}  // namespace mnb

using namespace mnb;

extern "C" {

mnb_status mnb_sample(const mnb_sample_args* a) {
    if (!a || a->B < 0 || a->V < 1 || !dec::valid_dt(a->dtype)) return MNB_ERR_INVALID_ARG;
    if (a->B > 1 && (a->row_stride < a->V || a->row_stride >= (int64_t(1) << 38))) return MNB_ERR_INVALID_ARG;
    if (a->V > kMaxVocab || a->B >= (int64_t(1) << 28)) return MNB_ERR_UNSUPPORTED;
    if (a->B == 0) return MNB_OK;
    if (!a->logits || !a->u || !a->tokens || !dec::aligned_to(a->logits, dec::dt_bytes(a->dtype)) || !dec::aligned_to(a->u, 4) ||
        !dec::aligned_to(a->tokens, 4) || !dec::aligned_to(a->probs, 4) || !dec::aligned_to(a->temperature, 4) ||
        !dec::aligned_to(a->top_k, 4) || !dec::aligned_to(a->top_p, 4) || !dec::aligned_to(a->min_p, 4))
        return MNB_ERR_INVALID_ARG;
    SampleParams p{};
    p.status = device_status_word();
    if (!p.status) return dec::status_of(cudaErrorUnknown);
    p.logits = a->logits;
    p.temperature = a->temperature;
    p.top_k = a->top_k;
    p.top_p = a->top_p;
    p.min_p = a->min_p;
    p.u = a->u;
    p.tokens = a->tokens;
    p.probs = a->probs;
    p.V = (int)a->V;
    p.stride = a->B > 1 ? a->row_stride : a->V;
    while (((int64_t)p.V >> p.extra) >= (1 << 19)) ++p.extra;  // V * 2^(43 - extra) below 2^63
    p.cut = 36;  // V weights of 2^-cut are below 2^-36
    while ((int64_t(1) << (p.cut - 36)) < p.V) ++p.cut;
    p.cut = std::max(p.cut, 44);
    if (inject_launch_failure()) return MNB_ERR_CUDA;
    const cudaStream_t s = (cudaStream_t)a->stream;
    ProfileScope prof("mnb_sample", s);
    cudaError_t e;
    switch (a->dtype) {
        case MNB_F32: e = launch_sample<kF32>(p, a->B, s); break;
        case MNB_F16: e = launch_sample<kF16>(p, a->B, s); break;
        default: e = launch_sample<kBF16>(p, a->B, s); break;
    }
    if (e == cudaSuccess) prof.done("sample");
    return dec::status_of(e);
}

}  // extern "C"
