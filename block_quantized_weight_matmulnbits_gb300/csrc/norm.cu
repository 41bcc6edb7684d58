// mnb_rms_norm: the residual's addition, the root-mean-square norm of the sum
// and, if wanted, its int8 codes with a scale for each block of a row:
//
//   s = x + r,   y = s * rsqrt(mean(s^2) + eps) * gain,   q = round(y / a), a = max |y| / 127
//
// One pass: a CTA holds its row's sums in registers (up to 4 vectors of 16
// bytes a thread, 8 for f32) between the sum of squares and the outputs, so x
// and r are read once and every output is written once; about six flops a value,
// so the bytes bound it.  Sums are f32: a thread's own in order, then a shuffle
// tree, then the warps' in order, so results repeat.  A block's maximum is a
// shuffle over its lanes (blocks up to a warp's 32 vectors) or an integer
// maximum in shared memory (larger ones), on the bits of |y|: a NaN is the
// largest of all and reaches the block's scale.
//
// Measured: 4999 rows of 5120 f16 with a residual 38.6 us (5300 GB/s, 0.78 of a
// copy); 16384 rows of 4096 bf16 to codes of blocks of 32 in 98 us (4880 GB/s),
// bound there by instructions (36 a value) and by 32 warps an SM (with 80 and 128 registers a
// thread instead of 64, so 24 and 16 warps: 108 and 127 us); 64 rows
// of 8192 2.7 us, a launch and one chain of load, reduction and store.
#include <algorithm>
#include <cmath>

#include "decoder.h"

namespace mnb {
namespace {

struct NormParams {
    const void* x;
    const void* r;
    const void* w;
    void* s_out;
    void* y;
    int8_t* codes;
    float* scales;
    int64_t rows, x_st, r_st, s_st, y_st;
    int width, padded;  // values of a row; the same with the last block filled up (codes)
    int bs_shift;       // log2 of the block (codes)
    int blocks;         // of a row
    int w_dt, y_dt;
    float eps, inv_width, offset;  // of the gain: 0 or 1
};

template <int DT> struct Elem { using T = uint16_t; };
template <> struct Elem<kF32> { using T = float; };

template <int DT, int V>
__device__ __forceinline__ void widen(const uint4& raw, float (&f)[V]) {
    const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == kF32) {
            f[i] = __uint_as_float(u[i]);
        } else if constexpr (DT == kBF16) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        } else {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
}

template <int DT, int V>
__device__ __forceinline__ uint4 narrow(const float (&f)[V]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == kF32) {
            u[i] = __float_as_uint(f[i]);
        } else if constexpr (DT == kBF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// V values at p + i of a row of n (type DT); WIDE: one 16-byte access, i + V <= n or i >= n.
template <int DT, int V, bool WIDE>
__device__ __forceinline__ void load_row(const void* p, int64_t at, int i, int n, float (&f)[V]) {
    if constexpr (WIDE) {
        const uint4 raw = i < n ? *reinterpret_cast<const uint4*>(static_cast<const typename Elem<DT>::T*>(p) + at + i)
                                : make_uint4(0, 0, 0, 0);
        widen<DT, V>(raw, f);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = i + j < n ? load_f32(p, at + i + j, DT) : 0.f;
    }
}

// Stores V values as type dt (the row's own type in one access when WIDE).
template <int DT, int V, bool WIDE>
__device__ __forceinline__ void store_row(void* p, int dt, int64_t at, int i, int n, const float (&f)[V]) {
    if (i >= n) return;
    if (WIDE && dt == DT) {
        *reinterpret_cast<uint4*>(static_cast<typename Elem<DT>::T*>(p) + at + i) = narrow<DT, V>(f);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (i + j < n) store_f32(p, at + i + j, f[j], dt);
    }
}

__device__ __forceinline__ float max_or_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
// 1 / a to 2^-23 for normal a and 1 / a.
__device__ __forceinline__ float recip(float a) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
}

template <int DT, int VPT, bool WIDE>
__global__ void __launch_bounds__(1024) rms_norm_kernel(NormParams p) {
    constexpr int V = DT == kF32 ? 4 : 8;
    extern __shared__ uint32_t amax_s[];  // [2][blocks] of blocks wider than a warp
    __shared__ float part[2][32];
    const int tid = threadIdx.x, lane = tid & 31, warps = blockDim.x >> 5;
    const bool wide_blocks = p.codes && (1 << p.bs_shift) > 32 * V;
    int parity = 0;
    if (wide_blocks) {
        for (int i = tid; i < 2 * p.blocks; i += blockDim.x) amax_s[i] = 0u;
    }
    griddep_wait();
    griddep_launch_dependents();
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, parity ^= 1) {
        float s[VPT][V];
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            load_row<DT, V, WIDE>(p.x, row * p.x_st, (k * blockDim.x + tid) * V, p.width, s[k]);
        if (p.r) {
            float r[VPT][V];
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                load_row<DT, V, WIDE>(p.r, row * p.r_st, (k * blockDim.x + tid) * V, p.width, r[k]);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
#pragma unroll
                for (int j = 0; j < V; ++j) s[k][j] += r[k][j];
            }
        }
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
#pragma unroll
            for (int j = 0; j < V; ++j) sum = fmaf(s[k][j], s[k][j], sum);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (lane == 0) part[parity][tid >> 5] = sum;
        __syncthreads();
        // the sum as stored may take the place of x or r: every thread has read its own values above
        if (p.s_out) {
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                store_row<DT, V, WIDE>(p.s_out, DT, row * p.s_st, (k * blockDim.x + tid) * V, p.width, s[k]);
        }
        sum = lane < warps ? part[parity][lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float rs = __frsqrt_rn(fmaf(sum, p.inv_width, p.eps));
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int i = (k * blockDim.x + tid) * V;
            float g[V];
            if (p.w) {
                if (WIDE && p.w_dt == DT) {
                    load_row<DT, V, WIDE>(p.w, 0, i, p.width, g);
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j) g[j] = i + j < p.width ? load_f32(p.w, i + j, p.w_dt) : 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s[k][j] *= rs;
                if (p.w) s[k][j] *= g[j] + p.offset;
            }
            if (p.y) store_row<DT, V, WIDE>(p.y, p.y_dt, row * p.y_st, i, p.width, s[k]);
        }
        if (!p.codes) continue;
        uint32_t* const am = amax_s + parity * p.blocks;
        uint32_t top[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            float most = 0.f;
            const int i = (k * blockDim.x + tid) * V;
#pragma unroll
            for (int j = 0; j < V; ++j)  // (values past the row are zeros)
                most = max_or_nan(most, fabsf(s[k][j]));
            top[k] = __float_as_uint(most) & 0x7FFFFFFFu;
            if (!wide_blocks) {
                // a block is an aligned group of bs / V lanes
                for (int o = 1; o < (1 << p.bs_shift) / V; o <<= 1) top[k] = max(top[k], __shfl_xor_sync(0xFFFFFFFFu, top[k], o));
            } else {
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) top[k] = max(top[k], __shfl_xor_sync(0xFFFFFFFFu, top[k], o));
                if (lane == 0 && i < p.padded) atomicMax(&am[i >> p.bs_shift], top[k]);
            }
        }
        if (wide_blocks) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int i = (k * blockDim.x + tid) * V;
                if (i < p.padded) top[k] = am[i >> p.bs_shift];
            }
            // the other half is clear again before the next row's maxima: its readers are past two barriers
            for (int i = tid; i < p.blocks; i += blockDim.x) amax_s[(parity ^ 1) * p.blocks + i] = 0u;
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int i = (k * blockDim.x + tid) * V;
            if (i >= p.padded) continue;
            // an infinity or NaN in the block: its scale is NaN and its codes are 0
            const bool bad = top[k] >= 0x7F800000u;
            const float a = bad ? __uint_as_float(0x7FC00000u) : __fdiv_rn(__uint_as_float(top[k]), 127.0f);
            if ((i & ((1 << p.bs_shift) - 1)) == 0) p.scales[row * p.blocks + (i >> p.bs_shift)] = a;
            uint32_t word[V / 4];
            if (!(a > 0.f)) {
#pragma unroll
                for (int j = 0; j < V / 4; ++j) word[j] = 0u;
            } else {
                // y / a rounded half away from zero: by the reciprocal (127 times its 2^-23 and the quotient's own rounding
                // are below 2^-15 of a step), which matters only beside a half, where the division decides, as it does for
                // scales without a normal reciprocal.  The sum with 1.5 * 2^23 has the code in its low byte.
                const float r = recip(a);
                uint32_t code[V];
                float off = 0.f;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float m = fmaf(s[k][j], r, 12582912.f);
                    off = fmaxf(off, fabsf(fmaf(s[k][j], r, 12582912.f - m)));
                    code[j] = __float_as_uint(m);
                }
                const bool near = off > 0.49993f || a < 0x1p-100f;
                if (near) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float q = roundf(__fdiv_rn(s[k][j], a));
                        code[j] = (uint32_t)(int)fminf(fmaxf(q, -127.f), 127.f);
                    }
                }
#pragma unroll
                for (int j = 0; j < V; j += 4)
                    word[j >> 2] = __byte_perm(__byte_perm(code[j], code[j + 1], 0x0040), __byte_perm(code[j + 2], code[j + 3], 0x0040), 0x5410);
            }
            int8_t* dst = p.codes + row * p.padded + i;  // padded is a multiple of 16, codes 16-byte aligned
            if constexpr (V == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(word[0], word[1]);
            else *reinterpret_cast<uint32_t*>(dst) = word[0];
        }
    }
}

template <int DT, int VPT>
cudaError_t launch_vpt(const NormParams& p, int threads, bool wide, cudaStream_t s) {
    // CTAs of 2048 threads an SM; half of them are resident at 64 registers (1024 to 16384 threads an SM take the same time)
    const int64_t fit = std::max(1, 2048 / threads) * (int64_t)dec::kSms;
    const unsigned grid = (unsigned)std::min<int64_t>(p.rows, fit);
    constexpr int V = DT == kF32 ? 4 : 8;
    const size_t smem = p.codes && (1 << p.bs_shift) > 32 * V ? (size_t)p.blocks * 8 : 0;
    return wide ? dec::launch_pdl(rms_norm_kernel<DT, VPT, true>, dim3(grid), dim3(threads), smem, s, 1, p)
                : dec::launch_pdl(rms_norm_kernel<DT, VPT, false>, dim3(grid), dim3(threads), smem, s, 1, p);
}

template <int DT>
cudaError_t launch_norm(const NormParams& p, bool wide, cudaStream_t s) {
    constexpr int V = DT == kF32 ? 4 : 8;
    const int vecs = ((p.codes ? p.padded : p.width) + V - 1) / V;
    // few rows: as many threads as a row has vectors, up to 1024 (one round trip of loads); many: up to 4 vectors a thread,
    // so that fewer threads wait at the barrier of a row (16384 rows of 4096 to codes: 98 us with 128 threads, 111 with
    // 256, 148 with 512; 4999 rows of 5120: 38.5, 38.5, 41.5)
    const int want = p.rows <= 2 * dec::kSms ? 1024 : 128;
    int vpt = 1;
    while (vpt < (DT == kF32 ? 8 : 4) && vecs > vpt * want) vpt *= 2;
    const int threads = std::min(1024, ((vecs + vpt - 1) / vpt + 31) / 32 * 32);
    switch (vpt) {
        case 1: return launch_vpt<DT, 1>(p, threads, wide, s);
        case 2: return launch_vpt<DT, 2>(p, threads, wide, s);
        case 4: return launch_vpt<DT, 4>(p, threads, wide, s);
        default:
            if constexpr (DT == kF32) return launch_vpt<DT, 8>(p, threads, wide, s);
            return cudaErrorNotSupported;
    }
}

constexpr int64_t kMaxWidth = 32768;  // 1024 threads of 4 vectors of 8 (f32: 8 of 4)

}  // namespace
}  // namespace mnb

using namespace mnb;

extern "C" {

mnb_status mnb_rms_norm(const mnb_rms_norm_args* a) {
    if (!a || a->T < 0 || a->width < 1 || !dec::valid_dt(a->dtype) || !(a->eps >= 0.f) || std::isinf(a->eps) ||
        (a->flags & ~MNB_NORM_UNIT_OFFSET) != 0)
        return MNB_ERR_INVALID_ARG;
    if (a->weight && !dec::valid_dt(a->weight_dtype)) return MNB_ERR_INVALID_ARG;
    if (a->y && !dec::valid_dt(a->out_dtype)) return MNB_ERR_INVALID_ARG;
    if (a->residual_out && !a->residual) return MNB_ERR_INVALID_ARG;
    if ((a->codes != nullptr) != (a->scales != nullptr)) return MNB_ERR_INVALID_ARG;
    if (a->codes && (!dec::pow2(a->block_size) || a->block_size < 16)) return MNB_ERR_INVALID_ARG;
    if (a->T == 0) return MNB_OK;
    if (a->width > kMaxWidth) return MNB_ERR_UNSUPPORTED;
    // a stride along one row steps nowhere
    const bool many = a->T > 1;
    const int64_t st[4] = {many ? a->x_stride : a->width, many && a->residual ? a->residual_stride : a->width,
                           many && a->residual_out ? a->residual_out_stride : a->width, many && a->y ? a->y_stride : a->width};
    for (int64_t v : st)
        if (v < a->width || v >= (int64_t(1) << 38)) return MNB_ERR_INVALID_ARG;
    const int eb = dec::dt_bytes(a->dtype);
    if (!a->x || (!a->y && !a->codes && !a->residual_out)) return MNB_ERR_INVALID_ARG;
    if (!dec::aligned_to(a->x, eb) || !dec::aligned_to(a->residual, eb) || !dec::aligned_to(a->residual_out, eb) ||
        (a->weight && !dec::aligned_to(a->weight, dec::dt_bytes(a->weight_dtype))) ||
        (a->y && !dec::aligned_to(a->y, dec::dt_bytes(a->out_dtype))) || !dec::aligned_to(a->codes, 16) ||
        !dec::aligned_to(a->scales, 4))
        return MNB_ERR_INVALID_ARG;
    // an output in an input's place has its values where the input's are
    if (a->y && ((a->y == a->x && (a->out_dtype != a->dtype || st[3] != st[0])) ||
                 (a->y == a->residual && (a->out_dtype != a->dtype || st[3] != st[1]))))
        return MNB_ERR_INVALID_ARG;
    if (a->residual_out && ((a->residual_out == a->x && st[2] != st[0]) || (a->residual_out == a->residual && st[2] != st[1])))
        return MNB_ERR_INVALID_ARG;
    if (a->T >= (int64_t(1) << 38)) return MNB_ERR_UNSUPPORTED;

    NormParams p{};
    p.x = a->x;
    p.r = a->residual;
    p.w = a->weight;
    p.s_out = a->residual_out;
    p.y = a->y;
    p.codes = a->codes;
    p.scales = a->scales;
    p.rows = a->T;
    p.x_st = st[0];
    p.r_st = st[1];
    p.s_st = st[2];
    p.y_st = st[3];
    p.width = (int)a->width;
    p.padded = p.width;
    if (a->codes) {
        const int64_t bs = a->block_size;
        p.blocks = (int)((a->width + bs - 1) / bs);
        if (bs * p.blocks >= (int64_t(1) << 31)) return MNB_ERR_UNSUPPORTED;
        while ((int64_t(1) << p.bs_shift) < bs) ++p.bs_shift;
        p.padded = (int)(bs * p.blocks);
        if (p.padded > kMaxWidth) return MNB_ERR_UNSUPPORTED;
    }
    p.w_dt = a->weight_dtype;
    p.y_dt = a->out_dtype;
    p.offset = (a->flags & MNB_NORM_UNIT_OFFSET) ? 1.f : 0.f;
    p.eps = a->eps;
    p.inv_width = 1.0f / (float)a->width;
    // 16-byte accesses where every row of the type's own arrays allows them
    const int V = 16 / eb;
    bool wide = a->width % V == 0 && dec::aligned_to(a->x, 16) && p.x_st % V == 0;
    if (a->residual) wide = wide && dec::aligned_to(a->residual, 16) && p.r_st % V == 0;
    if (a->residual_out) wide = wide && dec::aligned_to(a->residual_out, 16) && p.s_st % V == 0;
    if (a->y && a->out_dtype == a->dtype) wide = wide && dec::aligned_to(a->y, 16) && p.y_st % V == 0;
    if (a->weight && a->weight_dtype == a->dtype) wide = wide && dec::aligned_to(a->weight, 16);
    if (inject_launch_failure()) return MNB_ERR_CUDA;
    const cudaStream_t s = (cudaStream_t)a->stream;
    ProfileScope prof("mnb_rms_norm", s);
    cudaError_t e;
    switch (a->dtype) {
        case MNB_F32: e = launch_norm<kF32>(p, wide, s); break;
        case MNB_F16: e = launch_norm<kF16>(p, wide, s); break;
        default: e = launch_norm<kBF16>(p, wide, s); break;
    }
    if (e == cudaSuccess) prof.done("rms_norm");
    return dec::status_of(e);
}

}  // extern "C"
