// Rotary positions, alone and with the append of a step's keys and values to
// the paged cache, and the table of cosines and sines they read.
//
//   (a, b) -> (a c - b s, b c + a s),   c, s = table row of the token's position
//
// with (a, b) = depths (i, i + r/2) or (2i, 2i + 1), i < r/2, as ONNX Runtime's
// com.microsoft::RotaryEmbedding pairs them.  Three flops a value: the kernel is
// bound by the bytes of x and y, so all it has to do is keep enough wide loads
// in flight.  A thread owns one 16-byte vector (half layout: the two vectors of
// its pairs) of up to four heads of one token: the table values are read once
// for them, and their loads are independent.  Neighbouring threads take
// neighbouring vectors of neighbouring heads, so a warp's accesses are whole
// lines.  The append is the same pass with another address for k and v.
//
// Measured on a GB300 (6800 GB/s copy): 10031 tokens of 48 heads x 128 in bf16,
// half layout, turned and appended: 40.1 us, 6210 GB/s (48 us with one head a
// thread, 42.5 with two); 4999 x 18 x 96 in f32, interleaved, 64 of 96 depths:
// 14.2 us, 4950 GB/s, the ramp and tail of a short kernel.  One token: 7 us, the
// launch and a chain of lookups (length, page, table row).
#include <cmath>

#include "decoder.h"

namespace mnb {
namespace {

constexpr int kThreads = 256;

struct RotParams {
    const void* src[3];            // q, k, v (or x)
    int64_t src_ts[3], src_hs[3];  // token and head strides, elements
    void* dst[3];                  // q_out (or y), k_pages, v_pages
    int64_t out_ts, out_hs;        // strides of dst[0]
    int64_t page_stride, token_stride, head_stride;
    const float* cos;
    const float* sin;
    const int32_t* positions;      // null: the token's place in its sequence
    const int32_t* q_start;        // null: no cache (mnb_rotary)
    const int32_t* kv_lens;
    const int32_t* tables;
    int64_t table_stride, num_pages, n_pos;
    int64_t T;
    int batch, page_shift;
    int h_q, h_k;                  // heads 0 .. h_q - 1 are q, the next h_k k, the next h_k v
    int rot, n_pair, per_head;     // turned depths, vectors (pairs of vectors) that turn, items a head
    int groups;                    // head groups: a thread's heads are g, g + groups, ...
    float sign;                    // -1: the inverse rotation
    int* status;
};

template <int DT> struct Elem;
template <> struct Elem<kF32> { using T = float; };
template <> struct Elem<kF16> { using T = __half; };
template <> struct Elem<kBF16> { using T = __nv_bfloat16; };

template <int DT>
__device__ __forceinline__ float widen(typename Elem<DT>::T v) {
    if constexpr (DT == kF32) return v;
    else if constexpr (DT == kF16) return __half2float(v);
    else return __bfloat162float(v);
}
template <int DT>
__device__ __forceinline__ typename Elem<DT>::T narrow(float v) {
    if constexpr (DT == kF32) return v;
    else if constexpr (DT == kF16) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

// V consecutive values, one access of V * sizeof(T) bytes when WIDE.
template <int DT, int V, bool WIDE>
struct Pack {
    using T = typename Elem<DT>::T;
    T v[V];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (WIDE && sizeof(T) * V == 16) *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
        else if constexpr (WIDE) *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(p);
        else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = p[i];
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (WIDE && sizeof(T) * V == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
        else if constexpr (WIDE) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(v);
        else {
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] = v[i];
        }
    }
};

template <int N>
__device__ __forceinline__ void load_floats(float (&r)[N], const float* p) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(p + i));
            r[i] = f.x; r[i + 1] = f.y; r[i + 2] = f.z; r[i + 3] = f.w;
        }
    } else if constexpr (N == 2) {
        const float2 f = __ldg(reinterpret_cast<const float2*>(p));
        r[0] = f.x; r[1] = f.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = __ldg(p + i);
    }
}

// V: values a vector holds.  HPT: heads a thread handles.
template <int DT, int V, bool WIDE, bool INTER, int HPT>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotParams p) {
    using T = typename Elem<DT>::T;
    constexpr int NV = INTER ? 1 : 2;         // vectors of an item that turns
    constexpr int NC = INTER ? V / 2 : V;     // table values of an item
    const int64_t per_token = (int64_t)p.groups * p.per_head;
    const int64_t base = (int64_t)blockIdx.x * kThreads;
    const int64_t t0 = base / per_token;      // the same for the block
    const uint32_t off = (uint32_t)(base - t0 * per_token) + threadIdx.x;
    const uint32_t dt = off / (uint32_t)per_token;
    const uint32_t r = off - dt * (uint32_t)per_token;
    const int64_t t = t0 + dt;
    griddep_wait();
    griddep_launch_dependents();
    if (t >= p.T) return;
    const int g = (int)(r / (uint32_t)p.per_head);
    const int c = (int)(r - (uint32_t)g * (uint32_t)p.per_head);

    const bool turns = c < p.n_pair;
    const int i0 = turns ? c * V : p.rot + (c - p.n_pair) * (WIDE ? V : 1);  // first depth of the item
    const int half = p.rot >> 1;
    const int heads = p.h_q + 2 * p.h_k;

    // The values first: their loads need nothing that is looked up below.
    Pack<DT, V, WIDE> a[HPT], b[HPT];
#pragma unroll
    for (int j = 0; j < HPT; ++j) {
        const int h = g + j * p.groups;
        if (h < heads) {
            const int seg = h < p.h_q ? 0 : h < p.h_q + p.h_k ? 1 : 2;
            const int hh = h - (seg == 0 ? 0 : seg == 1 ? p.h_q : p.h_q + p.h_k);
            const T* in = static_cast<const T*>(p.src[seg]) + t * p.src_ts[seg] + hh * p.src_hs[seg] + i0;
            if (WIDE || turns) a[j].load(in);
            else a[j].v[0] = *in;  // a copied depth; D - rot may be odd
            if (NV == 2 && turns) b[j].load(in + half);
        }
    }

    int64_t pos, row = 0;  // position for the table, offset of the token's row in the pages
    if (p.q_start) {
        if (t >= p.q_start[p.batch]) return;
        const int b = dec::sequence_of(p.q_start, p.batch, t);
        const int64_t place = (int64_t)p.kv_lens[b] - p.q_start[b + 1] + t;
        const int64_t col = place >> p.page_shift;
        int64_t page = -1;
        if (place >= 0 && col < p.table_stride) page = p.tables[(int64_t)b * p.table_stride + col];
        if (page < 0 || page >= p.num_pages) {
            set_status(p.status, MNB_ERR_INVALID_ARG);
            return;
        }
        row = page * p.page_stride + (place & ((1 << p.page_shift) - 1)) * p.token_stride;
        pos = p.positions ? p.positions[t] : place;
    } else {
        pos = p.positions[t];
    }
    if (pos < 0 || pos >= p.n_pos) {
        set_status(p.status, MNB_ERR_INVALID_ARG);
        return;
    }
    float cs[NC], sn[NC];
    if (turns) {
        const int64_t at = pos * half + (INTER ? i0 / 2 : i0);
        load_floats(cs, p.cos + at);
        load_floats(sn, p.sin + at);
#pragma unroll
        for (int i = 0; i < NC; ++i) sn[i] *= p.sign;
    }
#pragma unroll
    for (int j = 0; j < HPT; ++j) {
        const int h = g + j * p.groups;
        if (h >= heads) continue;
        const int seg = h < p.h_q ? 0 : h < p.h_q + p.h_k ? 1 : 2;
        const int hh = h - (seg == 0 ? 0 : seg == 1 ? p.h_q : p.h_q + p.h_k);
        if (turns && seg < 2) {
            if constexpr (INTER) {
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const float x = widen<DT>(a[j].v[2 * i]), y = widen<DT>(a[j].v[2 * i + 1]);
                    a[j].v[2 * i] = narrow<DT>(fmaf(x, cs[i], -(y * sn[i])));
                    a[j].v[2 * i + 1] = narrow<DT>(fmaf(y, cs[i], x * sn[i]));
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float x = widen<DT>(a[j].v[i]), y = widen<DT>(b[j].v[i]);
                    a[j].v[i] = narrow<DT>(fmaf(x, cs[i], -(y * sn[i])));
                    b[j].v[i] = narrow<DT>(fmaf(y, cs[i], x * sn[i]));
                }
            }
        }
        T* out = static_cast<T*>(p.dst[seg]) + (seg == 0 ? t * p.out_ts + hh * p.out_hs : row + hh * p.head_stride) + i0;
        if (WIDE || turns) a[j].store(out);
        else *out = a[j].v[0];
        if (NV == 2 && turns) b[j].store(out + half);
    }
}

template <int DT, int V, bool WIDE, bool INTER>
cudaError_t launch_as(RotParams p, int64_t D, cudaStream_t s) {
    const int heads = p.h_q + 2 * p.h_k;
    p.n_pair = INTER ? p.rot / V : p.rot / 2 / V;
    p.per_head = p.n_pair + (int)((D - p.rot) / (WIDE ? V : 1));
    // Several heads a thread once that still leaves two full blocks' worth of
    // threads per SM; one below, where more threads hide more latency.  Four of
    // one vector each (interleaved pairs), three of two vectors (halves): 10031
    // tokens x 48 heads x 128, bf16: halves 40.2 us with three, 41.5 with four,
    // 44.2 with six; interleaved 43.2 with four, 47.4 with three.
    constexpr int kMany = INTER ? 4 : 3;
    const bool many = WIDE && p.T * heads * p.per_head >= (int64_t)4 * 2048 * dec::kSms;
    p.groups = many ? (heads + kMany - 1) / kMany : heads;
    const int64_t items = p.T * p.groups * p.per_head;
    const int64_t blocks = (items + kThreads - 1) / kThreads;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    if constexpr (WIDE) {
        if (many)
            return dec::launch_pdl(rotary_kernel<DT, V, WIDE, INTER, kMany>, dim3((unsigned)blocks), dim3(kThreads), 0, s, 1, p);
    }
    return dec::launch_pdl(rotary_kernel<DT, V, WIDE, INTER, 1>, dim3((unsigned)blocks), dim3(kThreads), 0, s, 1, p);
}

template <int DT, bool INTER>
cudaError_t launch_dt(const RotParams& p, int64_t D, int bytes, cudaStream_t s) {
    constexpr int E = DT == kF32 ? 4 : 2;
    switch (bytes) {
        case 16: return launch_as<DT, 16 / E, true, INTER>(p, D, s);
        case 8: return launch_as<DT, 8 / E, true, INTER>(p, D, s);
        default: return launch_as<DT, INTER ? 2 : 1, false, INTER>(p, D, s);
    }
}

// Widest access (16, 8 or single values: 0) that every base, stride and part of a head allows.
struct Width {
    int e, bytes = 16;
    explicit Width(int esize) : e(esize) {}
    void base(const void* q) {
        while (bytes && !dec::aligned_to(q, (size_t)bytes)) bytes = bytes == 16 ? 8 : 0;
    }
    void elems(int64_t n) {
        while (bytes && (n * e) % bytes != 0) bytes = bytes == 16 ? 8 : 0;
    }
};

cudaError_t launch_rotary(const RotParams& p, int64_t D, int dtype, int flags, int bytes, cudaStream_t s) {
    const bool inter = (flags & MNB_ROTARY_INTERLEAVED) != 0;
    switch (dtype) {
        case kF32: return inter ? launch_dt<kF32, true>(p, D, bytes, s) : launch_dt<kF32, false>(p, D, bytes, s);
        case kF16: return inter ? launch_dt<kF16, true>(p, D, bytes, s) : launch_dt<kF16, false>(p, D, bytes, s);
        default: return inter ? launch_dt<kBF16, true>(p, D, bytes, s) : launch_dt<kBF16, false>(p, D, bytes, s);
    }
}

int width_of(const RotParams& p, int64_t D, int dtype, int flags) {
    Width w(dec::dt_bytes(dtype));
    const bool cache = p.q_start != nullptr;
    for (int i = 0; i < (cache ? 3 : 1); ++i) {
        if (i == 0 && p.h_q == 0) continue;
        w.base(p.src[i]);
        w.base(p.dst[i]);
        w.elems(p.src_ts[i]);
        w.elems(p.src_hs[i]);
    }
    if (p.h_q) {
        w.elems(p.out_ts);
        w.elems(p.out_hs);
    }
    // (the cache's strides are multiples of 16 bytes)
    w.elems((flags & MNB_ROTARY_INTERLEAVED) ? p.rot : p.rot / 2);
    w.elems(D - p.rot);
    if (w.bytes && (!dec::aligned_to(p.cos, 16) || !dec::aligned_to(p.sin, 16))) w.bytes = 0;
    return w.bytes;
}

struct TableParams {
    float* cos;
    float* sin;
    int64_t n_pos;
    int half, scaling;
    double log2_base, rot, factor, trained_len, low, high, attn;
};

constexpr int kTableRows = 64;

// One frequency per thread, kTableRows positions each.  f64 throughout: the
// table is made once, and a position of 10^5 times an f32 frequency would be
// off by a hundredth of a radian.
__global__ void __launch_bounds__(128) rotary_table_kernel(const TableParams p) {
    griddep_wait();
    const int i = (int)(blockIdx.y * blockDim.x + threadIdx.x);
    if (i >= p.half) return;
    const double f0 = exp2(-2.0 * i / p.rot * p.log2_base);
    double f = f0;
    if (p.scaling == MNB_ROPE_LINEAR) f = f0 / p.factor;
    if (p.scaling == MNB_ROPE_BY_PARTS) {
        const double turns = p.trained_len * f0 / 6.283185307179586476925286766559;
        const double g = fmin(1.0, fmax(0.0, (turns - p.low) / (p.high - p.low)));
        f = g * f0 + (1.0 - g) * f0 / p.factor;
    }
    const int64_t first = (int64_t)blockIdx.x * kTableRows;
    for (int r = 0; r < kTableRows; ++r) {
        const int64_t pos = first + r;
        if (pos >= p.n_pos) return;
        double s, c;
        sincos((double)pos * f, &s, &c);
        p.cos[pos * p.half + i] = (float)(p.attn * c);
        p.sin[pos * p.half + i] = (float)(p.attn * s);
    }
}

bool valid_sizes(int64_t T, int64_t H, int64_t D, int64_t rot, int64_t n_pos) {
    return T >= 0 && T < (int64_t(1) << 31) && H >= 1 && H <= 65535 && D >= 1 && D <= 4096 && rot >= 2 && rot <= D &&
           rot % 2 == 0 && n_pos >= 1 && n_pos < (int64_t(1) << 31);
}
bool valid_strides(int64_t ts, int64_t hs) {
    const int64_t most = int64_t(1) << 39;
    return ts >= 0 && hs >= 0 && ts < most && hs < most;
}

}  // namespace
}  // namespace mnb

using namespace mnb;

extern "C" {

mnb_status mnb_rotary_table(float* cos_table, float* sin_table, int64_t n_pos, int64_t rot_dim, double base,
                            mnb_rope_scaling scaling, double factor, double trained_len, double low, double high,
                            double attn_factor, mnb_stream_t stream) {
    if (!cos_table || !sin_table || !dec::aligned_to(cos_table, 4) || !dec::aligned_to(sin_table, 4)) return MNB_ERR_INVALID_ARG;
    if (n_pos < 1 || n_pos >= (int64_t(1) << 31) || rot_dim < 2 || rot_dim > 4096 || rot_dim % 2 != 0) return MNB_ERR_INVALID_ARG;
    if (!(base > 0) || !std::isfinite(base) || !std::isfinite(attn_factor)) return MNB_ERR_INVALID_ARG;
    if (scaling < MNB_ROPE_NONE || scaling > MNB_ROPE_BY_PARTS) return MNB_ERR_INVALID_ARG;
    if (scaling != MNB_ROPE_NONE && (!(factor > 0) || !std::isfinite(factor))) return MNB_ERR_INVALID_ARG;
    if (scaling == MNB_ROPE_NTK && rot_dim == 2) return MNB_ERR_INVALID_ARG;
    if (scaling == MNB_ROPE_BY_PARTS &&
        (!(trained_len > 0) || !std::isfinite(trained_len) || !(low < high) || !std::isfinite(low) || !std::isfinite(high)))
        return MNB_ERR_INVALID_ARG;
    if (inject_launch_failure()) return MNB_ERR_CUDA;
    TableParams p{};
    p.cos = cos_table;
    p.sin = sin_table;
    p.n_pos = n_pos;
    p.half = (int)(rot_dim / 2);
    p.scaling = scaling;
    p.rot = (double)rot_dim;
    p.log2_base = std::log2(base);
    if (scaling == MNB_ROPE_NTK) p.log2_base += std::log2(factor) * p.rot / (p.rot - 2.0);
    p.factor = factor;
    p.trained_len = trained_len;
    p.low = low;
    p.high = high;
    p.attn = attn_factor;
    const dim3 grid((unsigned)((n_pos + kTableRows - 1) / kTableRows), (unsigned)((p.half + 127) / 128));
    return dec::status_of(dec::launch_pdl(rotary_table_kernel, grid, dim3(128), 0, (cudaStream_t)stream, 1, p));
}

mnb_status mnb_rotary(const void* x, void* y, const int32_t* positions, const float* cos_table,
                      const float* sin_table, int64_t T, int64_t H, int64_t D, int64_t rot_dim, int64_t n_pos,
                      int64_t x_token_stride, int64_t x_head_stride, int64_t y_token_stride, int64_t y_head_stride,
                      mnb_dtype dtype, int flags, mnb_stream_t stream) {
    if (!valid_sizes(T, H, D, rot_dim, n_pos) || !dec::valid_dt(dtype) ||
        (flags & ~(MNB_ROTARY_INTERLEAVED | MNB_ROTARY_INVERSE)) != 0 || !valid_strides(x_token_stride, x_head_stride) ||
        !valid_strides(y_token_stride, y_head_stride))
        return MNB_ERR_INVALID_ARG;
    if (T == 0) return MNB_OK;
    const size_t e = (size_t)dec::dt_bytes(dtype);
    if (!x || !y || !positions || !cos_table || !sin_table || !dec::aligned_to(x, e) || !dec::aligned_to(y, e) ||
        !dec::aligned_to(positions, 4) || !dec::aligned_to(cos_table, 4) || !dec::aligned_to(sin_table, 4))
        return MNB_ERR_INVALID_ARG;
    RotParams p{};
    p.status = device_status_word();
    if (!p.status) return dec::status_of(cudaErrorUnknown);
    p.src[0] = x;
    p.src_ts[0] = x_token_stride;
    p.src_hs[0] = x_head_stride;
    p.dst[0] = y;
    p.out_ts = y_token_stride;
    p.out_hs = y_head_stride;
    p.cos = cos_table;
    p.sin = sin_table;
    p.positions = positions;
    p.n_pos = n_pos;
    p.T = T;
    p.h_q = (int)H;
    p.rot = (int)rot_dim;
    p.sign = (flags & MNB_ROTARY_INVERSE) ? -1.f : 1.f;
    if (inject_launch_failure()) return MNB_ERR_CUDA;
    ProfileScope prof("mnb_rotary", (cudaStream_t)stream);
    const cudaError_t err = launch_rotary(p, D, dtype, flags, width_of(p, D, dtype, flags), (cudaStream_t)stream);
    if (err == cudaSuccess) prof.done("rotary");
    return dec::status_of(err);
}

mnb_status mnb_rotary_append(const mnb_rotary_args* a, const mnb_kv_cache* c) {
    if (!a || !dec::valid_cache(c)) return MNB_ERR_INVALID_ARG;
    const int64_t qh = a->q ? a->q_heads : 0;
    if (!valid_sizes(a->T, a->q ? a->q_heads : 1, c->head_dim, a->rot_dim, a->n_pos) ||
        (a->flags & ~(MNB_ROTARY_INTERLEAVED | MNB_ROTARY_INVERSE)) != 0 ||
        !valid_strides(a->k_token_stride, a->k_head_stride) || !valid_strides(a->v_token_stride, a->v_head_stride) ||
        (a->q && (!valid_strides(a->q_token_stride, a->q_head_stride) ||
                  !valid_strides(a->q_out_token_stride, a->q_out_head_stride))))
        return MNB_ERR_INVALID_ARG;
    if (a->T == 0) return MNB_OK;
    const size_t e = (size_t)dec::dt_bytes(c->dtype);
    if (!a->k || !a->v || !a->cos_table || !a->sin_table || !a->q_start || (a->q && !a->q_out)) return MNB_ERR_INVALID_ARG;
    if (!dec::aligned_to(a->k, e) || !dec::aligned_to(a->v, e) || !dec::aligned_to(a->cos_table, 4) ||
        !dec::aligned_to(a->sin_table, 4) || !dec::aligned_to(a->q_start, 4) || !dec::aligned_to(a->positions, 4) ||
        (a->q && (!dec::aligned_to(a->q, e) || !dec::aligned_to(a->q_out, e))))
        return MNB_ERR_INVALID_ARG;
    RotParams p{};
    p.status = device_status_word();
    if (!p.status) return dec::status_of(cudaErrorUnknown);
    const void* src[3] = {a->q, a->k, a->v};
    const int64_t ts[3] = {a->q_token_stride, a->k_token_stride, a->v_token_stride};
    const int64_t hs[3] = {a->q_head_stride, a->k_head_stride, a->v_head_stride};
    void* dst[3] = {a->q_out, c->k_pages, c->v_pages};
    for (int i = 0; i < 3; ++i) {
        p.src[i] = src[i];
        p.src_ts[i] = ts[i];
        p.src_hs[i] = hs[i];
        p.dst[i] = dst[i];
    }
    p.out_ts = a->q_out_token_stride;
    p.out_hs = a->q_out_head_stride;
    p.page_stride = c->page_stride;
    p.token_stride = c->token_stride;
    p.head_stride = c->head_stride;
    p.cos = a->cos_table;
    p.sin = a->sin_table;
    p.positions = a->positions;
    p.q_start = a->q_start;
    p.kv_lens = c->kv_lens;
    p.tables = c->tables;
    p.table_stride = c->table_stride;
    p.num_pages = c->num_pages;
    p.n_pos = a->n_pos;
    p.T = a->T;
    p.batch = (int)c->batch;
    p.page_shift = 0;
    while ((1 << p.page_shift) < c->page_size) ++p.page_shift;
    p.h_q = (int)qh;
    p.h_k = c->kv_heads;
    p.rot = (int)a->rot_dim;
    p.sign = (a->flags & MNB_ROTARY_INVERSE) ? -1.f : 1.f;
    if (inject_launch_failure()) return MNB_ERR_CUDA;
    ProfileScope prof("mnb_rotary_append", (cudaStream_t)a->stream);
    const cudaError_t err =
        launch_rotary(p, c->head_dim, c->dtype, a->flags, width_of(p, c->head_dim, c->dtype, a->flags), (cudaStream_t)a->stream);
    if (err == cudaSuccess) prof.done("rotary_append");
    return dec::status_of(err);
}

}  // extern "C"
