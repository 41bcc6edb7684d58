// Host side of the many-row attention kernel: tensor maps, the cut of few
// units into ranges of keys, workspace and launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "attn_tc.cuh"

namespace mnb {
namespace attn {
namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return (EncodeTiledFn) nullptr;
        }
        return reinterpret_cast<EncodeTiledFn>(ptr);
    }();
    return fn;
}

struct Plan {
    int tokens, splits;
    int64_t units;
};

// Units and splits from the bounds of a call.  A wave of 152 CTAs takes as
// long as its key tiles plus about four tiles' worth of prologue and epilogue
// (2 to 8 choose the same cut in most cases); the cut with the least waves *
// (tiles + 4) is taken.  A cut pays its partial results, a tile a wave, and the
// join, about four tiles, and it must save 5 % beyond them, because unequal
// units (a causal chunk's) pack better than whole waves.  32 / 8 heads x 128,
// cut against uncut, us:
//   not cut for it: 300 tokens 19 - 12, 500 over 1000 keys 27 - 20, 1500 over
//     3000 85 - 63, 4096 over 8192 345 - 281, 32 sequences of 64 over 8000 281 - 227
//   still cut: 40 over 1000 15.5 - 18.6, 300 over 2000 26 - 31, 500 over 4000
//     43 - 52, 2048 over 32000 700 - 733, 500 over 32000 194 - 367
// max_pieces: the partial results (units x ranges) that the workspace has room
// for.  seen: most keys that a unit sees where a window bounds them (they may
// begin inside a tile), or 0.
Plan make_plan(int64_t batch, int64_t T, int64_t q_heads, int64_t kv_heads, int64_t max_kv, int64_t max_pieces, int64_t seen) {
    Plan pl;
    const int64_t group = q_heads / kv_heads;
    pl.tokens = (int)(tca::kRows / group);
    pl.units = (T / (2 * pl.tokens) + (batch < T ? batch : T)) * kv_heads;
    pl.splits = 1;
    int64_t tiles = (max_kv + tca::kKeys - 1) / tca::kKeys;
    if (seen > 0) tiles = std::min(tiles, (seen + tca::kKeys - 1) / tca::kKeys + 1);
    double best = 0;
    for (int64_t s = 1; s <= 64 && s <= tiles; ++s) {
        if (s > 1 && pl.units * s > max_pieces) break;
        const int64_t waves = (pl.units * s + 151) / 152;
        double cost = (double)waves * (double)((tiles + s - 1) / s + 4);
        if (s > 1) cost = cost * 1.05 + (double)(pl.units * s) / 152.0 + 4;
        if (s == 1 || cost < best) {
            best = cost;
            pl.splits = (int)s;
        }
    }
    return pl;
}

// How one box can bring both halves of 128 depths: rows split into groups of 8, halves and groups as dimensions of their
// own, which leaves one more for pages and key heads.  The heads go beside the halves where a head follows the other
// at once (tokens before heads), or beside the pages where a page is a number of heads (heads before tokens).
struct OneBox {
    bool ok;
    int64_t page_step, head_step;  // in the last dimension
    int head_halves;               // in the dimension of halves
    int64_t halves, last, last_stride;
};
OneBox one_box(const AttnParams& p) {
    OneBox b{};
    if (p.D != 128) return b;
    const int64_t pages = p.num_pages;
    if (p.kv_heads == 1 || p.head_stride == 128) {
        b = {true, 1, 0, 2, 2 * (int64_t)p.kv_heads, pages, p.page_stride};
    } else if (p.head_stride > 0 && p.page_stride % p.head_stride == 0) {
        const int64_t ratio = p.page_stride / p.head_stride;
        // (the page after the last one stands for none: it has to lie past the last head of the last page)
        b = {ratio >= p.kv_heads && (pages + 1) * ratio < (int64_t(1) << 31), ratio, 1, 0, 2, (pages - 1) * ratio + p.kv_heads,
             p.head_stride};
    }
    return b;
}

// Partial results of 256 rows: O and (m, l).
size_t piece_bytes(int64_t D) { return (size_t)256 * ((D <= 64 ? 64 : 128) + 2) * 4; }

template <int DT, int DP, bool ONE>
cudaError_t launch_as(const AttnParams& p, const Plan& pl, cudaStream_t s) {
    using S = tca::Shape<DP, ONE>;
    EncodeTiledFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const CUtensorMapDataType dt = DT == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    CUtensorMap maps[3];
    std::memset(maps, 0, sizeof(maps));
    {
        const cuuint64_t dims[4] = {(cuuint64_t)p.D, (cuuint64_t)p.group, (cuuint64_t)p.kv_heads, (cuuint64_t)p.T};
        const cuuint64_t st[3] = {(cuuint64_t)p.q_hs * 2, (cuuint64_t)p.q_hs * 2 * (cuuint64_t)p.group, (cuuint64_t)p.q_ts * 2};
        const cuuint32_t box[4] = {64, (cuuint32_t)p.group, 1, (cuuint32_t)pl.tokens};
        if (enc(&maps[0], dt, 4, const_cast<void*>(p.q), dims, st, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorNotSupported;
    }
    const int page = 1 << p.page_shift, rows = page < tca::kKeys ? page : tca::kKeys;
    tca::TcParams tp{};
    for (int i = 0; i < 2; ++i) {
        if constexpr (ONE) {
            const OneBox b = one_box(p);
            const cuuint64_t dims[5] = {64, 8, (cuuint64_t)b.halves, (cuuint64_t)(page / 8), (cuuint64_t)b.last};
            const cuuint64_t st[4] = {(cuuint64_t)p.token_stride * 2, 128, (cuuint64_t)p.token_stride * 16, (cuuint64_t)b.last_stride * 2};
            const cuuint32_t box[5] = {64, 8, 2, (cuuint32_t)(rows / 8), 1};
            if (enc(&maps[1 + i], dt, 5, const_cast<void*>(i ? p.v : p.k), dims, st, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
                return cudaErrorNotSupported;
            tp.page_step = b.page_step;
            tp.head_step = b.head_step;
            tp.head_halves = b.head_halves;
            continue;
        }
        const cuuint64_t dims[4] = {(cuuint64_t)p.D, (cuuint64_t)page, (cuuint64_t)p.kv_heads, (cuuint64_t)p.num_pages};
        const cuuint64_t st[3] = {(cuuint64_t)p.token_stride * 2, (cuuint64_t)p.head_stride * 2, (cuuint64_t)p.page_stride * 2};
        const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1};
        if (enc(&maps[1 + i], dt, 4, const_cast<void*>(i ? p.v : p.k), dims, st, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorNotSupported;
    }
    tp.tokens = pl.tokens;
    tp.units = (int)pl.units;
    tp.splits = pl.splits;
    tp.box_rows = rows;
    tp.part_o = static_cast<float*>(p.workspace);
    tp.part_ml = reinterpret_cast<float2*>(tp.part_o + (size_t)pl.units * pl.splits * 256 * DP);
    AttnParams q = p;
    tp.negate = p.scale_log2 < 0.f;
    q.scale_log2 = std::fabs(p.scale_log2);
    auto kern = tca::attn_tc_kernel<DT, DP, ONE>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    e = dec::launch_pdl(kern, dim3((unsigned)(pl.units * pl.splits)), dim3(tca::kThreads), S::kSmem, s, 1, q, tp, maps[0], maps[1], maps[2]);
    if (e != cudaSuccess || pl.splits == 1) return e;
    return dec::launch_pdl(tca::attn_tc_join_kernel<DT, DP>, dim3((unsigned)(pl.units * 32)), dim3(256), 0, s, 1, p, tp);
}

}  // namespace

// From 33 rows a key head on; from 17 on where the keys that the call sees are many.  There the few-row kernel reads and
// walks them twice (two row tiles of 16), which costs less than this kernel's longer start while they are few.  By their
// bytes, this kernel against the few-row one, us (16 sequences of 8 new tokens unless said):
//   16 / 4 heads x 64:  17 MB 25 - 17, 33 MB 29 - 21, 66 MB 37 - 44, 131 MB 54 - 72, 524 MB 150 - 203;
//                       32000 keys under a window of 1024 (17 MB) 25 - 17, of 4096 (67 MB) 37 - 46
//   32 / 8 x 128:       33 MB 21 - 21, 66 MB 29 - 35, 131 MB 42 - 70; under a window of 1024 (68 MB) 29 - 44
//   4 sequences of it:  33 MB 27 - 21, 66 MB 35 - 35, 131 MB 48 - 52;  one: 33 MB 29 - 27, 66 MB 37 - 34, 131 MB 50 - 49
bool tc_serves(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t D, int64_t max_q, int64_t keys, int dtype) {
    const int64_t group = q_heads / kv_heads, rows = max_q * group;
    if (dtype == kF32 || D > 128 || group > tca::kRows || rows <= 16) return false;
    const double bytes = (double)batch * (double)keys * (double)(kv_heads * D) * 4.0;
    return rows > 32 || bytes > 100e6 || (bytes > 50e6 && batch * kv_heads >= 32);
}

// A call with more units may want fewer pieces than one with less (a full wave is not cut), so the size reported is no
// less than kSharedPieces as soon as that many could be of use: a buffer sized for the largest call of a program then
// serves its smaller ones at full speed (81 MB at 128 depths), up to those that want more than four waves of pieces.
constexpr int64_t kSharedPieces = 4 * 152;

size_t tc_workspace_bytes(int64_t batch, int64_t T, int64_t q_heads, int64_t kv_heads, int64_t D, int64_t max_kv) {
    const Plan pl = make_plan(batch, T, q_heads, kv_heads, max_kv, INT64_MAX, 0);
    const int64_t tiles = (max_kv + tca::kKeys - 1) / tca::kKeys, most = pl.units * std::min<int64_t>(64, tiles);
    const int64_t shared = tiles > 1 ? std::min(kSharedPieces, most) : 0;
    return (size_t)std::max(shared, pl.splits == 1 ? 0 : pl.units * pl.splits) * piece_bytes(D);
}

cudaError_t launch_tc(const AttnParams& p, cudaStream_t s) {
    // (a unit's first row sees window keys, its last one as many further on, or the sequence to its end)
    const int64_t rows = p.causal ? std::min<int64_t>(2 * (tca::kRows / p.group), p.max_q) : p.max_q;
    const int64_t seen = p.window > 0 ? p.window + rows - 1 : 0;
    const Plan pl = make_plan(p.batch, p.T, p.q_heads, p.kv_heads, p.max_kv, (int64_t)(p.workspace_bytes / piece_bytes(p.D)), seen);
    if (pl.units * pl.splits * 32 > 0x7FFFFFFF) return cudaErrorNotSupported;
    if (p.D <= 64) return p.dtype == kF16 ? launch_as<kF16, 64, false>(p, pl, s) : launch_as<kBF16, 64, false>(p, pl, s);
    if (one_box(p).ok) {
        const cudaError_t e = p.dtype == kF16 ? launch_as<kF16, 128, true>(p, pl, s) : launch_as<kBF16, 128, true>(p, pl, s);
        if (e != cudaErrorNotSupported) return e;
    }
    return p.dtype == kF16 ? launch_as<kF16, 128, false>(p, pl, s) : launch_as<kBF16, 128, false>(p, pl, s);
}

}  // namespace attn
}  // namespace mnb
