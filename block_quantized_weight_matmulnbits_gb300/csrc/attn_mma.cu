// Host side of the few-row attention kernel: grid, workspace and launches.
#include "attn_mma.cuh"

namespace mnb {
namespace attn {
namespace {

// The grid of the first kernel is fixed (two CTAs on each of 152 SMs, one
// for head_dim above 128), so the workspace does not depend on the device.
constexpr int ctas_of(int dp) { return dp == 256 ? 152 : 304; }

template <int DT, int DP>
cudaError_t launch_as(const AttnParams& p, cudaStream_t s) {
    SplitParams sp{};
    sp.ctas = ctas_of(DP);
    // Uncut units save the join where most CTAs get one: 38 sequences of 300 keys (304 units) 12.7 -> 10.7 us, 28 of 700 19.6 ->
    // 16.9, 28 of 1000 27.8 -> 25.3; 20 of 1000 lose by it, 18.9 -> 22.6, as half the CTAs stay idle, but 12 tiles at most
    // would cost the others more.
    sp.whole_tiles = 16;
    // One sequence of 8000 keys, 8 key heads: 14.5, 14.4, 13.5, 16.7 us at 1, 2, 4, 8; of 60000, one key head: 21.3, 21.4, 19.9, 19.9.
    sp.min_tiles = 4;
    sp.part_o = static_cast<float*>(p.workspace);
    sp.part_ml = reinterpret_cast<float2*>(sp.part_o + (size_t)sp.ctas * 2 * mma::kRows * DP);
    sp.cut = reinterpret_cast<int4*>(sp.part_ml + (size_t)sp.ctas * 2 * mma::kRows);
    const int64_t some = p.T * p.group / mma::kRows + (p.batch < p.T ? p.batch : p.T);
    const int64_t each = (int64_t)p.batch * (((int64_t)p.max_q * p.group + mma::kRows - 1) / mma::kRows);
    const int64_t units = (int64_t)p.kv_heads * (some < each ? some : each);  // at most
    const int64_t keys = p.window > 0 && (int64_t)p.window + p.max_q < p.max_kv ? (int64_t)p.window + p.max_q : p.max_kv;
    // Few units of a moderate context: a cluster each.  A CTA takes about 5 us and 0.6 us for each 64 keys of its range;
    // the even cut over all SMs starts at about 14 us (its division, its second kernel) and wins beyond 12 tiles a CTA
    // (56 sequences of up to 2106 keys, two key heads: 20.5 us cut evenly, 22.0 us on clusters of two; one of 777 keys,
    // eight key heads: 7.7 us on clusters of eight, 16.8 us cut evenly).
    int cl = 1;
    while (cl < 8 && units * cl * 2 <= 152 * mma::Shape<DP, true>::kCtasPerSm) cl *= 2;
    if (cl > 1 && keys <= (int64_t)768 * cl) {
        auto kern = mma::attn_mma_kernel<DT, DP, true>;
        constexpr int smem = mma::Shape<DP, true>::kSmem;
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        return dec::launch_pdl(kern, dim3((unsigned)(units * cl)), dim3(mma::kThreads), smem, s, cl, p, sp);
    }
    auto kern = mma::attn_mma_kernel<DT, DP, false>;
    constexpr int smem = mma::Shape<DP, false>::kSmem;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    e = dec::launch_pdl(kern, dim3(sp.ctas), dim3(mma::kThreads), smem, s, 1, p, sp);
    if (e != cudaSuccess) return e;
    // No unit is cut when the bounds already say that each is short and has a CTA.
    if (units <= sp.ctas && keys / mma::kKeys + 2 <= sp.whole_tiles) return cudaSuccess;
    auto join = attn_join_kernel<DT, DP, mma::kRows>;
    const int64_t rows = (int64_t)p.max_q * p.group;
    return dec::launch_pdl(join, dim3(sp.ctas, (unsigned)(rows < mma::kRows ? rows : mma::kRows)), dim3(128), 0, s, 1, p, sp);
}

template <int DT>
cudaError_t launch_dt(const AttnParams& p, cudaStream_t s) {
    if (p.D <= 64) return launch_as<DT, 64>(p, s);
    if (p.D <= 128) return launch_as<DT, 128>(p, s);
    return launch_as<DT, 256>(p, s);
}

}  // namespace

size_t mma_workspace_bytes(int D) {
    const int dp = D <= 64 ? 64 : D <= 128 ? 128 : 256;
    return (size_t)ctas_of(dp) * (2 * mma::kRows * (dp + 2) * 4 + sizeof(int4));
}

cudaError_t launch_mma(const AttnParams& p, cudaStream_t s) {
    return p.dtype == kF16 ? launch_dt<kF16>(p, s) : launch_dt<kBF16>(p, s);
}

}  // namespace attn
}  // namespace mnb
