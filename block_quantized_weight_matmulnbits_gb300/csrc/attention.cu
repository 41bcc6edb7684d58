// mnb_paged_attention: argument checks and the choice of a kernel.
#include <algorithm>
#include <cmath>

#include "attention.h"

using namespace mnb;

extern "C" {

size_t mnb_attention_workspace_size(int64_t batch, int64_t T, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                    int64_t max_q, int64_t max_kv, mnb_dtype dtype) {
    const int64_t i31 = int64_t(1) << 31;
    if (batch < 1 || T < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || head_dim < 8 || head_dim % 8 != 0 ||
        head_dim > 256 || max_q < 1 || max_kv < 0 || batch >= i31 || T >= i31 || max_q >= i31 || max_kv >= i31)
        return 0;
    if (dtype != MNB_F16 && dtype != MNB_BF16) return 0;
    // the few-row kernel also takes what the many-row one declines
    size_t n = attn::mma_workspace_bytes((int)head_dim);
    if (attn::tc_serves(batch, q_heads, kv_heads, head_dim, max_q, max_kv, dtype)) {
        const size_t t = attn::tc_workspace_bytes(batch, T, q_heads, kv_heads, head_dim, max_kv);
        n = t > n ? t : n;
    }
    return (n + 255) & ~size_t(255);
}

mnb_status mnb_paged_attention(const mnb_attention_args* a, const mnb_kv_cache* c) {
    if (!a || !dec::valid_cache(c)) return MNB_ERR_INVALID_ARG;
    const int64_t i31 = int64_t(1) << 31;
    if (a->T < 0 || a->T >= i31 || a->q_heads < 1 || a->q_heads > 65535 || a->q_heads % c->kv_heads != 0 || a->max_q < 1 ||
        a->max_q >= (i31 >> 1) || a->max_kv < 0 || a->max_kv >= (i31 >> 1) || a->window < 0 || a->window >= i31 ||
        (a->causal != 0 && a->causal != 1) || !std::isfinite(a->scale) || c->head_dim % 8 != 0 || c->head_dim > 256)
        return MNB_ERR_INVALID_ARG;
    const int64_t vec = 16 / dec::dt_bytes(c->dtype);
    // a stride along one token or one head steps nowhere: it is not checked, and a plain one stands in for it
    const int64_t D = c->head_dim, HD = a->q_heads * D;
    const int64_t st[4] = {a->T > 1 ? a->q_token_stride : HD, a->q_heads > 1 ? a->q_head_stride : D,
                           a->T > 1 ? a->o_token_stride : HD, a->q_heads > 1 ? a->o_head_stride : D};
    for (int64_t x : st)
        if (x < 0 || x % vec != 0 || x >= (int64_t(1) << 38)) return MNB_ERR_INVALID_ARG;
    if (a->T == 0) return MNB_OK;
    if (a->T * a->q_heads >= i31) return MNB_ERR_UNSUPPORTED;
    if (!a->q || !a->o || !a->q_start || !dec::aligned_to(a->q, 16) || !dec::aligned_to(a->o, 16) ||
        !dec::aligned_to(a->lse, 4) || !dec::aligned_to(a->q_start, 4))
        return MNB_ERR_INVALID_ARG;
    // the least: the few-row kernel's; the many-row one cuts the context as far as the rest goes
    const size_t least = c->dtype == MNB_F32 ? 0 : attn::mma_workspace_bytes(c->head_dim);
    if (least && (!a->workspace || a->workspace_bytes < least)) return MNB_ERR_NO_MEM;
    if (a->workspace && !dec::aligned_to(a->workspace, 256)) return MNB_ERR_INVALID_ARG;

    attn::AttnParams p{};
    p.status = device_status_word();
    if (!p.status) return dec::status_of(cudaErrorUnknown);
    p.q = a->q;
    p.o = a->o;
    p.lse = a->lse;
    p.k = c->k_pages;
    p.v = c->v_pages;
    p.tables = c->tables;
    p.kv_lens = c->kv_lens;
    p.q_start = a->q_start;
    p.T = a->T;
    p.table_stride = c->table_stride;
    p.q_ts = st[0];
    p.q_hs = st[1];
    p.o_ts = st[2];
    p.o_hs = st[3];
    p.page_stride = c->page_stride;
    p.token_stride = c->token_stride;
    p.head_stride = c->head_stride;
    p.batch = (int)c->batch;
    p.q_heads = (int)a->q_heads;
    p.kv_heads = c->kv_heads;
    p.group = (int)(a->q_heads / c->kv_heads);
    p.D = c->head_dim;
    while ((1 << p.page_shift) < c->page_size) ++p.page_shift;
    p.num_pages = (int)c->num_pages;
    p.max_q = (int)a->max_q;
    p.max_kv = (int)a->max_kv;
    p.window = (int)a->window;
    p.causal = a->causal;
    p.scale = a->scale;
    p.scale_log2 = a->scale * attn::kLog2e;
    // a masked score is -inf before it is scaled; 2^-100 leaves every finite score at 0
    if (std::fabs(p.scale_log2) < 0x1p-100f) p.scale_log2 = 0x1p-100f;
    p.workspace = a->workspace;
    p.workspace_bytes = a->workspace_bytes;
    p.dtype = c->dtype;
    uint32_t hint;
    wait_limits(&p.wait_limit, &hint);
    // these kernels' waits take no hint, whatever MNB_WAIT_MODE says, and begin behind the preceding kernel
    if (hint || p.wait_limit > kWaitTries) p.wait_limit = kWaitTries;
    if (inject_launch_failure()) return MNB_ERR_CUDA;
    ProfileScope prof("mnb_paged_attention", (cudaStream_t)a->stream);
    const cudaStream_t s = (cudaStream_t)a->stream;
    const char* family = "attn_f32";
    cudaError_t e = cudaErrorNotSupported;
    if (c->dtype == MNB_F32) {
        e = attn::launch_f32(p, s);
    } else {
        // the keys that a sequence's new tokens see
        const int64_t keys = a->window > 0 ? std::min(a->max_kv, a->window + a->max_q) : a->max_kv;
        if (attn::tc_serves(p.batch, p.q_heads, p.kv_heads, p.D, p.max_q, keys, p.dtype)) {
            family = "attn_tc";
            e = attn::launch_tc(p, s);
        }
        if (e == cudaErrorNotSupported) {
            family = "attn_mma";
            e = attn::launch_mma(p, s);
        }
    }
    if (e == cudaSuccess) prof.done(family);
    return dec::status_of(e);
}

}  // extern "C"
