// serving.cu -- C ABI of the operators around bounded and shared decode caches:
// hyb_prefix_attn_fwd (attention over a prefix of entries that the whole batch
// shares).  Argument checks on the host, launches on the caller's stream.
#include "common.cuh"

namespace hyb {

static bool ws_ok(const void *ws, size_t ws_bytes, size_t need)
{
    return need == 0 || (ws && ws_bytes >= need && !(reinterpret_cast<uintptr_t>(ws) & 255u));
}

// Sizes shared by the workspace query and the call; HYB_OK when the call's
// index arithmetic holds for them.
static hyb_status check_prefix(const hyb_problem *p, int Np)
{
    hyb_status st = check_problem(p, false);
    if (st != HYB_OK)
        return st;
    if (Np < 0 || !(p->scale >= 0.f) || (p->W > 0 && p->Lkv <= 0))
        return HYB_ERR_INVALID_ARG;
    // query rows, and entries and window positions, are counted in 32 bits
    if (p->topk > 0 || (long long)p->B * p->Lq * p->Hq >= (1LL << 31) || (long long)Np + p->Nc >= (1LL << 30) ||
        p->W >= (1 << 30))
        return HYB_ERR_UNSUPPORTED;
    return HYB_OK;
}

}  // namespace hyb

using namespace hyb;

extern "C" {

size_t hyb_prefix_workspace_size(const hyb_problem *p, int Np)
{
    if (check_prefix(p, Np) != HYB_OK)
        return 0;
    return prefix_workspace_bytes(p->B, p->Lq, p->Lkv, p->Hq, p->Hkv, p->d, Np, p->Nc, p->W);
}

hyb_status hyb_prefix_attn_fwd(const hyb_problem *p, int Np, const void *q, const void *kp, const void *vp,
                               const void *kc, const void *vc, const void *k_raw, const void *v_raw, void *o,
                               float *lse, void *ws, size_t ws_bytes, cudaStream_t stream)
{
    NvtxRange nvtx_range("hyb_prefix_attn_fwd");
    const hyb_status st = check_prefix(p, Np);
    if (st != HYB_OK)
        return st;
    if (!q || !o || !aligned16(q) || !aligned16(o))
        return HYB_ERR_INVALID_ARG;
    if (Np > 0 && (!kp || !vp || !aligned16(kp) || !aligned16(vp)))
        return HYB_ERR_INVALID_ARG;
    if (p->Nc > 0 && (!kc || !vc || !aligned16(kc) || !aligned16(vc)))
        return HYB_ERR_INVALID_ARG;
    if (p->W > 0 && (!k_raw || !v_raw || !aligned16(k_raw) || !aligned16(v_raw)))
        return HYB_ERR_INVALID_ARG;
    if (!ws_ok(ws, ws_bytes, hyb_prefix_workspace_size(p, Np)))
        return HYB_ERR_WORKSPACE;
    return cuda_status(launch_prefix_attn(p->B, p->Lq, p->Lkv, p->Hq, p->Hkv, p->d, Np, p->Nc, p->m, p->W,
                                          softmax_scale(p), p->q_pos, p->kv_pos0, q, kp, vp, kc, vc, k_raw,
                                          v_raw, o, lse, ws, stream, num_sms_current()));
}

}  // extern "C"
