// serving.cu -- C ABI of the operators around bounded and shared decode caches:
// hyb_prefix_attn_fwd (attention over a prefix of entries that the whole batch
// shares), hyb_attn_weights (the weight each cached entry received),
// hyb_evict_select and hyb_cache_compact (eviction by that weight).  Argument
// checks on the host, launches on the caller's stream.
#include "common.cuh"

namespace hyb {

static bool aligned4(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 3u) == 0;
}

static bool ws_ok(const void *ws, size_t ws_bytes, size_t need)
{
    return need == 0 || (ws && ws_bytes >= need && !(reinterpret_cast<uintptr_t>(ws) & 255u));
}

// Sizes, tiling and split shared by the workspace query and the call; HYB_OK
// when the call's index arithmetic holds for them.
static hyb_status check_prefix(const hyb_problem *p, int Np, PrefixParams &a)
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
    a = PrefixParams{};
    a.B = p->B;
    a.Lq = p->Lq;
    a.Lkv = p->Lkv;
    a.Hq = p->Hq;
    a.Hkv = p->Hkv;
    a.Np = Np;
    a.Nc = p->Nc;
    a.m = p->m;
    a.W = p->W;
    a.q_pos = p->q_pos;
    a.kv_pos0 = p->kv_pos0;
    a.scale_log2 = softmax_scale(p) * 1.4426950408889634f;
    return prefix_plan(a, p->d) ? HYB_OK : HYB_ERR_UNSUPPORTED;
}

// Checks and launch shared by the two compaction entry points: t holds, per
// cache, source, destination and row bytes; absent caches have both NULL.
static hyb_status compact_common(const hyb_problem *p, const int32_t *keep, int n_keep, int No,
                                 const CompactTensor *t, int n, cudaStream_t stream)
{
    if (!p || p->B <= 0 || p->Nc <= 0 || n_keep <= 0 || No < n_keep || !keep || !aligned4(keep))
        return HYB_ERR_INVALID_ARG;
    if (p->Nc >= (1 << 30) || No >= (1 << 30))
        return HYB_ERR_UNSUPPORTED;
    bool some = false;
    for (int i = 0; i < n; ++i) {
        if (!t[i].src != !t[i].dst)
            return HYB_ERR_INVALID_ARG;
        if (!t[i].src)
            continue;
        some = true;
        if (t[i].row_bytes <= 0 || t[i].row_bytes % 4 != 0 || (reinterpret_cast<uintptr_t>(t[i].src) & 3u) ||
            (reinterpret_cast<uintptr_t>(t[i].dst) & 3u))
            return HYB_ERR_INVALID_ARG;
        // rows move to lower indices while other rows are still read: no output
        // may share memory with any input or other output
        const uintptr_t d0 = reinterpret_cast<uintptr_t>(t[i].dst);
        const uintptr_t d1 = d0 + (uintptr_t)p->B * No * t[i].row_bytes;
        for (int k = 0; k < n; ++k) {
            const uintptr_t s0 = reinterpret_cast<uintptr_t>(t[k].src);
            const uintptr_t e0 = reinterpret_cast<uintptr_t>(t[k].dst);
            if (t[k].src && s0 < d1 && d0 < s0 + (uintptr_t)p->B * p->Nc * t[k].row_bytes)
                return HYB_ERR_INVALID_ARG;
            if (k != i && t[k].dst && e0 < d1 && d0 < e0 + (uintptr_t)p->B * No * t[k].row_bytes)
                return HYB_ERR_INVALID_ARG;
        }
        const uintptr_t k0 = reinterpret_cast<uintptr_t>(keep);
        if (k0 < d1 && d0 < k0 + (uintptr_t)p->B * n_keep * sizeof(int32_t))
            return HYB_ERR_INVALID_ARG;
    }
    if (!some)
        return HYB_ERR_INVALID_ARG;
    return cuda_status(launch_cache_compact(t, n, p->B, p->Nc, No, keep, n_keep, stream));
}

}  // namespace hyb

using namespace hyb;

extern "C" {

size_t hyb_prefix_workspace_size(const hyb_problem *p, int Np)
{
    PrefixParams a;
    return check_prefix(p, Np, a) == HYB_OK ? prefix_workspace(a, p->d) : 0;
}

hyb_status hyb_prefix_attn_fwd(const hyb_problem *p, int Np, const void *q, const void *kp, const void *vp,
                               const void *kc, const void *vc, const void *k_raw, const void *v_raw, void *o,
                               float *lse, void *ws, size_t ws_bytes, cudaStream_t stream)
{
    NvtxRange nvtx_range("hyb_prefix_attn_fwd");
    PrefixParams a;
    const hyb_status st = check_prefix(p, Np, a);
    if (st != HYB_OK)
        return st;
    if (!q || !o || !aligned16(q) || !aligned16(o) || !aligned4(lse) || !aligned4(p->q_pos) || !aligned4(p->kv_pos0))
        return HYB_ERR_INVALID_ARG;
    if (Np > 0 && (!kp || !vp || !aligned16(kp) || !aligned16(vp)))
        return HYB_ERR_INVALID_ARG;
    if (p->Nc > 0 && (!kc || !vc || !aligned16(kc) || !aligned16(vc)))
        return HYB_ERR_INVALID_ARG;
    if (p->W > 0 && (!k_raw || !v_raw || !aligned16(k_raw) || !aligned16(v_raw)))
        return HYB_ERR_INVALID_ARG;
    if (!ws_ok(ws, ws_bytes, prefix_workspace(a, p->d)))
        return HYB_ERR_WORKSPACE;
    a.o = static_cast<__nv_bfloat16 *>(o);
    a.lse = lse;
    return cuda_status(launch_prefix_attn(a, p->d, q, kp, vp, kc, vc, k_raw, v_raw, ws, stream));
}

hyb_status hyb_attn_weights(const hyb_problem *p, const void *q, const void *kc, const float *lse,
                            const int32_t *idx, int e0, float *acc, int accumulate, cudaStream_t stream)
{
    NvtxRange nvtx_range("hyb_attn_weights");
    hyb_status st = check_problem(p, false);
    if (st != HYB_OK)
        return st;
    if (e0 < 0 || !(p->scale >= 0.f) || p->Nc <= 0 || !q || !kc || !lse || !acc || !aligned16(q) || !aligned16(kc) ||
        !aligned4(lse) || !aligned4(acc) || !aligned4(idx) || !aligned4(p->q_pos))
        return HYB_ERR_INVALID_ARG;
    if (!idx != (p->topk <= 0))
        return HYB_ERR_INVALID_ARG;
    if (idx && p->Lq != 1)
        return HYB_ERR_UNSUPPORTED;   // one query token a call over a selection
    if ((long long)p->B * p->Lq * p->Hq >= (1LL << 31) || (long long)e0 + p->Nc >= (1LL << 30) ||
        p->W >= (1 << 30))
        return HYB_ERR_UNSUPPORTED;
    return cuda_status(launch_attn_weights(p->B, p->Lq, p->Hq, p->Hkv, p->d, p->Nc, p->m, p->W, e0, p->topk,
                                           softmax_scale(p), p->q_pos, q, kc, lse, idx, acc, accumulate != 0,
                                           stream, num_sms_current()));
}

hyb_status hyb_evict_select(const float *acc, int B, int Nc, const int32_t *n_valid, int n_keep, int n_first,
                            int n_last, int32_t *keep, cudaStream_t stream)
{
    NvtxRange nvtx_range("hyb_evict_select");
    if (!acc || !keep || B <= 0 || Nc <= 0 || n_keep <= 0 || n_first < 0 || n_last < 0 ||
        (long long)n_first + n_last > n_keep || !aligned4(acc) || !aligned4(n_valid) || !aligned4(keep))
        return HYB_ERR_INVALID_ARG;
    if (B > 65535 || Nc >= (1 << 30) || n_keep >= (1 << 30))
        return HYB_ERR_UNSUPPORTED;
    return cuda_status(launch_evict_select(acc, B, Nc, n_valid, n_keep, n_first, n_last, keep, stream,
                                           num_sms_current()));
}

hyb_status hyb_cache_compact(const hyb_problem *p, const int32_t *keep, int n_keep, int No, const void *kc,
                             const void *vc, const void *kic, const float *acc, void *kc_out, void *vc_out,
                             void *kic_out, float *acc_out, cudaStream_t stream)
{
    NvtxRange nvtx_range("hyb_cache_compact");
    if (!p || p->Hkv <= 0 || p->d <= 0)
        return HYB_ERR_INVALID_ARG;
    const long long kv = (long long)p->Hkv * p->d * 2;
    const CompactTensor t[] = {{kc, kc_out, kv}, {vc, vc_out, kv}, {kic, kic_out, (long long)p->di * 2}, {acc, acc_out, 4}};
    return compact_common(p, keep, n_keep, No, t, 4, stream);
}

hyb_status hyb_cache_compact_fp4(const hyb_problem *p, const int32_t *keep, int n_keep, int No,
                                 const uint8_t *kc_codes, const float *kc_qp, const uint8_t *vc_codes,
                                 const float *vc_qp, const uint8_t *kic_codes, const float *kic_qp,
                                 const float *acc, uint8_t *kc_codes_out, float *kc_qp_out,
                                 uint8_t *vc_codes_out, float *vc_qp_out, uint8_t *kic_codes_out,
                                 float *kic_qp_out, float *acc_out, cudaStream_t stream)
{
    NvtxRange nvtx_range("hyb_cache_compact_fp4");
    if (!p || p->Hkv <= 0 || p->d <= 0 || !kc_codes != !kc_qp || !vc_codes != !vc_qp || !kic_codes != !kic_qp)
        return HYB_ERR_INVALID_ARG;
    const long long codes = (long long)p->Hkv * p->d / 2, qp = (long long)p->Hkv * 8;
    const CompactTensor t[] = {{kc_codes, kc_codes_out, codes}, {kc_qp, kc_qp_out, qp},
                               {vc_codes, vc_codes_out, codes}, {vc_qp, vc_qp_out, qp},
                               {kic_codes, kic_codes_out, p->di / 2}, {kic_qp, kic_qp_out, 8},
                               {acc, acc_out, 4}};
    return compact_common(p, keep, n_keep, No, t, 7, stream);
}

}  // extern "C"
