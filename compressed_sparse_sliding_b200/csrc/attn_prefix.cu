// attn_prefix.cu -- stage 3 for a batch whose sequences share a prefix of
// compressed entries ("deepseek-v4" blog, section 1, HCA and SWA: one softmax
// over every visible compressed entry and the raw window).  Entries 0 .. Np-1
// are stored once, [Np, Hkv, D]; a sequence's own entries and window follow.
//
// Mathematics.  A softmax over a union of key sets joins exactly: with
// m_i = max s, l_i = sum exp(s - m_i), o_i = sum exp(s - m_i) v over set i,
//   o = sum_i exp(m_i - M) o_i / sum_i exp(m_i - M) l_i,  M = max_i m_i,
//   lse = M + log sum_i exp(m_i - M) l_i.
// So the shared entries are attended to by the query rows of ALL sequences as
// one tall matrix (each K / V tile is read once for 256 rows instead of once a
// sequence), the rest by each sequence's rows, and long key ranges are split
// over CTAs; prefix_combine_kernel joins the parts.
//
// Work item = one 128-key tile stream (a split of the shared entries, or of one
// sequence's own entries followed by its window) and two query tiles:
//   pair       two 128-row query tiles read the same keys (MMA-bound: K / V
//              tiles are fetched once for 256 rows);
//   alternate  where there is a single query tile, the two softmax warpgroups
//              take its even and odd key tiles, each with its own maximum, sum
//              and O, and store two parts (HBM-bound: twice the tiles in flight).
// A query tile holds hpt heads of one KV group x tpt tokens (hpt = min(g, 128),
// tpt = 128 / hpt), fetched by one TMA box; rows past hpt * tpt are not used.
//
// Roles (384 threads) as in the dense prefill kernel: warps 0-3 / 4-7 softmax
// and epilogue of query tile A / B (thread = TMEM lane = query row), warp 8 TMA
// producer (K and V rings of two 32 KB stages each), warp 9 MMA issue, all lanes
// active: it also zeroes, in shared memory, the V rows of a tile that no query
// of the item sees, so that whatever such cache rows hold (0 x NaN = NaN)
// never enters O.  Masked scores are replaced, not added to, for the same reason.
#include "common.cuh"

namespace hyb {

constexpr int kPfThreads = 384;
constexpr int kPfSoftmaxRegs = 208;   // 2 x 128 x 208 + 128 x 88 = 384 x 168 (the launch budget)
constexpr int kPfOtherRegs = 88;
constexpr int kPfBM = 128;
constexpr int kPfBN = 128;
constexpr int kPfStages = 2;
// The split is planned for this many SMs on every device, so that the workspace
// size is a function of the problem alone.
constexpr int kPfPlanSMs = 148;

struct PrefixParams {
    int B, Lq, Lkv, Hq, Hkv, g, Np, Nc, m, W;
    int hpt, tpt, nht;            // heads and tokens of a query tile, head tiles of a KV group
    int p_tiles, p_units, p_ns;   // shared entries: query tiles per KV head, items per KV head, splits
    int o_tiles, o_units, o_ns;   // own keys: the same per sequence and KV head
    int p_pair, o_pair;           // 1: pair, 0: alternate
    int p_parts, n_parts;         // partial results per row: of the shared entries, in all
    int n_items_p, n_items;
    long long rows;               // B * Lq * Hq
    float scale_log2;
    const int32_t *q_pos, *kv_pos0;
    float *part_o;                // [n_parts][rows][D], not normalised
    float2 *part_ml;              // [n_parts][rows] (maximum in log2 units, sum); sum 0: no key, part_o not written
    __nv_bfloat16 *o;             // [B, Lq, Hq, D]
    float *lse;                   // [B, Hq, Lq] or NULL
};

template <int D>
struct PrefixSmem {
    static constexpr int Q_BYTES = kPfBM * D * 2;
    static constexpr int KV_BYTES = kPfBN * D * 2;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = 2 * Q_BYTES;
    static constexpr int OFF_V = OFF_K + kPfStages * KV_BYTES;
    static constexpr int OFF_BAR = OFF_V + kPfStages * KV_BYTES;
    static constexpr int OFF_MISC = OFF_BAR + 32 * 8;
    static constexpr int BYTES = OFF_MISC + 16 * 4;
};

// barrier slots (two each from PB_KF on)
enum { PB_QF = 0, PB_QE = 1, PB_KF = 2, PB_KE = 4, PB_VF = 6, PB_VE = 8, PB_SF = 10, PB_PF = 12, PB_OF = 14,
       PB_OE = 16, PB_DONE = 18 };

struct PrefixItem {
    bool pre, pair;      // shared entries?  two query tiles?
    int b, kvh, part;    // sequence (own keys), KV head, first partial result
    int tok0[2], h0[2];  // first token (of the batch's B * Lq, or of the sequence) and head of each query tile
    bool val[2];         // warpgroup has work
    int ntok;            // tokens of the range tok0 counts in
    int nent;            // entries that some row of the item sees
    int rlo, nraw;       // first raw row and number of raw rows that some row sees
    int nte;             // entry tiles before the raw tiles
    int t0, nt;          // first key tile and number of key tiles of this split
    int nsteps;
    long long kv0;
};

// Entries visible to position pos: those ending before its window.
__device__ __forceinline__ int pf_visible(long long pos, int m, int W, int n)
{
    const long long a = pos - W + 1;
    if (a <= 0)
        return 0;
    const unsigned long long v = (unsigned long long)a < (1ull << 32) ? (unsigned)a / (unsigned)m
                                                                       : (unsigned long long)a / (unsigned)m;
    return v < (unsigned long long)n ? (int)v : n;
}

__device__ __forceinline__ int pf_pos(const PrefixParams &p, int flat)
{
    return p.q_pos ? p.q_pos[flat] : flat % p.Lq;
}

// The item w, computed by a whole warp (the positions of its tokens decide how
// many keys there are).
template <int D>
__device__ __forceinline__ PrefixItem prefix_item(const PrefixParams &p, int w, int lane)
{
    PrefixItem it;
    it.pre = w < p.n_items_p;
    int units, s, ns, u;
    if (it.pre) {
        units = p.p_units;
        ns = p.p_ns;
        it.pair = p.p_pair != 0;
        u = w % units;
        const int r = w / units;
        it.kvh = r % p.Hkv;
        s = r / p.Hkv;
        it.b = 0;
        it.part = it.pair ? s : 2 * s;
        it.ntok = p.B * p.Lq;
        it.kv0 = 0;
    } else {
        w -= p.n_items_p;
        units = p.o_units;
        ns = p.o_ns;
        it.pair = p.o_pair != 0;
        s = w % ns;
        int r = w / ns;
        u = r % units;
        r /= units;
        it.kvh = r % p.Hkv;
        it.b = r / p.Hkv;
        it.part = p.p_parts + (it.pair ? s : 2 * s);
        it.ntok = p.Lq;
        it.kv0 = p.kv_pos0 ? p.kv_pos0[it.b] : 0;
    }
    int pmax = INT_MIN, pmin = INT_MAX;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int tile = it.pair ? 2 * u + x : u;
        it.val[x] = tile < (it.pre ? p.p_tiles : p.o_tiles);
        it.tok0[x] = (tile / p.nht) * p.tpt;
        it.h0[x] = it.kvh * p.g + (tile % p.nht) * p.hpt;
        if (!it.val[x])
            continue;
        const int end = min(it.tok0[x] + p.tpt, it.ntok);
        for (int t = it.tok0[x] + lane; t < end; t += 32) {
            const int pos = pf_pos(p, it.pre ? t : it.b * p.Lq + t);
            pmax = max(pmax, pos);
            pmin = min(pmin, pos);
        }
    }
    pmax = __reduce_max_sync(0xffffffffu, pmax);
    pmin = __reduce_min_sync(0xffffffffu, pmin);
    const int nv = pf_visible(pmax, p.m, p.W, p.Np + p.Nc);
    it.nent = it.pre ? min(nv, p.Np) : max(nv - p.Np, 0);
    it.nte = (it.nent + kPfBN - 1) / kPfBN;
    it.rlo = it.nraw = 0;
    if (!it.pre && p.W > 0) {
        const long long lo = max(0ll, max(0ll, (long long)pmin - p.W + 1) - it.kv0);
        const long long hi = min((long long)p.Lkv - 1, (long long)pmax - it.kv0);
        if (hi >= lo) {
            it.rlo = (int)lo;
            it.nraw = (int)(hi - lo + 1);
        }
    }
    const int T = it.nte + (it.nraw + kPfBN - 1) / kPfBN;
    it.t0 = (int)((long long)T * s / ns);
    it.nt = (int)((long long)T * (s + 1) / ns) - it.t0;
    it.nsteps = it.pair ? it.nt : (it.nt + 1) / 2;
    return it;
}

// Key tile that warpgroup x works on in step i (relative to t0), or -1.
__device__ __forceinline__ int pf_tile(const PrefixItem &it, int i, int x)
{
    const int t = it.pair ? i : 2 * i + x;
    return i >= 0 && it.val[x] && t < it.nt ? t : -1;
}

template <int D>
__global__ void __launch_bounds__(kPfThreads, 1)
prefix_attn_kernel(const __grid_constant__ CUtensorMap tm_qp, const __grid_constant__ CUtensorMap tm_qo,
                   const __grid_constant__ CUtensorMap tm_kp, const __grid_constant__ CUtensorMap tm_vp,
                   const __grid_constant__ CUtensorMap tm_kc, const __grid_constant__ CUtensorMap tm_vc,
                   const __grid_constant__ CUtensorMap tm_kr, const __grid_constant__ CUtensorMap tm_vr,
                   const PrefixParams p)
{
    pdl_wait();      // launched as a programmatic dependent: the previous kernel's writes
    pdl_trigger();   // are visible from here on; the next kernel may start its launch
    using SM = PrefixSmem<D>;
    constexpr int NCB = D / 64;
    extern __shared__ __align__(1024) uint8_t pf_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(pf_smem_raw) + 1023) &
                                                ~(uintptr_t)1023);
    uint8_t *sQ = smem + SM::OFF_Q;
    uint8_t *sK = smem + SM::OFF_K;
    uint8_t *sV = smem + SM::OFF_V;
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + SM::OFF_BAR);
    int *misc = reinterpret_cast<int *>(smem + SM::OFF_MISC);
    volatile int *abort_flag = misc + 1;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(&bar[PB_QF], 1);
        mbar_init(&bar[PB_QE], 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar[PB_KF + s], 1);
            mbar_init(&bar[PB_KE + s], 1);
            mbar_init(&bar[PB_VF + s], 1);
            mbar_init(&bar[PB_VE + s], 1);
            mbar_init(&bar[PB_SF + s], 1);
            mbar_init(&bar[PB_PF + s], 128);
            mbar_init(&bar[PB_OF + s], 1);
            mbar_init(&bar[PB_OE + s], 128);
        }
        mbar_init(&bar[PB_DONE], 1);
        mbar_fence_init();
        misc[1] = 0;
    }
    if (warp == 9)
        tmem_alloc(reinterpret_cast<uint32_t *>(&misc[0]), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)misc[0];
    constexpr uint32_t TM_S[2] = {0, kPfBN};
    constexpr uint32_t TM_O[2] = {2 * kPfBN, 2 * kPfBN + 128};
    if (warp == 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPfOtherRegs));
        // ================================ producer ================================
        const uint32_t q_bytes = (uint32_t)p.hpt * p.tpt * D * 2;
        uint32_t kc = 0, vc = 0, nq = 0;
        bool ok = true;
        for (int w = blockIdx.x; ok && w < p.n_items; w += gridDim.x) {
            const PrefixItem it = prefix_item<D>(p, w, lane);
            if (lane == 0) {
                if (nq > 0 && !mbar_wait(&bar[PB_QE], (nq - 1) & 1, abort_flag))
                    ok = false;
                if (ok) {
                    const int nqt = it.pair && it.val[1] ? 2 : 1;
                    mbar_arrive_expect_tx(&bar[PB_QF], nqt * q_bytes);
                    for (int x = 0; x < nqt; ++x)
                        for (int cb = 0; cb < NCB; ++cb)
                            tma_load_4d(sQ + x * SM::Q_BYTES + cb * kPfBM * 128, it.pre ? &tm_qp : &tm_qo,
                                        &bar[PB_QF], cb * 64, it.h0[x], it.tok0[x], it.pre ? 0 : it.b);
                    ++nq;
                }
                const int per = it.pair ? 1 : 2;   // key tiles of a step
                for (int i = 0; ok && i < it.nt; i += per) {
                    for (int kv = 0; ok && kv < 2; ++kv) {
                        uint32_t &cnt = kv ? vc : kc;
                        uint8_t *ring = kv ? sV : sK;
                        uint64_t *full = &bar[kv ? PB_VF : PB_KF], *empty = &bar[kv ? PB_VE : PB_KE];
                        for (int j = i; j < min(i + per, it.nt); ++j) {
                            const int t = it.t0 + j;
                            const bool ent = t < it.nte;
                            const int row0 = ent ? t * kPfBN : it.rlo + (t - it.nte) * kPfBN;
                            const CUtensorMap *map = kv ? (!ent ? &tm_vr : it.pre ? &tm_vp : &tm_vc)
                                                        : (!ent ? &tm_kr : it.pre ? &tm_kp : &tm_kc);
                            const uint32_t st = cnt % kPfStages;
                            if (cnt >= kPfStages &&
                                !mbar_wait(&empty[st], ((cnt / kPfStages) - 1) & 1, abort_flag)) {
                                ok = false;
                                break;
                            }
                            mbar_arrive_expect_tx(&full[st], SM::KV_BYTES);
                            for (int cb = 0; cb < NCB; ++cb)
                                tma_load_4d(ring + st * SM::KV_BYTES + cb * kPfBN * 128, map, &full[st], cb * 64,
                                            it.kvh, row0, it.pre ? 0 : it.b);
                            ++cnt;
                        }
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        }
        if (lane == 0) {
            // unwinding: wait for the last copies issued into every slot
            if (nq > 0)
                drain_wait(&bar[PB_QF], (nq - 1) & 1);
            for (uint32_t c = (kc > kPfStages ? kc - kPfStages : 0); c < kc; ++c)
                drain_wait(&bar[PB_KF + c % kPfStages], (c / kPfStages) & 1);
            for (uint32_t c = (vc > kPfStages ? vc - kPfStages : 0); c < vc; ++c)
                drain_wait(&bar[PB_VF + c % kPfStages], (c / kPfStages) & 1);
        }
    } else if (warp == 9) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPfOtherRegs));
        // ================================ MMA issue ================================
        const uint32_t idesc_qk = idesc_bf16(kPfBM, kPfBN, false, false);
        const uint32_t idesc_pv = idesc_bf16(kPfBM, D, false, true);
        const uint32_t aQ = smem_u32(sQ), aK = smem_u32(sK), aV = smem_u32(sV);
        uint32_t kc = 0, vc = 0, nq = 0;
        uint32_t pcnt[2] = {0, 0};
        bool ok = true;
        // every lane waits; the warp goes on only if all of them got through
        auto wait = [&](int b, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(&bar[b], parity, abort_flag)) != 0;
        };
        for (int w = blockIdx.x; ok && w < p.n_items; w += gridDim.x) {
            const PrefixItem it = prefix_item<D>(p, w, lane);
            ok = wait(PB_QF, nq & 1);
            bool first_pv[2] = {true, true};
            bool waited_oe = nq == 0;
            for (int i = 0; ok && i <= it.nsteps; ++i) {
                for (int x = 0; ok && x < 2; ++x) {
                    const int tp = pf_tile(it, i - 1, x);
                    const int tc = i < it.nsteps ? pf_tile(it, i, x) : -1;
                    // stages are waited for by the first user of a tile
                    const bool first_use = !it.pair || x == 0;
                    if (tp >= 0) {
                        const uint32_t vs = vc % kPfStages;
                        if (first_use) {
                            if (!(ok = wait(PB_VF + vs, (vc / kPfStages) & 1)))
                                break;
                            const int t = it.t0 + tp;
                            const int seen = t < it.nte ? it.nent - t * kPfBN : it.nraw - (t - it.nte) * kPfBN;
                            if (seen < kPfBN) {
                                // rows that no query of the item sees take no part, whatever they hold
                                for (int cb = 0; cb < NCB; ++cb)
                                    for (int c = seen * 8 + lane; c < kPfBN * 8; c += 32)
                                        *reinterpret_cast<uint4 *>(sV + vs * SM::KV_BYTES + cb * kPfBN * 128 +
                                                                   c * 16) = make_uint4(0, 0, 0, 0);
                                fence_proxy_async_smem();
                                __syncwarp();
                            }
                        }
                        if (!waited_oe) {
                            // both epilogues of the previous item have read O
                            if (!(ok = wait(PB_OE + 0, (nq - 1) & 1) && wait(PB_OE + 1, (nq - 1) & 1)))
                                break;
                            waited_oe = true;
                        }
                        if (!(ok = wait(PB_PF + x, pcnt[x] & 1)))
                            break;
                        ++pcnt[x];
                        tc_fence_after();
                        if (lane == 0) {
#pragma unroll
                            for (int kk = 0; kk < kPfBN / 16; ++kk) {
                                const uint64_t db = sw128_desc(aV + vs * SM::KV_BYTES + kk * 16 * 128,
                                                               kPfBN * 128, 1024);
                                mma_bf16_ts(tmem + TM_O[x], tmem + TM_S[x] + kk * 8, db, idesc_pv,
                                            (first_pv[x] && kk == 0) ? 0u : 1u);
                            }
                        }
                        first_pv[x] = false;
                        if (!it.pair || x == 1 || !it.val[1]) {
                            if (lane == 0)
                                mma_commit(&bar[PB_VE + vs]);
                            ++vc;
                        }
                    }
                    if (tc >= 0) {
                        const uint32_t ks = kc % kPfStages;
                        if (first_use && !(ok = wait(PB_KF + ks, (kc / kPfStages) & 1)))
                            break;
                        tc_fence_after();
                        if (lane == 0) {
                            const uint32_t a = aQ + (it.pair ? x : 0) * SM::Q_BYTES;
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint64_t da = sw128_desc(a + (kk >> 2) * kPfBM * 128 + (kk & 3) * 32, 16,
                                                               1024);
                                const uint64_t db = sw128_desc(aK + ks * SM::KV_BYTES + (kk >> 2) * kPfBN * 128 +
                                                                   (kk & 3) * 32,
                                                               16, 1024);
                                mma_bf16_ss(tmem + TM_S[x], da, db, idesc_qk, kk > 0 ? 1u : 0u);
                            }
                            mma_commit(&bar[PB_SF + x]);
                        }
                        if (!it.pair || x == 1 || !it.val[1]) {
                            if (lane == 0)
                                mma_commit(&bar[PB_KE + ks]);
                            ++kc;
                        }
                    }
                }
                if (ok && lane == 0 && (i == it.nsteps - 1 || it.nsteps == 0))
                    mma_commit(&bar[PB_QE]);
            }
            if (!ok)
                break;
            if (!waited_oe &&   // one wait an item even without a PV
                !(ok = wait(PB_OE + 0, (nq - 1) & 1) && wait(PB_OE + 1, (nq - 1) & 1)))
                break;
            if (lane == 0)
                for (int x = 0; x < 2; ++x)
                    if (!first_pv[x])
                        mma_commit(&bar[PB_OF + x]);
            ++nq;
        }
        if (lane == 0) {
            mma_commit(&bar[PB_DONE]);
            drain_wait(&bar[PB_DONE], 0);
        }
    } else if (warp >= 10) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPfOtherRegs));
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPfSoftmaxRegs));
        // ========================== softmax + epilogue ==========================
        const int x = warp >> 2;            // 0: tile A, 1: tile B
        const int quad = warp & 3;
        const int row = quad * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t tS = tl + TM_S[x];
        const uint32_t tO = tl + TM_O[x];
        const int rtok = row / p.hpt, rhead = row % p.hpt;
        uint32_t scnt = 0, ocnt = 0;
        bool ok = true;
        for (int w = blockIdx.x; ok && w < p.n_items; w += gridDim.x) {
            const PrefixItem it = prefix_item<D>(p, w, lane);
            const int tok = it.tok0[x] + rtok;
            const int h = it.h0[x] + rhead;
            const bool valid_row = it.val[x] && rtok < p.tpt && tok < it.ntok && h < (it.kvh + 1) * p.g;
            const int flat = it.pre ? tok : it.b * p.Lq + tok;
            int nv = 0, wlo = 0, whi = -1;   // visible entries; window as raw rows wlo..whi
            if (valid_row) {
                const long long pos = pf_pos(p, flat);
                nv = pf_visible(pos, p.m, p.W, p.Np + p.Nc);
                nv = it.pre ? min(nv, p.Np) : max(nv - p.Np, 0);
                if (it.nraw > 0) {
                    wlo = (int)max(0ll, max(0ll, pos - p.W + 1) - it.kv0);
                    whi = (int)min((long long)p.Lkv - 1, max(-1ll, pos - it.kv0));
                }
            }
            float m_ref = -INFINITY, l_sum = 0.f;
            bool any = false;
            for (int i = 0; i < it.nsteps; ++i) {
                const int tt = pf_tile(it, i, x);
                if (tt < 0)
                    continue;
                // valid columns c_lo..c_hi of this key tile for this row
                const int t = it.t0 + tt;
                int c_lo = 0, c_hi;
                if (t < it.nte) {
                    c_hi = min(nv - 1 - t * kPfBN, kPfBN - 1);
                } else {
                    const int base = it.rlo + (t - it.nte) * kPfBN;
                    c_lo = max(0, min(wlo - base, kPfBN));
                    c_hi = max(-1, min(whi - base, kPfBN - 1));
                }
                const bool full = __all_sync(0xffffffffu, c_lo == 0 && c_hi == kPfBN - 1);
                if (!__all_sync(0xffffffffu, mbar_wait(&bar[PB_SF + x], scnt & 1, abort_flag))) {
                    ok = false;
                    break;
                }
                ++scnt;
                tc_fence_after();
                float sv[kPfBN];
#pragma unroll
                for (int c = 0; c < kPfBN / 32; ++c)
                    tmem_ld32(tS + c * 32, *reinterpret_cast<float(*)[32]>(&sv[c * 32]));
                tmem_ld_wait();
                if (!full) {
#pragma unroll
                    for (int c = 0; c < kPfBN; ++c)
                        sv[c] = (c >= c_lo && c <= c_hi) ? sv[c] : -INFINITY;
                }
                // row max over eight independent 3-input max chains
                float tmax;
                {
                    float mk[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        float a = fmax3f(sv[16 * k], sv[16 * k + 1], sv[16 * k + 2]);
#pragma unroll
                        for (int q = 3; q < 15; q += 2)
                            a = fmax3f(a, sv[16 * k + q], sv[16 * k + q + 1]);
                        mk[k] = fmaxf(a, sv[16 * k + 15]);
                    }
                    tmax = fmax3f(fmax3f(mk[0], mk[1], mk[2]), fmax3f(mk[3], mk[4], mk[5]),
                                  fmaxf(mk[6], mk[7]));
                }
                tmax *= p.scale_log2;  // the scale is positive
                // the reference maximum moves (and O is rescaled) only when a
                // tile raises it by more than 2^8
                float alpha = 1.f;
                if (tmax > m_ref + 8.f) {
                    alpha = (m_ref == -INFINITY) ? 0.f : ex2_approx(m_ref - tmax);
                    m_ref = tmax;
                    l_sum *= alpha;
                }
                if (any && __any_sync(0xffffffffu, alpha != 1.f)) {
                    // O holds every earlier PV (S_full covers all MMAs issued before this QK)
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        float ov[32];
                        tmem_ld32(tO + c * 32, ov);
                        tmem_ld_wait();
#pragma unroll
                        for (int q = 0; q < 32; ++q)
                            ov[q] *= alpha;
                        tmem_st32(tO + c * 32, ov);
                    }
                }
                const float mu = (m_ref == -INFINITY) ? 0.f : m_ref;
                // P = exp2(s * scale - mu), rounded to bf16 (the MMA operand; its
                // relative error 2^-9 a term averages out below the output's own
                // rounding) over the first 64 columns of S; the row sum is of the
                // fp32 values
                const uint64_t sc2 = f2(p.scale_log2, p.scale_log2);
                const uint64_t nmu2 = f2(-mu, -mu);
                uint64_t lacc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                for (int c = 0; c < kPfBN / 32; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int q = 0; q < 32; q += 2) {
                        float x0, x1;
                        f2_split(fma_f2(f2(sv[c * 32 + q], sv[c * 32 + q + 1]), sc2, nmu2), x0, x1);
                        const float e0 = ex2_approx(x0);
                        const float e1 = ex2_approx(x1);
                        lacc[(q >> 1) & 3] = add_f2(lacc[(q >> 1) & 3], f2(e0, e1));
                        pk[q >> 1] = pack_bf16x2(e0, e1);
                    }
                    tmem_st16(tS + c * 16, pk);
                }
                {
                    float a0, a1, b0, b1;
                    f2_split(add_f2(lacc[0], lacc[1]), a0, a1);
                    f2_split(add_f2(lacc[2], lacc[3]), b0, b1);
                    l_sum += (a0 + a1) + (b0 + b1);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&bar[PB_PF + x]);
                any = true;
            }
            if (!ok)
                break;
            // epilogue: this item's part of the row
            if (any) {
                if (!__all_sync(0xffffffffu, mbar_wait(&bar[PB_OF + x], ocnt & 1, abort_flag))) {
                    ok = false;
                    break;
                }
                ++ocnt;
                tc_fence_after();
            }
            const size_t at = (size_t)(it.part + (it.pair ? 0 : x)) * p.rows + (size_t)flat * p.Hq + h;
            if (valid_row)
                p.part_ml[at] = make_float2(m_ref, l_sum);
            if (any) {
                const bool store = valid_row && l_sum != 0.f;
                float *orow = p.part_o + at * D;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float ov[32];
                    tmem_ld32(tO + c * 32, ov);
                    tmem_ld_wait();
                    if (store) {
#pragma unroll
                        for (int q = 0; q < 32; q += 4)
                            *reinterpret_cast<float4 *>(orow + c * 32 + q) =
                                make_float4(ov[q], ov[q + 1], ov[q + 2], ov[q + 3]);
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(&bar[PB_OE + x]);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc((uint32_t)misc[0], 512);
    }
}

// Joins the parts of each row: D / 4 lanes per row, four channels a lane.
template <int D>
__global__ void __launch_bounds__(256)
prefix_combine_kernel(const PrefixParams p)
{
    pdl_wait();
    pdl_trigger();
    constexpr int LPR = D / 4;
    const long long row = ((long long)blockIdx.x * 256 + threadIdx.x) / LPR;
    const int c = (threadIdx.x % LPR) * 4;
    if (row >= p.rows)
        return;
    float M = -INFINITY;
    bool some = false;
    for (int i = 0; i < p.n_parts; ++i) {
        const float2 ml = p.part_ml[(size_t)i * p.rows + row];
        if (ml.y != 0.f) {
            M = fmaxf(M, ml.x);
            some = true;
        }
    }
    float L = 0.f, a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
    for (int i = 0; i < p.n_parts; ++i) {
        const size_t at = (size_t)i * p.rows + row;
        const float2 ml = p.part_ml[at];
        if (ml.y != 0.f) {
            const float w = exp2f(ml.x - M);
            const float4 v = *reinterpret_cast<const float4 *>(p.part_o + at * D + c);
            L += w * ml.y;
            a0 += w * v.x;
            a1 += w * v.y;
            a2 += w * v.z;
            a3 += w * v.w;
        }
    }
    const float inv = some ? 1.f / L : 0.f;
    uint2 v;
    v.x = pack_bf16x2(a0 * inv, a1 * inv);
    v.y = pack_bf16x2(a2 * inv, a3 * inv);
    *reinterpret_cast<uint2 *>(p.o + row * D + c) = v;
    if (c == 0 && p.lse) {
        const long long bt = row / p.Hq;
        const int h = (int)(row % p.Hq);
        const long long b = bt / p.Lq, t = bt % p.Lq;
        p.lse[(b * p.Hq + h) * p.Lq + t] = some ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
    }
}

// How the work is split: fills the tiling and the split of p.
static void prefix_plan(PrefixParams &p)
{
    auto up = [](long long a, long long b) { return (a + b - 1) / b; };
    p.g = p.Hq / p.Hkv;
    p.hpt = p.g < kPfBM ? p.g : kPfBM;
    p.tpt = kPfBM / p.hpt;
    p.nht = (int)up(p.g, p.hpt);
    p.p_tiles = (int)(up((long long)p.B * p.Lq, p.tpt) * p.nht);
    p.o_tiles = (int)(up(p.Lq, p.tpt) * p.nht);
    p.p_pair = p.p_tiles > 1;
    p.o_pair = p.o_tiles > 1;
    p.p_units = p.p_pair ? (p.p_tiles + 1) / 2 : 1;
    p.o_units = p.o_pair ? (p.o_tiles + 1) / 2 : 1;
    p.rows = (long long)p.B * p.Lq * p.Hq;
    // key tiles of the two streams (raw rows: those of consecutive positions)
    const long long span = p.Lq < 2 * p.tpt ? p.Lq : 2 * p.tpt;
    long long raw = p.W > 0 ? (long long)p.W + span - 1 : 0;
    if (raw > p.Lkv)
        raw = p.Lkv;
    const long long Tp = up(p.Np, kPfBN), To = up(p.Nc, kPfBN) + up(raw, kPfBN);
    const long long Ip = Tp ? (long long)p.p_units * p.Hkv : 0;
    const long long Io = p.Nc > 0 || p.W > 0 ? (long long)p.o_units * p.Hkv * p.B : 0;
    // Equal chunks of key tiles for w waves of CTAs; of these, the least
    // waves x (chunk + what an item costs beside its tiles, about three tiles).
    const long long total = Ip * Tp + Io * To;
    long long best = -1, chunk = 1;
    for (long long w = 1; w <= 4; ++w) {
        long long c = up(total, w * kPfPlanSMs);
        if (c < 1)
            c = 1;
        for (int it = 0; it < 64 && Ip * up(Tp, c) + Io * up(To > 0 ? To : 1, c) > w * kPfPlanSMs; ++it) {
            if (c >= Tp && c >= To)
                break;
            c += up(c, 16);
        }
        const long long items = Ip * up(Tp, c) + Io * up(To > 0 ? To : 1, c);
        const long long longest = c < (Tp > To ? Tp : To) ? c : (Tp > To ? Tp : To);
        const long long cost = up(items, kPfPlanSMs) * (longest + 3);
        if (best < 0 || cost < best) {
            best = cost;
            chunk = c;
        }
    }
    p.p_ns = Ip ? (int)up(Tp, chunk) : 0;
    p.o_ns = Io ? (int)up(To > 0 ? To : 1, chunk) : 0;
    p.p_parts = p.p_ns * (p.p_pair ? 1 : 2);
    p.n_parts = p.p_parts + p.o_ns * (p.o_pair ? 1 : 2);
    p.n_items_p = (int)(Ip * p.p_ns);
    p.n_items = (int)(p.n_items_p + Io * p.o_ns);
}

static size_t prefix_ml_bytes(const PrefixParams &p)
{
    return ((size_t)p.n_parts * p.rows * sizeof(float2) + 255) & ~(size_t)255;
}

size_t prefix_workspace_bytes(int B, int Lq, int Lkv, int Hq, int Hkv, int d, int Np, int Nc, int W)
{
    PrefixParams p = {};
    p.B = B;
    p.Lq = Lq;
    p.Lkv = Lkv;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.Np = Np;
    p.Nc = Nc;
    p.W = W;
    prefix_plan(p);
    return prefix_ml_bytes(p) + (((size_t)p.n_parts * p.rows * d * sizeof(float) + 255) & ~(size_t)255);
}

template <int D>
static cudaError_t launch_prefix_t(PrefixParams &p, const void *q, const void *kp, const void *vp,
                                   const void *kc, const void *vc, const void *kr, const void *vr, void *ws,
                                   cudaStream_t stream, int num_sms)
{
    using SM = PrefixSmem<D>;
    p.part_ml = static_cast<float2 *>(ws);
    p.part_o = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + prefix_ml_bytes(p));
    if (p.n_items > 0) {
        // absent tensors: a map that no copy uses
        const bool own = p.Nc > 0, raw = p.W > 0 && p.Lkv > 0;
        CUtensorMap mqp, mqo, mkp, mvp, mkc, mvc, mkr, mvr;
        bool ok = make_map(&mqp, q, D, p.Hq, p.B * p.Lq, 1, p.hpt, p.tpt);
        ok &= make_map(&mqo, q, D, p.Hq, p.Lq, p.B, p.hpt, p.tpt);
        ok &= make_map(&mkp, p.Np ? kp : q, D, p.Hkv, p.Np ? p.Np : 1, 1, 1, kPfBN);
        ok &= make_map(&mvp, p.Np ? vp : q, D, p.Hkv, p.Np ? p.Np : 1, 1, 1, kPfBN);
        ok &= make_map(&mkc, own ? kc : q, D, p.Hkv, own ? p.Nc : 1, own ? p.B : 1, 1, kPfBN);
        ok &= make_map(&mvc, own ? vc : q, D, p.Hkv, own ? p.Nc : 1, own ? p.B : 1, 1, kPfBN);
        ok &= make_map(&mkr, raw ? kr : q, D, p.Hkv, raw ? p.Lkv : 1, raw ? p.B : 1, 1, kPfBN);
        ok &= make_map(&mvr, raw ? vr : q, D, p.Hkv, raw ? p.Lkv : 1, raw ? p.B : 1, 1, kPfBN);
        if (!ok)
            return cudaErrorInvalidValue;
        const size_t smem = 1024 + SM::BYTES;
        auto kern = prefix_attn_kernel<D>;
        // one CTA per SM: it takes all of the tensor memory
        const size_t ask = smem < 120 * 1024 ? 120 * 1024 : smem;
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ask);
        if (e != cudaSuccess)
            return e;
        e = check_reg_split(kern, kPfThreads, 256, kPfSoftmaxRegs, kPfOtherRegs);
        if (e != cudaSuccess)
            return e;
        const int grid = p.n_items < num_sms ? p.n_items : num_sms;
        e = launch_pdl(kern, dim3((unsigned)grid), dim3(kPfThreads), ask, stream, mqp, mqo, mkp, mvp, mkc, mvc,
                       mkr, mvr, p);
        if (e != cudaSuccess)
            return e;
    }
    const long long blocks = (p.rows * (D / 4) + 255) / 256;
    return launch_pdl(prefix_combine_kernel<D>, dim3((unsigned)blocks), dim3(256), 0, stream, p);
}

cudaError_t launch_prefix_attn(int B, int Lq, int Lkv, int Hq, int Hkv, int d, int Np, int Nc, int m, int W,
                               float scale, const int32_t *q_pos, const int32_t *kv_pos0, const void *q,
                               const void *kp, const void *vp, const void *kc, const void *vc, const void *kr,
                               const void *vr, void *o, float *lse, void *ws, cudaStream_t stream, int num_sms)
{
    PrefixParams p = {};
    p.B = B;
    p.Lq = Lq;
    p.Lkv = Lkv;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.Np = Np;
    p.Nc = Nc;
    p.m = m;
    p.W = W;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.q_pos = q_pos;
    p.kv_pos0 = kv_pos0;
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.lse = lse;
    prefix_plan(p);
    return d == 128 ? launch_prefix_t<128>(p, q, kp, vp, kc, vc, kr, vr, ws, stream, num_sms)
                    : launch_prefix_t<64>(p, q, kp, vp, kc, vc, kr, vr, ws, stream, num_sms);
}

}  // namespace hyb
