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
// Work item = one stream of 128-key tiles (a piece of the shared entries, or of
// one sequence's own entries followed by its window) and two query tiles:
//   pair       two 128-row query tiles read the same keys (MMA-bound: K / V
//              tiles are fetched once for 256 rows);
//   alternate  where there is a single query tile, the two softmax warpgroups
//              take its even and odd key tiles, each with its own maximum, sum
//              and O (HBM-bound: twice the tiles in flight), and store two parts
//              (or join them in TMEM, where every warp can read both O's of its
//              lanes, if nothing else follows).
// Where a sequence's own query rows fill the tiles (chunks of a prompt), or the
// prefix is short, the shared entries are not taken apart: an item's stream then is
// prefix, own entries, window, and if no item is cut the kernel writes o itself, with
// no parts and no second kernel.  prefix_plan takes whichever way it reckons faster.
// A query tile holds hpt heads of one KV group x tpt tokens (hpt = min(g, 128),
// tpt = 128 / hpt), fetched by one TMA box; rows past hpt * tpt are not used.
//
// Measured (one B200, both kernels, d = 128): two query tiles take a key tile in
// about 3900 clocks (1.2 PFLOP/s over the GPU; 2048 of them MMAs); 64 sequences, 64 / 1
// heads over 16384 shared and 2048 own entries: 62 us (0.6 PFLOP/s); 64 / 8 heads over
// 1024 and 64: 34 us, most of it what an item costs beside its tiles; chunks of 256
// tokens behind 2048 entries: 63 us.  Short items are bound by instruction fetch (the
// SM's instruction cache hits 83 % there, 95 % and more with long streams): keeping the
// code of the item loop short was worth more than fewer operations in it.
//
// Roles (640 threads):
//   warps 0-7   softmax + epilogue of query tile (or key stream) A, warps 8-15 of
//               B: two threads per TMEM lane (= query row), one for each half of the
//               tile's 128 keys; they exchange the row maximum through shared
//               memory.  A single thread per row issued an instruction every four
//               to five clocks whatever its work, and with two such warps a
//               scheduler the softmax took 2200 clocks a tile.
//   warp 16     TMA producer (K and V rings of two 32 KB stages each).
//   warps 17, 18 MMA issue for A and for B.  One thread for both left the tensor
//               pipe idle while it walked from barrier to barrier (a key tile of
//               a pair took 4650 clocks, 2048 of them MMAs); with a warp each the
//               two chains only meet in the tensor pipe.  They also zero, in shared memory, the
//               V rows of a tile that no query of the item sees, so that whatever
//               such cache rows hold (0 x NaN = NaN) never enters O.  Masked
//               scores are replaced, not added to, for the same reason.
//   warp 19     works out the items (the positions of an item's tokens decide how
//               many keys it has) three ahead, so that no role waits for global
//               loads between items.
#include <atomic>

#include "common.cuh"

namespace hyb {

// The phase of the given parity has completed (a try may sleep for a while first).
__device__ __forceinline__ bool mbar_test_wait(uint32_t addr, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(addr), "r"(parity)
        : "memory");
    return ok != 0;
}

// Bounded wait that tries the barrier some times before it looks at the clock
// and the limit (a load from global memory, several hundred clocks): the waits
// of these kernels are short and many, and their code is kept short (a role's loop
// runs once a tile, so what it fetches counts).  Gives up when the CTA's abort flag
// is up, or the limit expires (which raises it); `tries` is wait_tries().
__device__ __forceinline__ bool mbar_wait_short(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int tries)
{
    const uint32_t addr = smem_u32(bar);
    if (mbar_test_wait(addr, parity))
        return true;
    uint64_t t0 = 0;
#pragma unroll 1
    for (int it = 0;; ++it) {
        // (a try may sleep past a shortened limit)
        if (tries ? mbar_try_wait(addr, parity) : mbar_test_wait(addr, parity))
            return true;
        if (*abort_flag)
            return false;
        if (it < tries)
            continue;
        const uint64_t t = global_ns();
        if (t0 == 0)
            t0 = t;
        if (t - t0 > *reinterpret_cast<volatile uint64_t *>(&g_wait_limit_ns) || timed_out_somewhere()) {
            set_error(HYB_ERR_DEVICE_TIMEOUT);
            *abort_flag = 1;
            return false;
        }
    }
}

// None where the limit has been shortened.
__device__ __forceinline__ int wait_tries()
{
    return *reinterpret_cast<volatile uint64_t *>(&g_wait_limit_ns) >= kWaitLimitNs ? 64 : 0;
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t pred;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(pred));
    return pred != 0;
}

constexpr int kPfThreads = 640;
constexpr int kPfSoftmaxThreads = 512;
constexpr int kPfSoftmaxRegs = 104;   // 512 x 104 + 128 x 64 = 640 x 96 (the launch budget)
constexpr int kPfOtherRegs = 64;
constexpr int kPfBM = 128;
constexpr int kPfBN = 128;
constexpr int kPfStages = 2;
constexpr int kPfItemSlots = 3;
constexpr int kPfPolyPairs = 2;       // of eight pairs of exponentials
// The split is planned for this many SMs on every device, so that the workspace
// size is a function of the problem alone.
constexpr int kPfPlanSMs = 148;

struct PrefixParams {
    int B, Lq, Lkv, Hq, Hkv, g, Np, Nc, m, W;
    int hpt, tpt, nht;            // heads and tokens of a query tile, head tiles of a KV group
    int p_tiles, p_units;         // shared entries: query tiles and items per KV head
    int o_tiles, o_units;         // own keys: the same per sequence and KV head
    int p_pair, o_pair;           // 1: pair, 0: alternate
    int p_ns, p_pieces;           // shared entries: pieces of an item's keys, pieces in all
    // Own keys, as one stream of items of o_len units each (o_over of them stand
    // for an item's cost beside its tiles): CTAs below o_rem, which have one
    // piece of the shared entries more, take o_a units each, the others o_b.
    int o_len, o_over, o_rem, o_a, o_b, o_total;
    int ctas, ctas_used;          // planned for, and with work
    int p_parts, n_parts;         // partial results per row: of the shared entries, in all (upper bound)
    int merged, direct;           // own items go through the shared entries too; and write o themselves
    long long rows;               // B * Lq * Hq
    float scale_log2;
    const int32_t *q_pos, *kv_pos0;
    float *part_o;                // [n_parts][rows][D], not normalised
    float2 *part_ml;              // [n_parts][rows] (maximum in log2 units, sum); sum 0: no key, part_o not written
    __nv_bfloat16 *o;             // [B, Lq, Hq, D]
    float *lse;                   // [B, Hq, Lq] or NULL
};

// 2^x for a pair without the exponential unit: x = i + f with i the nearest
// integer (read off the low bits of x + 1.5 2^23), 2^f by its degree-5 minimax
// polynomial on [-1/2, 1/2] with 2^0 = 1 (fitted by iteratively reweighted least
// squares; 1.7e-7 off at most in fp32, relative, where the unit is 2^-22: lse is as good as
// with the unit alone), times 2^i from i in the exponent field.  Below -126 (masked
// scores are -infinity) the result is 0; x <= 8 here.  A NaN stays one, through the
// product (added to the exponent field, i would turn NaN's bits into those of a large
// number).
__device__ __forceinline__ void exp2_poly2(float x0, float x1, float &e0, float &e1)
{
    const uint64_t x = f2(x0, x1);
    const uint64_t t = add_f2(x, f2(12582912.f, 12582912.f));
    const uint64_t i = add_f2(t, f2(-12582912.f, -12582912.f));
    const uint64_t f = fma_f2(i, f2(-1.f, -1.f), x);
    uint64_t q = fma_f2(f, f2(0.00132647273f, 0.00132647273f), f2(0.00967151299f, 0.00967151299f));
    q = fma_f2(q, f, f2(0.0555073358f, 0.0555073358f));
    q = fma_f2(q, f, f2(0.240222424f, 0.240222424f));
    q = fma_f2(q, f, f2(0.693147004f, 0.693147004f));
    q = fma_f2(q, f, f2(1.f, 1.f));
    float t0, t1;
    f2_split(t, t0, t1);
    f2_split(mul_f2(q, f2(__uint_as_float((__float_as_uint(t0) << 23) + 0x3f800000u),
                          __uint_as_float((__float_as_uint(t1) << 23) + 0x3f800000u))), e0, e1);
    e0 = x0 < -126.f ? 0.f : e0;
    e1 = x1 < -126.f ? 0.f : e1;
}

// A work item, as the roles read it from shared memory.
struct PrefixItem {
    int last;            // 1: no further item
    int pre, pair;       // shared entries?  two query tiles?
    int b, kvh, part;    // sequence (own keys), KV head, first partial result
    int tok0[2], h0[2];  // first token (of the batch's B * Lq, or of the sequence) and head of each query tile
    int val1;            // the second query tile exists (pair)
    int ntok;            // tokens of the range tok0 counts in
    int npre, nent;      // shared and own entries that some row of the item sees
    int rlo, nraw;       // first raw row and number of raw rows that some row sees
    int ntp, nte;        // tiles: shared entries, own entries (then raw rows)
    int t0, nt;          // first key tile and number of key tiles of this piece
};

// What one token of an item sees.
struct PrefixToken {
    int nv;              // entries, shared and own
    int wlo, whi;        // raw rows
};

// Key tile t of an item: 0 shared entries, 1 own entries, 2 raw rows; and its number
// among its kind.
__device__ __forceinline__ int pf_kind(const PrefixItem &it, int &t)
{
    if (t < it.ntp)
        return 0;
    t -= it.ntp;
    if (t < it.nte)
        return 1;
    t -= it.nte;
    return 2;
}

template <int D>
struct PrefixSmem {
    static constexpr int Q_BYTES = kPfBM * D * 2;
    static constexpr int KV_BYTES = kPfBN * D * 2;
    static constexpr int STAGE_BYTES = 32 * 32;                        // per softmax warp: 32 rows x 8 channels
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = 2 * Q_BYTES;
    static constexpr int OFF_V = OFF_K + kPfStages * KV_BYTES;
    static constexpr int OFF_ST = OFF_V + kPfStages * KV_BYTES;
    static constexpr int OFF_MAX = OFF_ST + 16 * STAGE_BYTES;          // per softmax thread: a tile's maximum
    static constexpr int OFF_TOK = OFF_MAX + kPfSoftmaxThreads * 4;
    static constexpr int OFF_ITEM = OFF_TOK + kPfItemSlots * 256 * (int)sizeof(PrefixToken);
    static constexpr int OFF_BAR = (OFF_ITEM + kPfItemSlots * (int)sizeof(PrefixItem) + 15) / 16 * 16;
    static constexpr int OFF_MISC = OFF_BAR + 40 * 8;
    static constexpr int BYTES = OFF_MISC + 16 * 4;
};
static_assert(1024 + PrefixSmem<128>::BYTES <= 227 * 1024, "shared memory of a CTA");

// barrier slots (two each from PB_KF on, three item slots)
enum { PB_QF = 0, PB_QE = 1, PB_KF = 2, PB_KE = 4, PB_VF = 6, PB_VE = 8, PB_SF = 10, PB_PF = 12, PB_OF = 14,
       PB_OE = 16, PB_IF = 18, PB_IE = 21, PB_DONE = 24, PB_MEET = 25, PB_MEET4 = 33, PB_TURN = 37 };

// Entries visible to position pos: those ending before its window.
__device__ __forceinline__ int pf_visible(long long pos, int m, int W, int n)
{
    const long long a = pos - W + 1;
    if (a <= 0)
        return 0;
    const unsigned v = (unsigned)a / (unsigned)m;     // positions are 32-bit
    return v < (unsigned)n ? (int)v : n;
}

// First unit of CTA k's share of the own-key stream, and the CTA a unit is in.
__host__ __device__ __forceinline__ int pf_share(const PrefixParams &p, int k)
{
    const long long u = k < p.o_rem ? (long long)k * p.o_a
                                    : (long long)p.o_rem * p.o_a + (long long)(k - p.o_rem) * p.o_b;
    return u < p.o_total ? (int)u : p.o_total;
}

__host__ __device__ __forceinline__ int pf_cta(const PrefixParams &p, int u)
{
    const int head = p.o_rem * p.o_a;
    return u < head ? u / p.o_a : p.o_rem + (u - head) / p.o_b;
}

// a * b / c of non-negative numbers (a 64-bit division is a hundred instructions,
// which the items of short streams would fetch again and again).
__device__ __noinline__ int pf_muldiv64(int a, int b, int c)
{
    return (int)((long long)a * b / c);
}

__device__ __forceinline__ int pf_muldiv(int a, int b, int c)
{
    return __umulhi((unsigned)a, (unsigned)b) == 0 ? (int)((unsigned)a * (unsigned)b / (unsigned)c)
                                                   : pf_muldiv64(a, b, c);
}

// Key tiles before unit u of an item of T tiles.
__device__ __forceinline__ int pf_cut(const PrefixParams &p, int T, int u)
{
    return pf_muldiv(T, max(u - p.o_over, 0), p.o_len - p.o_over);
}

// Works out one item (whole warp): piece `s` of p_ns of the shared entries for
// item i, or units [u0, u1) of own-key item i.
__device__ __forceinline__ void prefix_item(const PrefixParams &p, bool pre, int i, int s, int u0, int u1, int lane,
                                            PrefixItem &out, PrefixToken *tokens)
{
    PrefixItem it;
    it.last = 0;
    it.pre = pre;
    int u;
    if (pre) {
        it.pair = p.p_pair;
        u = i % p.p_units;
        it.kvh = i / p.p_units;
        it.b = 0;
        it.part = it.pair ? s : 2 * s;
        it.ntok = p.B * p.Lq;
    } else {
        it.pair = p.o_pair;
        u = i % p.o_units;
        const int r = i / p.o_units;
        it.kvh = r % p.Hkv;
        it.b = r / p.Hkv;
        it.part = p.p_parts + (it.pair ? s : 2 * s);
        it.ntok = p.Lq;
    }
    const long long kv0 = !pre && p.kv_pos0 ? p.kv_pos0[it.b] : 0;
    const int tiles = pre ? p.p_tiles : p.o_tiles;
    int nmax = 0, rlo = INT_MAX, rhi = -1;
    it.val1 = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int tile = it.pair ? 2 * u + x : u;
        it.tok0[x] = (tile / p.nht) * p.tpt;
        it.h0[x] = it.kvh * p.g + (tile % p.nht) * p.hpt;
        if (tile >= tiles || (x == 1 && !it.pair))
            continue;
        it.val1 = x;
        for (int t = lane; t < p.tpt; t += 32) {
            PrefixToken tk = {0, 0, -1};
            if (it.tok0[x] + t < it.ntok) {
                const int flat = (pre ? 0 : it.b * p.Lq) + it.tok0[x] + t;
                const long long pos = p.q_pos ? p.q_pos[flat] : flat % p.Lq;
                tk.nv = pf_visible(pos, p.m, p.W, p.Np + p.Nc);
                nmax = max(nmax, tk.nv);
                if (!pre && p.W > 0) {
                    const long long lo = max(0ll, max(0ll, pos - p.W + 1) - kv0);
                    const long long hi = min((long long)p.Lkv - 1, pos - kv0);
                    if (hi >= lo) {
                        tk.wlo = (int)lo;
                        tk.whi = (int)hi;
                        rlo = min(rlo, tk.wlo);
                        rhi = max(rhi, tk.whi);
                    }
                }
            }
            tokens[x * 128 + t] = tk;
        }
    }
    nmax = __reduce_max_sync(0xffffffffu, nmax);
    it.npre = pre || p.merged ? min(nmax, p.Np) : 0;
    it.nent = pre ? 0 : max(nmax - p.Np, 0);
    it.rlo = __reduce_min_sync(0xffffffffu, rlo);
    rhi = __reduce_max_sync(0xffffffffu, rhi);
    it.nraw = rhi >= 0 ? rhi - it.rlo + 1 : 0;
    it.ntp = (it.npre + kPfBN - 1) / kPfBN;
    it.nte = (it.nent + kPfBN - 1) / kPfBN;
    const int T = it.ntp + it.nte + (it.nraw + kPfBN - 1) / kPfBN;
    if (pre) {
        it.t0 = pf_muldiv(T, s, p.p_ns);
        it.nt = pf_muldiv(T, s + 1, p.p_ns) - it.t0;
    } else {
        it.t0 = pf_cut(p, T, u0);
        it.nt = (u1 == p.o_len ? T : pf_cut(p, T, u1)) - it.t0;
    }
    if (lane == 0)
        out = it;
}

template <int D>
__global__ void __launch_bounds__(kPfThreads, 1)
prefix_attn_kernel(const __grid_constant__ CUtensorMap tm_qp, const __grid_constant__ CUtensorMap tm_qo,
                   const __grid_constant__ CUtensorMap tm_kp, const __grid_constant__ CUtensorMap tm_vp,
                   const __grid_constant__ CUtensorMap tm_kc, const __grid_constant__ CUtensorMap tm_vc,
                   const __grid_constant__ CUtensorMap tm_kr, const __grid_constant__ CUtensorMap tm_vr,
                   const PrefixParams p)
{
    using SM = PrefixSmem<D>;
    constexpr int NCB = D / 64;
    extern __shared__ __align__(1024) uint8_t pf_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(pf_smem_raw) + 1023) &
                                                ~(uintptr_t)1023);
    uint8_t *sQ = smem + SM::OFF_Q;
    uint8_t *sK = smem + SM::OFF_K;
    uint8_t *sV = smem + SM::OFF_V;
    PrefixToken *sTok = reinterpret_cast<PrefixToken *>(smem + SM::OFF_TOK);
    PrefixItem *sItem = reinterpret_cast<PrefixItem *>(smem + SM::OFF_ITEM);
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + SM::OFF_BAR);
    int *misc = reinterpret_cast<int *>(smem + SM::OFF_MISC);
    volatile int *abort_flag = misc + 1;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(&bar[PB_QF], 1);
        mbar_init(&bar[PB_QE], 2);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar[PB_KF + s], 1);
            mbar_init(&bar[PB_KE + s], 2);     // a commit of each MMA warp, or two of the one that uses it
            mbar_init(&bar[PB_VF + s], 1);
            mbar_init(&bar[PB_VE + s], 2);
            mbar_init(&bar[PB_SF + s], 1);
            mbar_init(&bar[PB_PF + s], 8);     // one arrival a warp
            mbar_init(&bar[PB_TURN + s], 8);
            mbar_init(&bar[PB_OF + s], 1);
            mbar_init(&bar[PB_OE + s], 16);    // both warpgroups (joint), or two from one
        }
        for (int s = 0; s < kPfItemSlots; ++s) {
            mbar_init(&bar[PB_IF + s], 1);
            mbar_init(&bar[PB_IE + s], 19);    // producer, MMA and softmax warps
        }
        mbar_init(&bar[PB_DONE], 2);
        for (int s = 0; s < 8; ++s)
            mbar_init(&bar[PB_MEET + s], 2);
        for (int s = 0; s < 4; ++s)
            mbar_init(&bar[PB_MEET4 + s], 4);
        mbar_fence_init();
        misc[1] = 0;
    }
    if (warp == 17)
        tmem_alloc(reinterpret_cast<uint32_t *>(&misc[0]), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)misc[0];
    pdl_wait();      // launched as a programmatic dependent: the previous kernel's writes
    pdl_trigger();   // are visible from here on; the next kernel may start its launch
    const int tries = wait_tries();
    // every lane waits; the warp goes on only if all of them got through
    auto wait = [&](int b, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait_short(&bar[b], parity, abort_flag, tries)) != 0;
    };
    // the n-th item of this CTA (false: none, or giving up); `release` after its last read
    auto item = [&](uint32_t n, PrefixItem &it) {
        if (!wait(PB_IF + n % kPfItemSlots, (n / kPfItemSlots) & 1))
            return false;
        it = sItem[n % kPfItemSlots];
        return it.last == 0;
    };
    auto release = [&](uint32_t n) {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&bar[PB_IE + n % kPfItemSlots]);
    };

    constexpr uint32_t TM_O = 2 * kPfBN;         // S_A, S_B, then O_A, O_B (128 columns each)
    if (warp >= 16)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPfOtherRegs));
    if (warp == 19) {
        // ================================ items ================================
        uint32_t n = 0;
        bool ok = true;
        auto next = [&](bool pre, int i, int s, int u0, int u1) {
            const uint32_t slot = n % kPfItemSlots;
            if (n >= kPfItemSlots && !wait(PB_IE + slot, (n / kPfItemSlots - 1) & 1))
                return false;
            if (i < 0) {
                if (lane == 0)
                    sItem[slot].last = 1;
            } else {
                prefix_item(p, pre, i, s, u0, u1, lane, sItem[slot], sTok + slot * 256);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bar[PB_IF + slot]);
            ++n;
            return true;
        };
        // pieces of the shared entries: the items of one KV head and piece number
        // lie side by side, so that they read the same tiles at the same time
        for (int q = blockIdx.x; ok && q < p.p_pieces; q += p.ctas) {
            const int u = q % p.p_units, r = q / p.p_units;
            ok = next(true, (r / p.p_ns) * p.p_units + u, r % p.p_ns, 0, 0);
        }
        const int end = p.o_total > 0 ? pf_share(p, blockIdx.x + 1) : 0;
        for (int u = p.o_total > 0 ? pf_share(p, blockIdx.x) : 0; ok && u < end;) {
            const int i = u / p.o_len, u0 = u - i * p.o_len, u1 = min(p.o_len, u0 + (end - u));
            ok = next(false, i, (int)blockIdx.x - pf_cta(p, i * p.o_len), u0, u1);
            u += u1 - u0;
        }
        if (ok)
            next(false, -1, 0, 0, 0);
    } else if (warp == 16) {
        // ================================ producer ================================
        const uint32_t q_bytes = (uint32_t)p.hpt * p.tpt * D * 2;
        uint32_t kc = 0, vc = 0, nq = 0, qn = 0;
        bool ok = true;
        PrefixItem it;
        while (ok && item(nq, it)) {
            release(nq);
            if (lane == 0) {
                ok = nq == 0 || mbar_wait_short(&bar[PB_QE], (nq - 1) & 1, abort_flag, tries);
                if (ok) {
                    mbar_arrive_expect_tx(&bar[PB_QF], (1 + it.val1) * q_bytes);
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        for (int cb = 0; x <= it.val1 && cb < NCB; ++cb)
                            tma_load_4d(sQ + x * SM::Q_BYTES + cb * kPfBM * 128, it.pre ? &tm_qp : &tm_qo,
                                        &bar[PB_QF], cb * 64, it.h0[x], it.tok0[x], it.b);
                    ++qn;
                }
                const int per = it.pair ? 1 : 2;   // key tiles of a step
                for (int i = 0; ok && i < it.nt; i += per) {
                    for (int kv = 0; ok && kv < 2; ++kv) {
                        uint32_t &cnt = kv ? vc : kc;
                        uint8_t *ring = kv ? sV : sK;
                        uint64_t *full = &bar[kv ? PB_VF : PB_KF], *empty = &bar[kv ? PB_VE : PB_KE];
                        for (int j = i; j < min(i + per, it.nt); ++j) {
                            int t = it.t0 + j;
                            const int kind = pf_kind(it, t);
                            const int row0 = (kind == 2 ? it.rlo : 0) + t * kPfBN;
                            const CUtensorMap *map = kv ? (kind == 0 ? &tm_vp : kind == 1 ? &tm_vc : &tm_vr)
                                                        : (kind == 0 ? &tm_kp : kind == 1 ? &tm_kc : &tm_kr);
                            const uint32_t st = cnt % kPfStages;
                            if (cnt >= kPfStages &&
                                !mbar_wait_short(&empty[st], ((cnt / kPfStages) - 1) & 1, abort_flag, tries)) {
                                ok = false;
                                break;
                            }
                            // The MMA warps wait for full stages by parity, and an item's
                            // first tiles may follow tiles that only the other warp waited
                            // for: K of tile n goes out once V of tile n - 2 has landed (K
                            // has, since Q was reloaded), so that a warp that has seen K of
                            // tile n is at most one phase of V behind.
                            if (!kv && j < 2 && cnt >= kPfStages &&
                                !mbar_wait_short(&bar[PB_VF + st], ((cnt / kPfStages) - 1) & 1, abort_flag, tries)) {
                                ok = false;
                                break;
                            }
                            mbar_arrive_expect_tx(&full[st], SM::KV_BYTES);
                            for (int cb = 0; cb < NCB; ++cb)
                                tma_load_4d(ring + st * SM::KV_BYTES + cb * kPfBN * 128, map, &full[st], cb * 64,
                                            it.kvh, row0, kind == 0 ? 0 : it.b);
                            ++cnt;
                        }
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            if (ok)
                ++nq;
        }
        if (lane == 0) {
            // unwinding: wait for the last copies issued into every slot
            if (qn > 0)
                drain_wait(&bar[PB_QF], (qn - 1) & 1);
            for (uint32_t c = (kc > kPfStages ? kc - kPfStages : 0); c < kc; ++c)
                drain_wait(&bar[PB_KF + c % kPfStages], (c / kPfStages) & 1);
            for (uint32_t c = (vc > kPfStages ? vc - kPfStages : 0); c < vc; ++c)
                drain_wait(&bar[PB_VF + c % kPfStages], (c / kPfStages) & 1);
        }
    } else if (warp >= 16) {
        // ================================ MMA issue ================================
        const int x = warp - 17;
        const uint32_t idesc_qk = idesc_bf16(kPfBM, kPfBN, false, false);
        const uint32_t idesc_pv = idesc_bf16(kPfBM, D, false, true);
        const uint64_t dK = sw128_desc(smem_u32(sK), 16, 1024);                 // K-major
        const uint64_t dV = sw128_desc(smem_u32(sV), kPfBN * 128, 1024);         // MN-major
        const uint32_t tS = tmem + x * kPfBN, tO = tmem + TM_O + x * 128;
        const bool leader = elect_one();
        uint32_t base = 0;            // key tiles of the items before this one
        uint32_t pcnt = 0, ocnt = 0, nq = 0;
        bool ok = true;
        PrefixItem it;
        while (item(nq, it)) {
            release(nq);
            // this warp's key tiles: all of a pair's, or every second one
            const int step = it.pair ? 1 : 2, first = it.pair ? (x <= it.val1 ? 0 : it.nt) : x;
            const uint64_t dq = sw128_desc(smem_u32(sQ) + (it.pair ? x : 0) * SM::Q_BYTES, 16, 1024);
            if (!(ok = wait(PB_QF, nq & 1)))
                break;
            // O is free once the epilogue of this warp's previous item with keys has
            // read it (items without keys for it have no epilogue to wait for)
            bool o_free = ocnt == 0;
            const bool alone = !it.pair || !it.val1;   // no other warp reads this one's tiles
            for (int t = first; t < it.nt + step; t += step) {
                if (t > first) {
                    const uint32_t n = base + t - step, vs = n % kPfStages;
                    if (!(ok = wait(PB_VF + vs, (n / kPfStages) & 1)))
                        break;
                    int kt = it.t0 + t - step;
                    const int kind = pf_kind(it, kt);
                    const int seen = (kind == 0 ? it.npre : kind == 1 ? it.nent : it.nraw) - kt * kPfBN;
                    if (seen < kPfBN) {
                        // rows that no query of the item sees take no part, whatever they hold
                        for (int cb = 0; cb < NCB; ++cb)
#pragma unroll 1
                            for (int c = seen * 8 + lane; c < kPfBN * 8; c += 32)
                                *reinterpret_cast<uint4 *>(sV + vs * SM::KV_BYTES + cb * kPfBN * 128 + c * 16) =
                                    make_uint4(0, 0, 0, 0);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (!o_free && !(ok = wait(PB_OE + x, (ocnt - 1) & 1)))
                        break;
                    o_free = true;
                    if (!(ok = wait(PB_PF + x, pcnt & 1)))
                        break;
                    ++pcnt;
                    tc_fence_after();
                    if (leader) {
                        // (addresses are the low bits of a descriptor, in 16-byte units)
                        const uint64_t dv = dV + (vs * SM::KV_BYTES >> 4);
#pragma unroll
                        for (int kk = 0; kk < kPfBN / 16; ++kk) {
                            // P of keys 64 .. 127 starts at column 64
                            mma_bf16_ts(tO, tS + (kk >> 2) * 64 + (kk & 3) * 8, dv + kk * 128, idesc_pv,
                                        (t == first + step && kk == 0) ? 0u : 1u);
                        }
                        mma_commit(&bar[PB_VE + vs]);
                        if (alone)
                            mma_commit(&bar[PB_VE + vs]);
                    }
                }
                if (t < it.nt) {
                    const uint32_t n = base + t, ks = n % kPfStages;
                    if (!(ok = wait(PB_KF + ks, (n / kPfStages) & 1)))
                        break;
                    tc_fence_after();
                    if (leader) {
                        const uint64_t dk = dK + (ks * SM::KV_BYTES >> 4);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            mma_bf16_ss(tS, dq + (kk >> 2) * (kPfBM * 8) + (kk & 3) * 2,
                                        dk + (kk >> 2) * (kPfBN * 8) + (kk & 3) * 2, idesc_qk, kk > 0 ? 1u : 0u);
                        }
                        mma_commit(&bar[PB_SF + x]);
                        mma_commit(&bar[PB_KE + ks]);
                        if (alone)
                            mma_commit(&bar[PB_KE + ks]);
                        if (t + step >= it.nt)
                            mma_commit(&bar[PB_QE]);
                    }
                }
            }
            if (!ok)
                break;
            if (leader)
                mma_commit(&bar[first < it.nt ? PB_OF + x : PB_QE]);
            ocnt += first < it.nt;
            base += it.nt;
            ++nq;
        }
        if (leader)
            mma_commit(&bar[PB_DONE]);
        __syncwarp();
        drain_wait(&bar[PB_DONE], 0);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPfSoftmaxRegs));
        // ========================== softmax + epilogue ==========================
        const int x = warp >> 3;            // 0: A, 1: B
        const int half = (warp >> 2) & 1;   // keys 64 half .. of a tile, channels D / 2 half .. of O
        const int quad = warp & 3;
        const int row = quad * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t tS = tl + x * kPfBN + half * 64;
        const uint32_t tO = tl + TM_O + x * 128 + half * (D / 2);
        const uint32_t tOA = tl + TM_O;         // O of A; O of B is 128 columns on
        float *mine = reinterpret_cast<float *>(smem + SM::OFF_MAX) + threadIdx.x;
        const float *other = reinterpret_cast<float *>(smem + SM::OFF_MAX) + (threadIdx.x ^ 128);
        // the two warps of a row quad meet: bounded, like every wait (a named barrier
        // would keep one of them for ever if the other gave up)
        uint32_t met = 0, met4 = 0;
        auto meet = [&]() {
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bar[PB_MEET + x * 4 + quad]);
            return wait(PB_MEET + x * 4 + quad, met++ & 1);
        };
        uint8_t *stage = smem + SM::OFF_ST + warp * SM::STAGE_BYTES;
        const int rtok = row / p.hpt, rhead = row % p.hpt;
        const uint64_t sc2 = f2(p.scale_log2, p.scale_log2);
        uint32_t scnt = 0, nq = 0;
        uint32_t o_par = 0;                 // bit y: parity of the next phase of stream y's O
        uint32_t turn = 0;                  // tiles taken in turns so far
        bool ok = true;
        PrefixItem it;
        while (ok && item(nq, it)) {
            const int step = it.pair ? 1 : 2, first = it.pair ? (x <= it.val1 ? 0 : it.nt) : x;
            const int xt = it.pair ? x : 0;
            const int tok = (xt ? it.tok0[1] : it.tok0[0]) + rtok;
            const int h = (xt ? it.h0[1] : it.h0[0]) + rhead;
            const bool valid_row = rtok < p.tpt && tok < it.ntok && h < (it.kvh + 1) * p.g && xt <= it.val1;
            PrefixToken tk = {0, 0, -1};   // nothing visible
            if (valid_row)
                tk = sTok[(nq % kPfItemSlots) * 256 + xt * 128 + rtok];
            release(nq);
            const bool warp_rows = __any_sync(0xffffffffu, valid_row);
            const bool turns = it.pair && it.val1;
            const int flat = (it.pre ? 0 : it.b * p.Lq) + tok;
            float m_ref = -INFINITY, l_sum = 0.f;
            for (int t = first; t < it.nt; t += step) {
                if (!(ok = wait(PB_SF + x, scnt & 1)))
                    break;
                ++scnt;
                tc_fence_after();
                if (warp_rows) {
                    // keys c_lo .. c_lo + c_n of this half of the tile are visible to this row
                    int c_lo = 0, c_hi, kt = it.t0 + t;
                    const int kind = pf_kind(it, kt);
                    const int r0 = kt * kPfBN + half * 64;
                    if (kind == 2) {
                        c_lo = max(0, tk.wlo - it.rlo - r0);
                        c_hi = min(tk.whi - it.rlo - r0, 63);
                    } else {
                        c_hi = min((kind == 0 ? min(tk.nv, p.Np) : tk.nv - p.Np) - 1 - r0, 63);
                    }
                    // (rows of no query go along with the others: nothing of theirs is kept)
                    const bool full = __all_sync(0xffffffffu, !valid_row || (c_lo == 0 && c_hi == 63));
                    if (c_hi < c_lo) {
                        c_lo = 1 << 20;
                        c_hi = c_lo;
                    }
                    const unsigned c_n = (unsigned)(c_hi - c_lo);
                    float v[64];
                    tmem_ld32(tS, *reinterpret_cast<float(*)[32]>(&v[0]));
                    tmem_ld32(tS + 32, *reinterpret_cast<float(*)[32]>(&v[32]));
                    tmem_ld_wait();
                    if (!full) {
#pragma unroll
                        for (int q = 0; q < 64; ++q)
                            v[q] = (unsigned)(q - c_lo) <= c_n ? v[q] : -INFINITY;
                    }
                    // row maximum
                    float tmax;
                    {
                        float mk[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float a = fmax3f(v[16 * k], v[16 * k + 1], v[16 * k + 2]);
#pragma unroll
                            for (int q = 3; q < 15; q += 2)
                                a = fmax3f(a, v[16 * k + q], v[16 * k + q + 1]);
                            mk[k] = fmaxf(a, v[16 * k + 15]);
                        }
                        tmax = fmaxf(fmaxf(mk[0], mk[1]), fmaxf(mk[2], mk[3]));
                    }
                    *mine = tmax;
                    if (!(ok = meet()))
                        break;
                    tmax = fmaxf(tmax, *other);
                    tmax *= p.scale_log2;  // the scale is positive
                    // the reference maximum moves (and O is rescaled) only when a
                    // tile raises it by more than 2^8
                    float alpha = 1.f;
                    if (tmax > m_ref + 8.f) {
                        alpha = (m_ref == -INFINITY) ? 0.f : ex2_approx(m_ref - tmax);
                        m_ref = tmax;
                        l_sum *= alpha;
                    }
                    if (t > first && __any_sync(0xffffffffu, alpha != 1.f)) {
                        // O holds every earlier PV (S_full covers all MMAs issued before this QK)
#pragma unroll 1
                        for (int c = 0; c < D / 2; c += 8) {
                            float ov[8];
                            tmem_ld8(tO + c, ov);
                            tmem_ld_wait();
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                ov[q] *= alpha;
                            tmem_st8(tO + c, ov);
                        }
                    }
                    // Turns: B's exponentials of a tile follow A's, and A's next ones follow
                    // B's, so that one query tile's run under the other's MMAs.  (Left
                    // alone the two fall into step: both exponentiate, then both wait.)
                    // Turns have barriers of their own and are counted over all items (those
                    // between may take none): A's turn n + 1 ends only once every A warp with
                    // rows has seen the end of B's turn n, and B's turn n only once every B
                    // warp with rows has seen the end of A's, so that neither barrier gets
                    // two phases ahead of a warp that waits by parity.
                    if (turns && (x || turn > 0) && !(ok = wait(PB_TURN + (x ^ 1), (x ? turn : turn - 1) & 1)))
                        break;
                    // P = exp2(s * scale - mu), rounded to bf16 (the MMA operand; its
                    // relative error 2^-8 a term averages out below the output's own
                    // rounding) over the first half of this thread's columns of S; the
                    // row sum is of the fp32 values.
                    // Some of the exponentials are polynomials: the unit's 16 a clock
                    // are what a pair's softmax would wait for.
                    const float mu = (m_ref == -INFINITY) ? 0.f : m_ref;
                    const uint64_t nmu2 = f2(-mu, -mu);
                    uint64_t lacc[2] = {0ull, 0ull};
#pragma unroll
                    for (int c = 0; c < 64; c += 32) {
                        uint32_t pk[16];
#pragma unroll
                        for (int q = c; q < c + 32; q += 2) {
                            float x0, x1;
                            f2_split(fma_f2(f2(v[q], v[q + 1]), sc2, nmu2), x0, x1);
                            if ((q >> 1) % 8 < kPfPolyPairs) {
                                float e0, e1;
                                exp2_poly2(x0, x1, e0, e1);
                                x0 = e0;
                                x1 = e1;
                            } else {
                                x0 = ex2_approx(x0);
                                x1 = ex2_approx(x1);
                            }
                            lacc[(q >> 1) & 1] = add_f2(lacc[(q >> 1) & 1], f2(x0, x1));
                            pk[(q - c) >> 1] = pack_bf16x2(x0, x1);
                        }
                        tmem_st16(tS + (c >> 1), pk);
                    }
                    float a0, a1;
                    f2_split(add_f2(lacc[0], lacc[1]), a0, a1);
                    l_sum += a0 + a1;
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (turns)                 // before P: the next tile's S follows it
                        mbar_arrive(&bar[PB_TURN + x]);
                    mbar_arrive(&bar[PB_PF + x]);
                }
                turn += turns;
            }
            if (!ok)
                break;
            // Epilogue: the O's that this warp frees, its own or (joint) both streams'.  A
            // warp without rows waits too: freeing takes no look at O, and one that ran
            // items ahead would stand in for a warp that still reads this item's.  So an O's
            // next phase needs this item freed by all sixteen warps.
            const bool joint = p.direct && !it.pair;
            const int o_end = joint ? min(it.nt, 2) : first < it.nt ? x + 1 : x;
#pragma unroll 1
            for (int y = joint ? 0 : x; ok && y < o_end; ++y) {
                ok = wait(PB_OF + y, (o_par >> y) & 1);
                o_par ^= 1u << y;
            }
            if (!ok)
                break;
            tc_fence_after();
            if (!p.direct) {
                // a part of the row: this warpgroup's O as it is, its maximum and sum
                if (warp_rows) {
                    *mine = l_sum;
                    if (!(ok = meet()))
                        break;
                    l_sum += *other;
                    if (!(ok = meet()))      // before the next item's first maximum
                        break;
                }
                const size_t at = (size_t)(it.part + (it.pair ? 0 : x)) * p.rows + (size_t)flat * p.Hq + h;
                if (valid_row && half == 0)
                    p.part_ml[at] = make_float2(m_ref, l_sum);
                const unsigned stored = __ballot_sync(0xffffffffu, valid_row && l_sum != 0.f);
                if (stored) {
                    float *orow = p.part_o + at * D + half * (D / 2);
                    if (__popc(stored) <= 8) {
                        // few rows: each lane writes its own
#pragma unroll 1
                        for (int c = 0; c < D / 2; c += 32) {
                            float ov[32];
                            tmem_ld32(tO + c, ov);
                            tmem_ld_wait();
                            if ((stored >> lane) & 1) {
#pragma unroll
                                for (int q = 0; q < 32; q += 4)
                                    *reinterpret_cast<float4 *>(orow + c + q) =
                                        make_float4(ov[q], ov[q + 1], ov[q + 2], ov[q + 3]);
                            }
                        }
                    } else {
                        // eight channels of the warp's rows at a time, through shared memory,
                        // so that a store instruction writes whole 32-byte sectors
                        const int r = lane >> 1, q = lane & 1;
                        float *dst[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            dst[k] = reinterpret_cast<float *>(__shfl_sync(
                                         0xffffffffu, reinterpret_cast<unsigned long long>(orow), r + 16 * k)) + 4 * q;
                        const uint8_t *src = stage + r * 32 + ((q ^ ((r >> 2) & 1)) << 4);
                        uint8_t *put = stage + lane * 32 + (((lane >> 2) & 1) << 4);
#pragma unroll 1
                        for (int c = 0; c < D / 2; c += 32) {
                            float ov[32];
                            tmem_ld32(tO + c, ov);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; e += 8) {
                                *reinterpret_cast<float4 *>(put) = make_float4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
                                *reinterpret_cast<float4 *>(stage + ((put - stage) ^ 16)) =
                                    make_float4(ov[e + 4], ov[e + 5], ov[e + 6], ov[e + 7]);
                                __syncwarp();
#pragma unroll
                                for (int k = 0; k < 2; ++k)
                                    if ((stored >> (r + 16 * k)) & 1)
                                        *reinterpret_cast<float4 *>(dst[k] + c + e) =
                                            *reinterpret_cast<const float4 *>(src + k * 512);
                                __syncwarp();
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && first < it.nt) {
                    mbar_arrive(&bar[PB_OE + x]);
                    mbar_arrive(&bar[PB_OE + x]);
                }
                ++nq;
                continue;
            }
            // The row's sum over both halves, and where an alternating item is joined the two
            // streams' maxima and sums: weights ws of this warpgroup's (pair) or of A's
            // and B's O, maximum m_ref and sum l_sum of the result.
            float ws[2] = {1.f, 0.f};
            if (warp_rows) {
                float2 *ml = reinterpret_cast<float2 *>(stage) + lane;
                const float2 *of = reinterpret_cast<const float2 *>(stage + ((warp ^ 4) - warp) * SM::STAGE_BYTES) + lane;
                const int hop = ((warp ^ 8) - warp) * SM::STAGE_BYTES / (int)sizeof(float2);
                *ml = make_float2(m_ref, l_sum);
                tc_fence_before();
                if (!joint) {
                    if (!(ok = meet()))
                        break;
                    l_sum += of->y;
                    if (!(ok = meet()))        // before the stage is written again
                        break;
                } else {
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&bar[PB_MEET4 + quad]);
                    if (!(ok = wait(PB_MEET4 + quad, met4++ & 1)))
                        break;
                    tc_fence_after();
                    const float l0 = l_sum + of->y, l1 = ml[hop].y + of[hop].y, m1 = ml[hop].x;
                    const float M = fmaxf(m_ref, m1);
                    const float w0 = l0 != 0.f ? exp2f(m_ref - M) : 0.f, w1 = l1 != 0.f ? exp2f(m1 - M) : 0.f;
                    ws[0] = x ? w1 : w0;
                    ws[1] = x ? w0 : w1;
                    l_sum = (l0 != 0.f ? l0 * w0 : 0.f) + (l1 != 0.f ? l1 * w1 : 0.f);
                    m_ref = M;
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&bar[PB_MEET4 + quad]);
                    if (!(ok = wait(PB_MEET4 + quad, met4++ & 1)))
                        break;
                }
            }
            const long long at = (long long)flat * p.Hq + h;
            const float inv = l_sum != 0.f ? 1.f / l_sum : 0.f;
            ws[0] *= inv;
            ws[1] *= inv;
            if (valid_row && half == 0 && (!joint || x == 0) && p.lse)
                p.lse[((long long)it.b * p.Hq + h) * p.Lq + flat - it.b * p.Lq] =
                    l_sum != 0.f ? (m_ref + log2f(l_sum)) * 0.6931471805599453f : -INFINITY;
            const unsigned stored = __ballot_sync(0xffffffffu, valid_row);    // (an empty row is 0)
            if (stored) {
                // this thread's channels: half of the row, or a quarter where A and B share it
                const int ch0 = joint ? (half * 2 + x) * (D / 4) : half * (D / 2);
                const int nch = joint ? D / 4 : D / 2;
                // O was written: in pairs with any tile, else by the streams that had one
                const bool o0 = joint ? it.nt > 0 : first < it.nt, o1 = joint && it.nt > 1;
                const uint32_t src = joint ? tOA : tl + TM_O + x * 128;
                uint8_t *orow = reinterpret_cast<uint8_t *>(p.o + at * D + ch0);
                const bool few = __popc(stored) <= 8;
                // through shared memory, 32 bytes of a row at a time, so that a store
                // instruction writes whole sectors of sixteen rows
                const int r = lane >> 1, q = lane & 1;
                uint8_t *dst[2];
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    dst[k] = reinterpret_cast<uint8_t *>(__shfl_sync(
                                 0xffffffffu, reinterpret_cast<unsigned long long>(orow), r + 16 * k)) + 16 * q;
                const uint8_t *get = stage + r * 32 + ((q ^ ((r >> 2) & 1)) << 4);
                uint8_t *put = stage + lane * 32, *put1;
                put1 = put + ((((lane >> 2) & 1) ^ 1) << 4);
                put += ((lane >> 2) & 1) << 4;
                auto put32 = [&](int off, const uint4 &lo, const uint4 &hi) {
                    if (few) {                 // each lane writes its own row
                        if ((stored >> lane) & 1) {
                            *reinterpret_cast<uint4 *>(orow + off) = lo;
                            *reinterpret_cast<uint4 *>(orow + off + 16) = hi;
                        }
                        return;
                    }
                    *reinterpret_cast<uint4 *>(put) = lo;
                    *reinterpret_cast<uint4 *>(put1) = hi;
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if ((stored >> (r + 16 * k)) & 1)
                            *reinterpret_cast<uint4 *>(dst[k] + off) = *reinterpret_cast<const uint4 *>(get + k * 512);
                    __syncwarp();
                };
#pragma unroll 1
                for (int c = 0; c < nch; c += 16) {
                    float ov[16];
                    if (o0) {
                        tmem_ld16(src + ch0 + c, ov);
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            ov[e] = 0.f;
                    }
                    if (o1) {
                        float o2[16];
                        tmem_ld16(src + 128 + ch0 + c, o2);
                        tmem_ld_wait();
                        // (a stream without keys for this row left nothing that counts)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            ov[e] = (ws[0] != 0.f ? ov[e] * ws[0] : 0.f) + (ws[1] != 0.f ? o2[e] * ws[1] : 0.f);
                    } else {
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            ov[e] = ws[0] != 0.f ? ov[e] * ws[0] : 0.f;
                    }
                    uint32_t pk[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        pk[e] = pack_bf16x2(ov[2 * e], ov[2 * e + 1]);
                    put32(c * 2, make_uint4(pk[0], pk[1], pk[2], pk[3]), make_uint4(pk[4], pk[5], pk[6], pk[7]));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (!joint) {
                    if (first < it.nt) {
                        mbar_arrive(&bar[PB_OE + x]);
                        mbar_arrive(&bar[PB_OE + x]);
                    }
                } else {
                    if (it.nt > 0)
                        mbar_arrive(&bar[PB_OE + 0]);
                    if (it.nt > 1)
                        mbar_arrive(&bar[PB_OE + 1]);
                }
            }
            ++nq;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc((uint32_t)misc[0], 512);
    }
}

// Joins the parts of each row: D / 4 lanes hold four channels each, U parts in
// flight; with WAYS > 1 (few rows, many parts) as many lane groups take every
// WAYS-th part of a row and meet in shared memory.  Bound: latency (on one GPU,
// 9 parts of 4096 rows: 64.1 us with the attention kernel at U = 4, 62.7 at 8;
// 4 parts: 35.6 against 36.9; 13 parts of 1300 rows: 31.8 one way, 28.0 eight).
template <int D, int WAYS, int U>
__global__ void __launch_bounds__(256) prefix_combine_kernel(const PrefixParams p)
{
    pdl_wait();
    pdl_trigger();
    constexpr int LPR = D / 4;
    constexpr int GROUPS = 256 / LPR;           // lane groups of the block
    const int grp = threadIdx.x / LPR, way = grp % WAYS;
    const long long row = (long long)blockIdx.x * (GROUPS / WAYS) + grp / WAYS;
    const int c = (threadIdx.x % LPR) * 4;
    const bool in = row < p.rows;
    // this row's parts: [0, np) and [p_parts, p_parts + no)
    int np = 0, no = 0;
    long long b = 0, t = 0;
    int h = 0;
    if (in) {
        const unsigned bt = (unsigned)row / (unsigned)p.Hq;     // rows fit 31 bits
        h = (int)((unsigned)row - bt * (unsigned)p.Hq);
        b = bt / (unsigned)p.Lq;
        t = bt - (unsigned)b * (unsigned)p.Lq;
        const int kvh = h / p.g, ht = (h - kvh * p.g) / p.hpt;
        np = p.p_parts;
        if (p.o_total > 0) {
            const int tile = ((int)t / p.tpt) * p.nht + ht;
            const int i = ((int)b * p.Hkv + kvh) * p.o_units + (p.o_pair ? tile >> 1 : tile);
            no = pf_cta(p, (i + 1) * p.o_len - 1) - pf_cta(p, i * p.o_len) + 1;
            no *= p.o_pair ? 1 : 2;
        }
    }
    float M = -INFINITY, L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = way; i0 < np + no; i0 += U * WAYS) {
        float2 ml[U];
        float4 v[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = i0 + k * WAYS;
            ml[k] = make_float2(-INFINITY, 0.f);
            if (i < np + no) {
                const size_t at = (size_t)(i < np ? i : p.p_parts + i - np) * p.rows + row;
                ml[k] = p.part_ml[at];
                // (a part without keys has no row: whatever is there is not used)
                v[k] = *reinterpret_cast<const float4 *>(p.part_o + at * D + c);
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (ml[k].y == 0.f)
                continue;
            const float m = fmaxf(M, ml[k].x);
            const float w0 = exp2f(M - m), w1 = exp2f(ml[k].x - m);
            M = m;
            L = L * w0 + ml[k].y * w1;
            a.x = a.x * w0 + v[k].x * w1;
            a.y = a.y * w0 + v[k].y * w1;
            a.z = a.z * w0 + v[k].z * w1;
            a.w = a.w * w0 + v[k].w * w1;
        }
    }
    if (WAYS > 1) {
        __shared__ float4 sa[256];
        __shared__ float2 sm[256];
        sa[threadIdx.x] = a;
        sm[threadIdx.x] = make_float2(M, L);
        __syncthreads();
        if (way != 0)
            return;
        for (int k = 1; k < WAYS; ++k) {
            const float2 o = sm[threadIdx.x + k * LPR];
            const float4 v = sa[threadIdx.x + k * LPR];
            if (o.y == 0.f)
                continue;
            const float m = fmaxf(M, o.x);
            const float w0 = exp2f(M - m), w1 = exp2f(o.x - m);
            M = m;
            L = L * w0 + o.y * w1;
            a.x = a.x * w0 + v.x * w1;
            a.y = a.y * w0 + v.y * w1;
            a.z = a.z * w0 + v.z * w1;
            a.w = a.w * w0 + v.w * w1;
        }
    }
    if (!in)
        return;
    const float inv = L != 0.f ? 1.f / L : 0.f;
    uint2 v;
    v.x = pack_bf16x2(a.x * inv, a.y * inv);
    v.y = pack_bf16x2(a.z * inv, a.w * inv);
    *reinterpret_cast<uint2 *>(p.o + row * D + c) = v;
    if (c == 0 && p.lse)
        p.lse[(b * p.Hq + h) * p.Lq + t] = L != 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
}

// How the work is split: fills the tiling and the split of p, by the costs below
// (1/8 us, measured on one B200 at d = 128).  False when the own-key stream does
// not fit 32-bit arithmetic.
constexpr int kPfPairCost = 17, kPfAltCost = 8;           // a key tile of each mode
constexpr int kPfPairItemCost = 40, kPfAltItemCost = 20;  // an item beside its tiles (256 or a few rows to store)
constexpr int kPfJoinCost = 24;                                     // the second kernel

static bool prefix_plan(PrefixParams &p, int d)
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
    p.ctas = kPfPlanSMs;
    // key tiles of the two streams (raw rows: those of consecutive positions)
    const long long span = p.Lq < 2 * p.tpt ? p.Lq : 2 * p.tpt;
    long long raw = p.W > 0 ? (long long)p.W + span - 1 : 0;
    if (raw > p.Lkv)
        raw = p.Lkv;
    const long long Tp = up(p.Np, kPfBN), To = up(p.Nc, kPfBN) + up(raw, kPfBN);
    const bool own = p.Nc > 0 || p.W > 0;
    const long long items = (long long)p.o_units * p.Hkv * p.B;       // of own keys
    const long long wp = p.p_pair ? kPfPairCost : kPfAltCost, wo = p.o_pair ? kPfPairCost : kPfAltCost;
    const long long over_p = p.p_pair ? kPfPairItemCost : kPfAltItemCost;
    const long long over = p.o_pair ? kPfPairItemCost : kPfAltItemCost, least = over + wo;   // a share worth its overhead
    p.o_over = (int)over;
    // the traffic of one part of every row, written and read once at about 4 TB/s
    const double part = (double)p.rows * (d * 4 + 8) * 2 / 4e6 * 8;
    double best = -1;
    long long a = 0, b = least, rem = 0, ns = 0, olen = 1, total = 0;
    bool merged = false, direct = false;
    auto take = [&](double cost, bool mg, bool di, long long ns_, long long rem_, long long a_, long long b_,
                    long long olen_, long long total_) {
        if (best >= 0 && cost >= best)
            return;
        best = cost;
        merged = mg;
        direct = di;
        ns = ns_;
        rem = rem_;
        a = a_;
        b = b_;
        olen = olen_;
        total = total_;
    };
    // one stream a sequence, through the shared entries as well: whole items, or cut
    if (Tp + To > 0) {
        const long long len = (Tp + To) * wo + over, all = items * len;
        const long long each = up(items, p.ctas);
        if (all < (1LL << 30)) {
            take((double)each * len, true, true, 0, 0, each * len, each * len, len, all);
            long long share = up(all, p.ctas);
            if (share < least)
                share = least;
            if (share < len)
                take((double)(share + over) + part * (double)((len / share + 1) * (p.o_pair ? 1 : 2)) + kPfJoinCost, true, false, 0, 0, share,
                     share, len, all);
        }
    }
    // Shared entries apart, as ns pieces of each of their items; own keys fill up the
    // CTAs with fewer pieces, or the others evenly: shares a (CTAs with one piece
    // more) and b; a share that cuts an item pays `over` again.
    if (Tp > 0) {
        const long long len = To * wo + over, all = own ? items * len : 0, Ip = (long long)p.p_units * p.Hkv;
        for (long long tiles = Tp, last = 0; tiles >= 1 && all < (1LL << 30); tiles -= 1 + tiles / 8) {
            const long long n = up(Tp, tiles);
            if (n > p.ctas)
                break;
            if (n == last)
                continue;
            last = n;
            const long long piece = up(Tp, n) * wp + over_p, pieces = Ip * n;
            const long long cnt = pieces / p.ctas, r = pieces % p.ctas;
            const long long quota = up(pieces * piece + all, p.ctas);
            for (int even = 0; even < (all ? 2 : 1); ++even) {
                long long sa = quota - (cnt + 1) * piece, sb = quota - cnt * piece;
                if (r == 0)
                    sa = sb;
                if (even || sa < least) {
                    sa = 0;
                    sb = up(all, p.ctas - r);
                }
                if (sb < least)
                    sb = least;
                if (sb >= 8 * len) {     // many items a CTA: whole ones, so that no row has a second part
                    sa = up(sa, len) * len;
                    sb = up(sb, len) * len;
                }
                const bool cut = all && sb % len != 0;
                long long longest = cnt * piece + (all ? sb : 0) + (cut ? over : 0);
                const long long other = r ? (cnt + 1) * piece + sa + (sa && cut ? over : 0) : 0;
                if (other > longest)
                    longest = other;
                take((double)longest + part * (double)(n * (p.p_pair ? 1 : 2) + (all ? (1 + cut) * (p.o_pair ? 1 : 2) : 0)) + kPfJoinCost, false, false, n, r, sa,
                     sb, len, all);
            }
        }
    }
    if (Tp + To > 0 && best < 0)
        return false;
    p.merged = merged;
    p.direct = direct;
    p.p_ns = (int)ns;
    p.p_parts = (int)ns * (p.p_pair ? 1 : 2);
    p.p_pieces = (int)(ns * p.p_units * p.Hkv);
    p.o_len = (int)olen;
    p.o_rem = (int)rem;
    p.o_a = (int)a;
    p.o_b = (int)b;
    p.o_total = (int)total;
    // most CTAs that an own item can be spread over
    long long o_parts = 0;
    if (total > 0 && !direct) {
        const long long small = a > 0 && a < b ? a : b;
        o_parts = b % olen == 0 && a % olen == 0 ? 1 : (olen - 2) / small + 2;
        if (total <= small)
            o_parts = 1;
        if (o_parts > p.ctas)
            o_parts = p.ctas;
        o_parts *= p.o_pair ? 1 : 2;
    }
    p.n_parts = p.p_parts + (int)o_parts;
    // CTAs with something to do
    p.ctas_used = p.p_pieces < p.ctas ? p.p_pieces : p.ctas;
    if (total > 0 && pf_cta(p, p.o_total - 1) + 1 > p.ctas_used)
        p.ctas_used = pf_cta(p, p.o_total - 1) + 1;
    return true;
}

static size_t prefix_ml_bytes(const PrefixParams &p)
{
    return ((size_t)p.n_parts * p.rows * sizeof(float2) + 255) & ~(size_t)255;
}

static std::atomic<unsigned long long> g_prefix_ready[2];     // devices, by head dim

static size_t prefix_workspace(const PrefixParams &p, int d)
{
    return prefix_ml_bytes(p) + (((size_t)p.n_parts * p.rows * d * sizeof(float) + 255) & ~(size_t)255);
}

// The checks and settings of a kernel that hold for the life of the process,
// made once per device (a function attribute call costs about a microsecond).
static bool prefix_set_up(int device, int d)
{
    return device >= 0 && device < 64 && ((g_prefix_ready[d == 128].load(std::memory_order_acquire) >> device) & 1);
}

template <int D>
static cudaError_t launch_prefix_t(PrefixParams &p, const void *q, const void *kp, const void *vp,
                                   const void *kc, const void *vc, const void *kr, const void *vr, void *ws,
                                   cudaStream_t stream)
{
    using SM = PrefixSmem<D>;
    p.part_ml = static_cast<float2 *>(ws);
    p.part_o = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + prefix_ml_bytes(p));
    if (p.ctas_used > 0) {
        // absent tensors: a map that no copy uses
        CUtensorMap mqp, mqo, mkp, mvp, mkc, mvc, mkr, mvr;
        bool ok = make_map(&mqp, q, D, p.Hq, p.B * p.Lq, 1, p.hpt, p.tpt);
        if (p.Np > 0) {
            ok &= make_map(&mkp, kp, D, p.Hkv, p.Np, 1, 1, kPfBN);
            ok &= make_map(&mvp, vp, D, p.Hkv, p.Np, 1, 1, kPfBN);
        } else {
            mkp = mvp = mqp;
        }
        if (p.o_total > 0)
            ok &= make_map(&mqo, q, D, p.Hq, p.Lq, p.B, p.hpt, p.tpt);
        else
            mqo = mqp;
        if (p.Nc > 0) {
            ok &= make_map(&mkc, kc, D, p.Hkv, p.Nc, p.B, 1, kPfBN);
            ok &= make_map(&mvc, vc, D, p.Hkv, p.Nc, p.B, 1, kPfBN);
        } else {
            mkc = mvc = mqp;
        }
        if (p.W > 0) {
            ok &= make_map(&mkr, kr, D, p.Hkv, p.Lkv, p.B, 1, kPfBN);
            ok &= make_map(&mvr, vr, D, p.Hkv, p.Lkv, p.B, 1, kPfBN);
        } else {
            mkr = mvr = mqp;
        }
        if (!ok)
            return cudaErrorInvalidValue;
        // one CTA per SM: it takes all of the tensor memory
        const size_t smem = 1024 + SM::BYTES < 120 * 1024 ? 120 * 1024 : 1024 + SM::BYTES;
        auto kern = prefix_attn_kernel<D>;
        int dev = -1;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess)
            return e;
        if (!prefix_set_up(dev, D)) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess)
                return e;
            e = check_reg_split(kern, kPfThreads, kPfSoftmaxThreads, kPfSoftmaxRegs, kPfOtherRegs);
            if (e != cudaSuccess)
                return e;
            if (dev < 64)
                g_prefix_ready[D == 128].fetch_or(1ull << dev, std::memory_order_release);
        }
        e = launch_pdl(kern, dim3((unsigned)p.ctas_used), dim3(kPfThreads), smem, stream, mqp, mqo, mkp, mvp, mkc,
                       mvc, mkr, mvr, p);
        if (e != cudaSuccess)
            return e;
    }
    if (p.direct)
        return cudaSuccess;
    // many parts, or few rows to fill the GPU with: eight lane groups share a row
    constexpr int GROUPS = 256 / (D / 4);
    const bool share = p.n_parts >= 64 || (p.n_parts >= 8 && p.rows <= 2048);
    const dim3 grid((unsigned)((p.rows * (share ? 8 : 1) + GROUPS - 1) / GROUPS));
    auto join = share ? prefix_combine_kernel<D, 8, 4>
                      : p.n_parts > 6 ? prefix_combine_kernel<D, 1, 8> : prefix_combine_kernel<D, 1, 4>;
    return launch_pdl(join, grid, dim3(256), 0, stream, p);
}

static cudaError_t launch_prefix_attn(PrefixParams &p, int d, const void *q, const void *kp, const void *vp,
                                      const void *kc, const void *vc, const void *kr, const void *vr, void *ws,
                                      cudaStream_t stream)
{
    return d == 128 ? launch_prefix_t<128>(p, q, kp, vp, kc, vc, kr, vr, ws, stream)
                    : launch_prefix_t<64>(p, q, kp, vp, kc, vc, kr, vr, ws, stream);
}

}  // namespace hyb
