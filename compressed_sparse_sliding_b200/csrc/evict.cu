// evict.cu -- eviction from bounded caches: which entries a sequence keeps by
// their accumulated attention weight, and the caches rewritten with them.
//
// evict_select_kernel.  Exact selection of the largest weights: the weights'
// order-preserving integer images are searched for the threshold by narrowing an
// interval over at most three 2048-bin histograms (the interval starts at the
// candidates' own minimum and maximum, so that the bins spread the values that
// occur), then the chosen entries are emitted in index order, lower index first
// among equal weights.  One cluster of up to 16 CTAs per sequence (8 where the device,
// or the part of it that the process has, cannot place sixteen); each CTA's
// slice lives in registers, K entries a thread, read once, coalesced.  Over
// distributed shared memory go only the non-empty bins, to the first CTA, which
// finds the threshold's bin and, as soon as that holds at most 2048 keys, collects
// those and finishes alone (when all 16 CTAs read the totals from the one that had
// them, a histogram took 8 us of which 1.5 were its counting).
// Emission is by ballots: word w of the slice's bit map is 32 entries, one block
// scan over the words' counts places them all.  Bound: latency (4 bytes read per
// entry; two cluster barriers a histogram).
// evict_select_long_kernel takes sequences of more entries than that cluster's threads
// hold (16 x 32768): a
// radix search with slices that are read again from L2 in each pass.
//
// cache_compact_kernel.  out[b, i] = cache[b, keep[b, i]], a gather of whole
// entries, for all of a sequence's caches in one launch.  Bound: HBM, twice the
// kept bytes.  A block copies a run of rows of one cache; a row's threads hold
// 16-byte pieces of four rows each, all loads before the first store.  (256-byte
// rows, half of 16384 kept: 6.0 TB/s, as cudaMemcpy moves the same bytes.)
#include <atomic>

#include "common.cuh"
#include "evict_plan.cuh"

namespace hyb {

constexpr int kEvBins = 2048;
constexpr int kEvList = 2 * kEvThreads; // keys that the first CTA finishes alone

// Larger weight, larger key; -0 equals +0, NaN ranks as -infinity.
__device__ __forceinline__ uint32_t ev_key(float x)
{
    if (x != x)
        x = -INFINITY;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct EvictParams {
    const float *acc;           // [B, Nc]
    const int32_t *n_valid;     // [B] or NULL
    int32_t *keep;              // [B, n_keep]
    int Nc, n_keep, n_first, n_last;
    int slice;                  // entries per CTA of the cluster
};

struct EvictShared {
    uint32_t hist[3][kEvBins];  // this CTA's counts
    uint32_t total[3][kEvBins]; // the cluster's (in its first CTA)
    uint32_t warp_a[32], warp_b[32];
    uint32_t bin, above, in_bin; // threshold bin of the pass, keys in higher bins and in it
    uint32_t lo_found, left_found, equal_found;   // the threshold, as the first CTA found it
    uint32_t list_n, list[kEvList];               // keys of the threshold's bin (first CTA)
    uint32_t greater, equal;    // this CTA's counts for the emission
    uint32_t lo, hi;            // this CTA's smallest and largest candidate
    uint32_t word_g[32 * kEvKeysMax], word_e[32 * kEvKeysMax];   // bit maps of the slice: kept for sure, at the threshold
    uint32_t word_at[32 * kEvKeysMax], word_eq[32 * kEvKeysMax]; // entries of either kind before a word
};

__device__ __forceinline__ void ev_cluster_add(uint32_t addr, uint32_t v)
{
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ uint32_t ev_cluster_take(uint32_t addr, uint32_t v)
{
    uint32_t old;
    asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(addr), "r"(v) : "memory");
    return old;
}

__device__ __forceinline__ void ev_cluster_st(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Exclusive scan of (a, b) over the block's threads; totals in ta, tb.
__device__ __forceinline__ void ev_scan2(EvictShared &sh, uint32_t &a, uint32_t &b, uint32_t &ta, uint32_t &tb)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t ia = a, ib = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t xa = __shfl_up_sync(0xffffffffu, ia, o), xb = __shfl_up_sync(0xffffffffu, ib, o);
        if (lane >= o) {
            ia += xa;
            ib += xb;
        }
    }
    __syncthreads();             // the previous scan's readers are done
    if (lane == 31) {
        sh.warp_a[warp] = ia;
        sh.warp_b[warp] = ib;
    }
    __syncthreads();
    uint32_t wa = sh.warp_a[lane], wb = sh.warp_b[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t xa = __shfl_up_sync(0xffffffffu, wa, o), xb = __shfl_up_sync(0xffffffffu, wb, o);
        if (lane >= o) {
            wa += xa;
            wb += xb;
        }
    }
    ta = __shfl_sync(0xffffffffu, wa, 31);
    tb = __shfl_sync(0xffffffffu, wb, 31);
    const uint32_t ea = __shfl_sync(0xffffffffu, wa, (warp + 31) & 31), eb = __shfl_sync(0xffffffffu, wb, (warp + 31) & 31);
    a = ia - a + (warp ? ea : 0);
    b = ib - b + (warp ? eb : 0);
}

// The sequence's entry count, and whether there is anything to evict; if not,
// the whole list is written here (every CTA of the cluster agrees).
__device__ __forceinline__ bool ev_count(const EvictParams &p, int b, int rank, int ranks, int &n)
{
    n = p.Nc;
    if (p.n_valid) {
        const int v = p.n_valid[b];
        n = min(max(v, 0), p.Nc);
        if (v != n && rank == 0 && threadIdx.x == 0)
            set_error(HYB_ERR_DEVICE_BOUNDS);
    }
    if (n > p.n_keep)
        return true;
    int32_t *keep = p.keep + (size_t)b * p.n_keep;
    for (int i = rank * kEvThreads + (int)threadIdx.x; i < p.n_keep; i += ranks * kEvThreads)
        keep[i] = i < n ? i : -1;
    return false;
}

__global__ void __launch_bounds__(kEvThreads, 1) evict_select_long_kernel(const EvictParams p)
{
    pdl_wait();      // launched as a programmatic dependent: the previous kernel's writes
    pdl_trigger();   // are visible from here on; the next kernel may start its launch
    extern __shared__ __align__(16) uint8_t ev_raw[];
    EvictShared &sh = *reinterpret_cast<EvictShared *>(ev_raw);
    const int ranks = (int)gridDim.x, rank = (int)blockIdx.x;     // one cluster per sequence, along x
    const int b = blockIdx.y;
    const float *acc = p.acc + (size_t)b * p.Nc;
    int32_t *keep = p.keep + (size_t)b * p.n_keep;
    int n;
    if (!ev_count(p, b, rank, ranks, n))
        return;
    // candidates: [n_first, n - n_last); the others are kept in any case
    const int c0 = p.n_first, c1 = n - p.n_last;
    const uint32_t want = (uint32_t)(p.n_keep - p.n_first - p.n_last);
    const int s0 = min(rank * p.slice, n), s1 = min(s0 + p.slice, n);
    const int a0 = max(s0, c0), a1 = min(s1, c1);
    for (int i = threadIdx.x; i < 3 * kEvBins; i += kEvThreads)
        (&sh.hist[0][0])[i] = 0;
    __syncthreads();
    auto key = [&](int j) { return ev_key(acc[j]); };

    // The threshold: after pass q, `prefix` holds the top bits of the want-th
    // largest key and `left` how many keys with that prefix are still wanted.
    uint32_t prefix = 0, left = want;
    if (want > 0) {
#pragma unroll 1
        for (int q = 0; q < 3; ++q) {
            const int shift = q == 0 ? 21 : q == 1 ? 10 : 0;
            const uint32_t mask = q == 2 ? 1023u : 2047u;
            const int bits = q == 2 ? 10 : 11;
            for (int j0 = a0; j0 < a1; j0 += kEvThreads) {
                const int j = j0 + (int)threadIdx.x;
                const uint32_t k = j < a1 ? key(j) : 0u;
                const bool in = j < a1 && (q == 0 || (k >> (shift + bits)) == prefix);
                const uint32_t bin = (k >> shift) & mask;
                // many equal weights (entries never attended to): one add a warp
                const uint32_t who = __ballot_sync(0xffffffffu, in);
                if (!who)
                    continue;
                const uint32_t lead = __shfl_sync(0xffffffffu, bin, __ffs(who) - 1);
                if (__all_sync(0xffffffffu, !in || bin == lead)) {
                    if ((threadIdx.x & 31) == 0)
                        atomicAdd(&sh.hist[q][lead], (uint32_t)__popc(who));
                } else if (in) {
                    atomicAdd(&sh.hist[q][bin], 1u);
                }
            }
            if (ranks > 1)
                cluster_sync_all();
            else
                __syncthreads();
            // thread i sums bins 2047 - 2i and 2046 - 2i over the cluster (descending)
            uint32_t hb[2];
            for (int e = 0; e < 2; ++e) {
                const int bin = kEvBins - 1 - 2 * (int)threadIdx.x - e;
                if (ranks > 1) {
                    hb[e] = 0;
                    for (int r = 0; r < ranks; ++r)
                        hb[e] += (uint32_t)cluster_ld(cluster_addr(&sh.hist[q][bin], r));
                } else {
                    hb[e] = sh.hist[q][bin];
                }
            }
            uint32_t before = hb[0] + hb[1], unused = 0, total, tu;
            ev_scan2(sh, before, unused, total, tu);
            for (int e = 0; e < 2; ++e) {
                if (before < left && before + hb[e] >= left) {
                    sh.bin = (uint32_t)(kEvBins - 1 - 2 * (int)threadIdx.x - e);
                    sh.above = before;
                }
                before += hb[e];
            }
            __syncthreads();
            prefix = (prefix << bits) | sh.bin;
            left -= sh.above;
            __syncthreads();
        }
    }
    // prefix is the threshold key; keys above it are kept, and the first `left`
    // equal ones.  This CTA's counts, for the other CTAs' offsets.
    auto classify = [&](int j, uint32_t &g, uint32_t &e) {
        g = e = 0;
        if (j >= s1)
            return;
        if (j < c0 || j >= c1) {
            g = 1;
        } else if (want > 0) {
            const uint32_t k = key(j);
            g = k > prefix;
            e = k == prefix;
        }
    };
    uint32_t base_g = 0, base_e = 0;
    if (ranks > 1) {
        uint32_t cg = 0, ce = 0, tg, te;
        for (int j = s0 + (int)threadIdx.x; j < s1; j += kEvThreads) {
            uint32_t g, e;
            classify(j, g, e);
            cg += g;
            ce += e;
        }
        ev_scan2(sh, cg, ce, tg, te);
        if (threadIdx.x == 0) {
            sh.greater = tg;
            sh.equal = te;
        }
        cluster_sync_all();
        for (int r = 0; r < rank; ++r) {
            base_g += (uint32_t)cluster_ld(cluster_addr(&sh.greater, r));
            base_e += (uint32_t)cluster_ld(cluster_addr(&sh.equal, r));
        }
        cluster_sync_all();      // nothing of this CTA's shared memory is read after this
    }
    // emission, in index order; thread i takes four consecutive entries a step
    for (int j0 = s0; j0 < s1; j0 += 4 * kEvThreads) {
        uint32_t g[4], e[4], sg = 0, se = 0, tg, te;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            classify(j0 + 4 * (int)threadIdx.x + i, g[i], e[i]);
            sg += g[i];
            se += e[i];
        }
        ev_scan2(sh, sg, se, tg, te);
        uint32_t og = base_g + sg, oe = base_e + se;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (g[i] || (e[i] && oe < left))
                keep[og + min(oe, left)] = j0 + 4 * (int)threadIdx.x + i;
            og += g[i];
            oe += e[i];
        }
        base_g += tg;
        base_e += te;
    }
}

// The bin that holds the left-th largest key of a histogram (block-wide; hist in
// this CTA): sh.bin, sh.above and sh.in_bin, readable afterwards.
__device__ __forceinline__ void ev_find_bin(EvictShared &sh, const uint32_t *hist, uint32_t left)
{
    const int b0 = kEvBins - 1 - 2 * (int)threadIdx.x;   // thread i: bins 2047 - 2i, 2046 - 2i
    const uint32_t hb[2] = {hist[b0], hist[b0 - 1]};
    uint32_t before = hb[0] + hb[1], unused = 0, ta, tb;
    ev_scan2(sh, before, unused, ta, tb);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (before < left && before + hb[e] >= left) {
            sh.bin = (uint32_t)(b0 - e);
            sh.above = before;
            sh.in_bin = hb[e];
        }
        before += hb[e];
    }
    __syncthreads();
}

// Narrows [lo, hi] to the bin just found; true when the threshold is settled:
// keys > lo are kept, and with `equal` the first `left` equal to lo.
__device__ __forceinline__ bool ev_narrow(uint32_t bin, uint32_t above, uint32_t in_bin, int shift, uint32_t &lo,
                                          uint32_t &hi, uint32_t &left, bool &equal)
{
    left -= above;
    const uint32_t start = lo + (bin << shift);
    if (in_bin == left) {          // the bin is taken whole
        lo = start - 1;            // (keys are at least 0x7fffff)
        left = 0;
        equal = false;
        return true;
    }
    hi = min(hi, start + ((1u << shift) - 1u));
    lo = start;
    return shift == 0;
}

// Shift that spreads [lo, hi] over the bins.
__device__ __forceinline__ int ev_shift(uint32_t lo, uint32_t hi)
{
    return max(0, 21 - __clz(hi - lo));
}

template <int K>
__global__ void __launch_bounds__(kEvThreads, 1) evict_select_kernel(const EvictParams p)
{
    pdl_wait();      // launched as a programmatic dependent: the previous kernel's writes
    pdl_trigger();   // are visible from here on; the next kernel may start its launch
    extern __shared__ __align__(16) uint8_t ev_raw[];
    EvictShared &sh = *reinterpret_cast<EvictShared *>(ev_raw);
    const int ranks = (int)gridDim.x, rank = (int)blockIdx.x;     // one cluster per sequence, along x
    const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int n;
    if (!ev_count(p, b, rank, ranks, n))
        return;
    const float *acc = p.acc + (size_t)b * p.Nc;
    int32_t *keep = p.keep + (size_t)b * p.n_keep;
    // candidates: [n_first, n - n_last); the others are kept in any case
    const int c0 = p.n_first, c1 = n - p.n_last;
    const uint32_t want = (uint32_t)(p.n_keep - p.n_first - p.n_last);
    const int s0 = rank * (K * kEvThreads);
    // entry s0 + 1024 i + thread; keys are never 0, which marks no candidate
    uint32_t key[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int j = s0 + i * kEvThreads + (int)threadIdx.x;
        key[i] = j >= c0 && j < c1 ? ev_key(acc[j]) : 0u;
    }
    for (int i = threadIdx.x; i < 6 * kEvBins; i += kEvThreads)
        (&sh.hist[0][0])[i] = 0;
    if (threadIdx.x == 0)
        sh.list_n = 0;
    uint32_t lo = 0xffffffffu, hi = 0u;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        hi = max(hi, key[i]);
        lo = min(lo, key[i] ? key[i] : 0xffffffffu);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        sh.warp_a[warp] = lo;
        sh.warp_b[warp] = hi;
    }
    __syncthreads();
    lo = __reduce_min_sync(0xffffffffu, sh.warp_a[lane]);
    hi = __reduce_max_sync(0xffffffffu, sh.warp_b[lane]);
    if (ranks > 1) {
        if (threadIdx.x == 0) {
            sh.lo = lo;
            sh.hi = hi;
        }
        cluster_sync_all();
        uint32_t l = 0xffffffffu, h = 0u;
        if (lane < ranks) {
            l = (uint32_t)cluster_ld(cluster_addr(&sh.lo, lane));
            h = (uint32_t)cluster_ld(cluster_addr(&sh.hi, lane));
        }
        lo = __reduce_min_sync(0xffffffffu, l);
        hi = __reduce_max_sync(0xffffffffu, h);
    }
    // The threshold: [lo, hi] holds the want-th largest key, and `left` keys of the
    // interval are still wanted.  Afterwards keys > lo are kept, and with `equal` the
    // first `left` equal to lo.
    uint32_t left = want;
    bool equal = true;
    if (want == 0) {
        lo = 0xffffffffu;
        left = 0;
    } else {
#pragma unroll 1
        for (int q = 0; q < 3; ++q) {
            const int shift = ev_shift(lo, hi);
#pragma unroll
            for (int i = 0; i < K; ++i) {
                const bool in = key[i] >= lo && key[i] <= hi;
                const uint32_t bin = (key[i] - lo) >> shift;
                // many equal weights (entries never attended to): one add a warp
                // where all lanes agree
                const uint32_t who = __ballot_sync(0xffffffffu, in);
                if (!who)
                    continue;
                const uint32_t lead = __shfl_sync(0xffffffffu, bin, __ffs(who) - 1);
                if (__all_sync(0xffffffffu, !in || bin == lead)) {
                    if (lane == 0)
                        atomicAdd(&sh.hist[q][lead], (uint32_t)__popc(who));
                } else if (in) {
                    atomicAdd(&sh.hist[q][bin], 1u);
                }
            }
            __syncthreads();
            if (ranks > 1) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int bin = 2 * (int)threadIdx.x + e;
                    if (sh.hist[q][bin])
                        ev_cluster_add(cluster_addr(&sh.total[q][bin], 0), sh.hist[q][bin]);
                }
                cluster_sync_all();
                if (rank == 0)
                    ev_find_bin(sh, sh.total[q], left);
                cluster_sync_all();
                if (rank != 0) {
                    if (threadIdx.x == 0) {
                        sh.bin = (uint32_t)cluster_ld(cluster_addr(&sh.bin, 0));
                        sh.above = (uint32_t)cluster_ld(cluster_addr(&sh.above, 0));
                        sh.in_bin = (uint32_t)cluster_ld(cluster_addr(&sh.in_bin, 0));
                    }
                    __syncthreads();
                }
            } else {
                ev_find_bin(sh, sh.hist[q], left);
            }
            const uint32_t in_bin = sh.in_bin;
            if (ev_narrow(sh.bin, sh.above, in_bin, shift, lo, hi, left, equal))
                break;
            if (ranks > 1 && in_bin <= (uint32_t)kEvList) {
                // few keys: the first CTA collects them and narrows on alone
#pragma unroll
                for (int i = 0; i < K; ++i) {
                    const bool in = key[i] >= lo && key[i] <= hi;
                    const uint32_t who = __ballot_sync(0xffffffffu, in);
                    if (!who)
                        continue;
                    uint32_t at = 0;
                    if (lane == 0)
                        at = ev_cluster_take(cluster_addr(&sh.list_n, 0), (uint32_t)__popc(who));
                    at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1u));
                    if (in)
                        ev_cluster_st(cluster_addr(&sh.list[at], 0), key[i]);
                }
                cluster_sync_all();
                if (rank == 0) {
#pragma unroll 1
                    for (int f = q + 1; f < 3; ++f) {
                        const int fs = ev_shift(lo, hi);
                        for (uint32_t i = threadIdx.x; i < in_bin; i += kEvThreads) {
                            const uint32_t k = sh.list[i];
                            if (k >= lo && k <= hi)
                                atomicAdd(&sh.hist[f][(k - lo) >> fs], 1u);
                        }
                        __syncthreads();
                        ev_find_bin(sh, sh.hist[f], left);
                        const bool done = ev_narrow(sh.bin, sh.above, sh.in_bin, fs, lo, hi, left, equal);
                        if (done)
                            break;
                    }
                    if (threadIdx.x == 0) {
                        sh.lo_found = lo;
                        sh.left_found = left;
                        sh.equal_found = equal;
                    }
                }
                cluster_sync_all();
                if (rank != 0) {
                    lo = (uint32_t)cluster_ld(cluster_addr(&sh.lo_found, 0));
                    left = (uint32_t)cluster_ld(cluster_addr(&sh.left_found, 0));
                    equal = cluster_ld(cluster_addr(&sh.equal_found, 0)) != 0;
                }
                break;
            }
        }
    }
    // bit maps, one word per 32 entries
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int j = s0 + i * kEvThreads + (int)threadIdx.x;
        const bool g = key[i] > lo || (j < n && (j < c0 || j >= c1));
        const uint32_t wg = __ballot_sync(0xffffffffu, g);
        const uint32_t we = __ballot_sync(0xffffffffu, equal && want > 0 && key[i] == lo && !g);
        if (lane == 0) {
            sh.word_g[i * 32 + warp] = wg;
            sh.word_e[i * 32 + warp] = we;
        }
    }
    __syncthreads();
    // entries before each word (word = thread where there are K x 32 words)
    uint32_t cg = 0, ce = 0, tg, te;
    if (threadIdx.x < 32 * K) {
        cg = __popc(sh.word_g[threadIdx.x]);
        ce = __popc(sh.word_e[threadIdx.x]);
    }
    ev_scan2(sh, cg, ce, tg, te);
    if (threadIdx.x < 32 * K) {
        sh.word_at[threadIdx.x] = cg;
        sh.word_eq[threadIdx.x] = ce;
    }
    uint32_t base_g = 0, base_e = 0;
    if (ranks > 1) {
        if (threadIdx.x == 0) {
            sh.greater = tg;
            sh.equal = te;
        }
        cluster_sync_all();
        uint32_t g = 0, e = 0;
        if (lane < rank) {
            g = (uint32_t)cluster_ld(cluster_addr(&sh.greater, lane));
            e = (uint32_t)cluster_ld(cluster_addr(&sh.equal, lane));
        }
        base_g = __reduce_add_sync(0xffffffffu, g);
        base_e = __reduce_add_sync(0xffffffffu, e);
        cluster_sync_all();      // nothing of this CTA's shared memory is read remotely after this
    } else {
        __syncthreads();
    }
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll 4
    for (int i = 0; i < K; ++i) {
        const int w = i * 32 + warp;
        const uint32_t wg = sh.word_g[w], we = sh.word_e[w];
        const uint32_t oe = base_e + sh.word_eq[w] + __popc(we & below);
        const uint32_t og = base_g + sh.word_at[w] + __popc(wg & below);
        if (((wg >> lane) & 1) || (((we >> lane) & 1) && oe < left))
            keep[og + min(oe, left)] = s0 + i * kEvThreads + (int)threadIdx.x;
    }
}

// The kernel that holds K keys per thread (0: the long one).
typedef void (*EvictKernel)(EvictParams);
static EvictKernel evict_kernel(int keys)
{
    switch (keys) {
    case 0: return evict_select_long_kernel;
    case 1: return evict_select_kernel<1>;
    case 2: return evict_select_kernel<2>;
    case 4: return evict_select_kernel<4>;
    case 8: return evict_select_kernel<8>;
    case 16: return evict_select_kernel<16>;
    default: return evict_select_kernel<32>;
    }
}

static void evict_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&at)[2], int ranks, int B, cudaStream_t stream)
{
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)ranks;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg = {};
    cfg.gridDim = dim3((unsigned)ranks, (unsigned)B);
    cfg.blockDim = dim3(kEvThreads);
    cfg.dynamicSmemBytes = sizeof(EvictShared);
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 2;
}

// The largest cluster that the current device can place, after setting the kernels'
// attributes; asked once per device (below 64), like the attributes.
static std::atomic<int> g_evict_cluster[64];

static cudaError_t evict_cluster(int &cluster)
{
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const bool known = dev >= 0 && dev < 64;
    cluster = known ? g_evict_cluster[dev].load(std::memory_order_acquire) : 0;
    if (cluster)
        return cudaSuccess;
    cluster = kEvCluster;
    for (int keys = 0; keys <= kEvKeysMax; keys = keys ? 2 * keys : 1) {
        EvictKernel kern = evict_kernel(keys);
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(EvictShared));
        if (e == cudaSuccess && keys)
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess)
            return e;
        if (!keys)
            continue;
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute at[2];
        evict_config(cfg, at, kEvCluster, 1, nullptr);
        cfg.attrs = &at[1];            // the cluster alone
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
        if (e != cudaSuccess)
            cudaGetLastError();        // (a part of a GPU may refuse the question itself)
        if (e != cudaSuccess || n < 1)
            cluster = kEvPortable;
    }
    if (known)
        g_evict_cluster[dev].store(cluster, std::memory_order_release);
    return cudaSuccess;
}

cudaError_t launch_evict_select(const float *acc, int B, int Nc, const int32_t *n_valid, int n_keep, int n_first,
                                int n_last, int32_t *keep, cudaStream_t stream, int num_sms)
{
    EvictParams p = {};
    p.acc = acc;
    p.n_valid = n_valid;
    p.keep = keep;
    p.Nc = Nc;
    p.n_keep = n_keep;
    p.n_first = n_first;
    p.n_last = n_last;
    int cluster = 0;
    const cudaError_t e = evict_cluster(cluster);
    if (e != cudaSuccess)
        return e;
    const EvictPlan plan = evict_plan(B, Nc, num_sms, cluster);
    p.slice = plan.slice;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute at[2];
    evict_config(cfg, at, plan.ranks, B, stream);
    return cudaLaunchKernelEx(&cfg, evict_kernel(plan.keys), p);
}

constexpr int kCpArrays = 7;
constexpr int kCpThreads = 256;
constexpr int kCpUnroll = 4;

struct CompactArray {
    const uint8_t *src;         // [B, Nc] rows
    uint8_t *dst;               // [B, No] rows
    int vec;                    // bytes of a piece: 16, 8 or 4
    int ppr;                    // pieces per row
    int tpr_log2;               // threads per row
    int rpb;                    // rows per block
    int bps;                    // blocks per sequence
    long long block0;           // first block of this array
};

struct CompactParams {
    CompactArray a[kCpArrays];
    int n_arrays, n_keep, Nc, No;
    const int32_t *keep;        // [B, n_keep]
};

template <typename V>
__device__ __forceinline__ void compact_rows(const CompactParams &p, const CompactArray &a, int b, int r0)
{
    const int c0 = threadIdx.x & ((1 << a.tpr_log2) - 1), rr = threadIdx.x >> a.tpr_log2;
    const int pass = kCpThreads >> a.tpr_log2;              // rows a step
    const V *src = reinterpret_cast<const V *>(a.src) + (size_t)b * p.Nc * a.ppr;
    V *dst = reinterpret_cast<V *>(a.dst) + ((size_t)b * p.No + r0) * a.ppr;
    const int32_t *keep = p.keep + (size_t)b * p.n_keep + r0;
    int e[kCpUnroll];
#pragma unroll
    for (int k = 0; k < kCpUnroll; ++k) {
        const int r = rr + k * pass;
        e[k] = r < p.n_keep - r0 ? __ldg(keep + r) : -1;
        if (e[k] >= p.Nc) {
            set_error(HYB_ERR_DEVICE_BOUNDS);
            e[k] = -1;
        }
    }
    for (int c = c0; c < a.ppr; c += 1 << a.tpr_log2) {
        V v[kCpUnroll];
#pragma unroll
        for (int k = 0; k < kCpUnroll; ++k)
            if (e[k] >= 0)
                v[k] = src[(size_t)e[k] * a.ppr + c];
#pragma unroll
        for (int k = 0; k < kCpUnroll; ++k)
            if (e[k] >= 0)
                dst[(size_t)(rr + k * pass) * a.ppr + c] = v[k];
    }
}

__global__ void __launch_bounds__(kCpThreads) cache_compact_kernel(const __grid_constant__ CompactParams p)
{
    pdl_wait();
    pdl_trigger();
    int w = 0;
    while (w + 1 < p.n_arrays && (long long)blockIdx.x >= p.a[w + 1].block0)
        ++w;
    const CompactArray &a = p.a[w];
    const unsigned k = (unsigned)(blockIdx.x - a.block0);
    const int b = (int)(k / (unsigned)a.bps), r0 = (int)(k % (unsigned)a.bps) * a.rpb;
    if (a.vec == 16)
        compact_rows<uint4>(p, a, b, r0);
    else if (a.vec == 8)
        compact_rows<uint2>(p, a, b, r0);
    else
        compact_rows<uint32_t>(p, a, b, r0);
}

// One cache to rewrite: rows of row_bytes (a multiple of four).
struct CompactTensor {
    const void *src;
    void *dst;
    long long row_bytes;
};

cudaError_t launch_cache_compact(const CompactTensor *t, int n, int B, int Nc, int No, const int32_t *keep,
                                 int n_keep, cudaStream_t stream)
{
    CompactParams p = {};
    p.n_keep = n_keep;
    p.Nc = Nc;
    p.No = No;
    p.keep = keep;
    long long blocks = 0;
    for (int i = 0; i < n; ++i) {
        if (!t[i].src)
            continue;
        CompactArray &a = p.a[p.n_arrays++];
        a.src = static_cast<const uint8_t *>(t[i].src);
        a.dst = static_cast<uint8_t *>(t[i].dst);
        // the widest piece that rows and both addresses allow
        const unsigned long long bits = (unsigned long long)t[i].row_bytes | reinterpret_cast<uintptr_t>(t[i].src) |
                                        reinterpret_cast<uintptr_t>(t[i].dst);
        a.vec = bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : 4;
        a.ppr = (int)(t[i].row_bytes / a.vec);
        a.tpr_log2 = 0;
        while ((1 << a.tpr_log2) < a.ppr && (1 << a.tpr_log2) < kCpThreads)
            ++a.tpr_log2;
        a.rpb = (kCpThreads >> a.tpr_log2) * kCpUnroll;
        a.bps = (n_keep + a.rpb - 1) / a.rpb;
        a.block0 = blocks;
        blocks += (long long)B * a.bps;
    }
    if (blocks == 0)
        return cudaSuccess;
    if (blocks >= (1LL << 31))
        return cudaErrorInvalidValue;
    return launch_pdl(cache_compact_kernel, dim3((unsigned)blocks), dim3(kCpThreads), 0, stream, p);
}

}  // namespace hyb
