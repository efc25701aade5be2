// evict.cu -- eviction from bounded caches: which entries a sequence keeps by
// their accumulated attention weight, and the caches rewritten with them.
//
// evict_select_kernel.  Exact selection of the largest weights by a radix
// search for the threshold: three histogram passes (11 + 11 + 10 bits of an
// order-preserving integer image of the weight), then one pass that emits the
// chosen entries in index order, lower index first among equal weights.  One
// cluster of up to eight CTAs per sequence: each holds a contiguous slice of the
// sequence's keys in shared memory (read from HBM once; slices that do not fit
// are read again from L2), and the CTAs add their histograms over distributed
// shared memory, so one long sequence still uses eight SMs.  Bound: latency (a
// few block-wide scans and four cluster barriers; 4 bytes read per entry).
//
// cache_compact_kernel.  out[b, i] = cache[b, keep[b, i]], a gather of whole
// entries, for all of a sequence's caches in one launch.  Bound: HBM, twice the
// kept bytes.  A block copies a run of rows of one cache in 16-byte pieces, eight
// loads per thread before the first store.
#include "common.cuh"

namespace hyb {

constexpr int kEvThreads = 1024;
constexpr int kEvBins = 2048;
constexpr int kEvSliceMax = 32768;      // keys of a slice held in shared memory (128 KB)
constexpr int kEvCluster = 8;

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
    int held;                   // the slice's keys stay in shared memory
};

struct EvictShared {
    uint32_t hist[3][kEvBins];
    uint32_t warp_a[32], warp_b[32];
    uint32_t bin, above;        // threshold bin of the pass, keys in higher bins
    uint32_t base_a, base_b;
    uint32_t greater, equal;    // this CTA's counts for the emission
};

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

__global__ void __launch_bounds__(kEvThreads, 1) evict_select_kernel(const EvictParams p)
{
    pdl_wait();      // launched as a programmatic dependent: the previous kernel's writes
    pdl_trigger();   // are visible from here on; the next kernel may start its launch
    __shared__ EvictShared sh;
    extern __shared__ __align__(16) uint32_t ev_keys[];
    const int ranks = (int)gridDim.x, rank = (int)blockIdx.x;     // one cluster per sequence, along x
    const int b = blockIdx.y;
    const float *acc = p.acc + (size_t)b * p.Nc;
    int32_t *keep = p.keep + (size_t)b * p.n_keep;
    int n = p.Nc;
    if (p.n_valid) {
        const int v = p.n_valid[b];
        n = min(max(v, 0), p.Nc);
        if (v != n && rank == 0 && threadIdx.x == 0)
            set_error(HYB_ERR_DEVICE_BOUNDS);
    }
    if (n <= p.n_keep) {         // nothing to evict (every CTA of the cluster agrees)
        for (int i = rank * kEvThreads + (int)threadIdx.x; i < p.n_keep; i += ranks * kEvThreads)
            keep[i] = i < n ? i : -1;
        return;
    }
    // candidates: [n_first, n - n_last); the others are kept in any case
    const int c0 = p.n_first, c1 = n - p.n_last;
    const uint32_t want = (uint32_t)(p.n_keep - p.n_first - p.n_last);
    const int s0 = min(rank * p.slice, n), s1 = min(s0 + p.slice, n);
    const int a0 = max(s0, c0), a1 = min(s1, c1);
    for (int i = threadIdx.x; i < 3 * kEvBins; i += kEvThreads)
        (&sh.hist[0][0])[i] = 0;
    if (p.held)
        for (int j = a0 + (int)threadIdx.x; j < a1; j += kEvThreads)
            ev_keys[j - s0] = ev_key(acc[j]);
    __syncthreads();
    auto key = [&](int j) { return p.held ? ev_keys[j - s0] : ev_key(acc[j]); };

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
    // more CTAs a sequence while SMs are free and a slice has work for its threads
    int ranks = 1;
    while (ranks < kEvCluster && (long long)B * ranks * 2 <= num_sms && Nc / (ranks * 2) >= 2 * kEvThreads)
        ranks *= 2;
    // ... and as many as let the keys stay in shared memory
    while (ranks < kEvCluster && (Nc + ranks - 1) / ranks > kEvSliceMax)
        ranks *= 2;
    // slices of whole 4-entry groups
    p.slice = ((Nc + ranks - 1) / ranks + 3) & ~3;
    p.held = p.slice <= kEvSliceMax;
    const size_t smem = p.held ? (size_t)p.slice * 4 : 0;
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kEvSliceMax * 4);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)ranks;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)ranks, (unsigned)B);
    cfg.blockDim = dim3(kEvThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
}

constexpr int kCpArrays = 7;
constexpr int kCpThreads = 256;
constexpr int kCpUnroll = 8;

struct CompactArray {
    const uint8_t *src;         // [B, Nc] rows
    uint8_t *dst;               // [B, No] rows
    int vec;                    // bytes of a piece: 16, 8 or 4
    int ppr;                    // pieces per row
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
__device__ __forceinline__ void compact_rows(const CompactParams &p, const CompactArray &a, int b, int r0, int nr)
{
    const V *src = reinterpret_cast<const V *>(a.src) + (size_t)b * p.Nc * a.ppr;
    V *dst = reinterpret_cast<V *>(a.dst) + ((size_t)b * p.No + r0) * a.ppr;
    const int32_t *keep = p.keep + (size_t)b * p.n_keep + r0;
    const int n = nr * a.ppr;
    for (int i0 = threadIdx.x; i0 < n; i0 += kCpThreads * kCpUnroll) {
        V v[kCpUnroll];
        int at[kCpUnroll];
#pragma unroll
        for (int k = 0; k < kCpUnroll; ++k) {
            const int i = i0 + k * kCpThreads;
            at[k] = -1;
            if (i < n) {
                const int r = (int)((unsigned)i / (unsigned)a.ppr), c = i - r * a.ppr;
                const int e = __ldg(keep + r);
                if (e >= p.Nc)
                    set_error(HYB_ERR_DEVICE_BOUNDS);
                if (e >= 0 && e < p.Nc) {
                    at[k] = i;
                    v[k] = src[(size_t)e * a.ppr + c];
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kCpUnroll; ++k)
            if (at[k] >= 0)
                dst[at[k]] = v[k];
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
    const int nr = min(a.rpb, p.n_keep - r0);
    if (a.vec == 16)
        compact_rows<uint4>(p, a, b, r0, nr);
    else if (a.vec == 8)
        compact_rows<uint2>(p, a, b, r0, nr);
    else
        compact_rows<uint32_t>(p, a, b, r0, nr);
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
        const int per = kCpThreads * kCpUnroll;
        a.rpb = a.ppr < per ? per / a.ppr : 1;
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
