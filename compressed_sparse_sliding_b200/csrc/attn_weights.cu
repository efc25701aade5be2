// attn_weights.cu -- the attention weight that each cached entry received:
//   acc[b, j] (+)= sum over query tokens t and heads h of
//                  exp(scale q[b, t, h] . kc[b, j, h / g] - lse[b, h, t])
// over the entries j that are visible to t (or that idx lists), with the lse of
// the attention that ran before.  What an eviction keeps a cache by.
//
// Mathematics and bound.  lse is known, so the softmax needs no running
// maximum: each score is exponentiated once and summed over the query rows.
// K is read once (2 d bytes per entry and KV head) and nothing of size
// rows x entries is ever stored; with few query rows (decode) the K stream from
// HBM bounds it, with many (the last tokens of a prompt) the exponentials.
//
// Layout.  S^T = K Q^T on tcgen05: keys are the MMA's M, so a TMEM lane is a key
// and the sum over query rows stays inside one thread.  Four epilogue warpgroups
// take key tiles in turn where a CTA has many (64 sequences x 16384 entries, 64
// heads: 47.5 us; all four on every tile: 62.2, same GPU and before the waits were
// shortened), and otherwise share every tile: every fourth 32-row column chunk, the
// sums added through shared memory.  Each entry has one owner, and equal calls give
// equal bits (only a selection adds with atomics, for entries listed more than once:
// their copies are equal, so any order gives the same sum).  A CTA owns a run of key
// tiles of one or more sequences, every CTA the same number of tiles that hold visible
// entries.  Four S buffers (4 x 128 TMEM columns) and the K stages keep copies, MMAs
// and exponentials of different tiles running together.  Query blocks (hpt heads x
// tpt tokens, up to 128 rows) stay in shared memory for the whole run where all of a
// sequence's fit 64 KB (decode: four K stages).  Otherwise they stream, through twice
// the bytes and beside two K stages, since a K tile then serves many blocks.
//
// Measured (one B200): 64 sequences x 16384 entries (three quarters visible), 64
// heads over one KV head of 128: 43.4 us, 4.6 TB/s of K; 1024 selected entries of
// each: 17 us with the copy of acc before it, of which the gather's and the
// barriers' latencies are most; 32 query tokens x 32 heads over 2 x 8192 entries:
// 16.6 us.  A streamed block takes about 1 us of a CTA: what writes its lse and counts
// was most of it (128 tokens: 54.8 us with two warps for that, 36.5 with the loads
// left out, 40.2 with four warps), and a tile that some query tokens do not see whole
// costs more than the others, so that the CTA that has it ends last (scalar reads
// of lse and counts there: 24.0 us in place of 19).
//
// Roles (768 threads): warps 0-15 epilogue (thread = key), warp 16 TMA producer,
// warp 17 MMA issue, warps 18 and 19 (without a selection 18 to 21) write the query
// blocks' lse and visible counts beside them, a slot always by the same warp; warps
// 20-23 gather the selected rows with cp.async when idx is given (16 lanes per row).
#include "common.cuh"

#include <atomic>

namespace hyb {

constexpr int kAwThreads = 768;
constexpr int kAwWgs = 4;           // epilogue warpgroups
// 512 x 88 + 256 x 64 = 768 x 80 (the launch's registers); one share for all spills
// more: 46.0 us for the decode case above where the split takes 44.4
constexpr int kAwEpiRegs = 88, kAwOtherRegs = 64;
constexpr int kAwBM = 128;          // keys of a tile
constexpr int kAwKStages = 4;       // with resident queries; 2 with streamed ones
constexpr int kAwSBufs = 4;
constexpr int kAwQBytes = 64 * 1024;   // resident queries; streamed ones have two K stages' bytes more
constexpr int kAwQStages = 16;      // barrier slots; the bytes usually bind first
// Sequences whose visible counts a CTA sums up at its start, to cut the stream of
// all visible tiles evenly, and the positions it reads for that; with more, a
// CTA's share counts full caches and its many sequences even out.
constexpr int kAwCounted = 1024, kAwPositions = 8192;
constexpr int kAwZero = 4096;       // entries zeroed at a time

struct WeightParams {
    int B, Lq, Hq, Hkv, g, Nc, m, W, e0, K;
    int hpt, tpt, nht, ntt;         // heads and tokens of a query block; head and token tiles of a KV head
    int split;                      // 1: the epilogue warpgroups share a tile's columns; 0: take alternate tiles
    int NB;                         // MMA columns of a block (rows rounded up to 16)
    int nqs, resident;              // query slots; all blocks of a sequence fit them
    int tiles;                      // key tiles of a full cache (idx: of the selection)
    int counted;                    // runs by visible tiles (see kAwCounted)
    int accumulate;
    float scale_log2;
    const int32_t *q_pos, *idx;
    const float *lse;
    const __nv_bfloat16 *kc;
    float *acc;
};

template <int D>
struct WeightSmem {
    static constexpr int K_BYTES = kAwBM * D * 2;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = kAwQBytes;
    static constexpr int OFF_COL = OFF_K + kAwKStages * K_BYTES;     // -lse (log2) per column, then counts
    // streamed queries have the bytes of two K stages more for their slots
    static constexpr int Q_STREAM = kAwQBytes + (kAwKStages - 2) * K_BYTES;
    static constexpr int NCOL = Q_STREAM / (D * 2);                  // columns of all slots together
    static constexpr int OFF_SUM = OFF_COL + NCOL * 8;               // [2][3][128] sums of the other warpgroups
    static constexpr int OFF_NV = OFF_SUM + 2 * (kAwWgs - 1) * kAwBM * 4;   // [kAwCounted] visible entries
    static constexpr int OFF_CUM = OFF_NV + kAwCounted * 4;          // [kAwCounted + 1] visible tiles before
    static constexpr int OFF_BAR = OFF_CUM + (kAwCounted + 4) * 4;
    static constexpr int OFF_MISC = OFF_BAR + 64 * 8;
    static constexpr int BYTES = OFF_MISC + 128;
};
static_assert(1024 + WeightSmem<128>::BYTES <= 227 * 1024, "shared memory of a CTA");

// barrier slots
enum { WB_QF = 0, WB_QE = 16, WB_KF = 32, WB_KE = 36, WB_SF = 40, WB_SE = 44, WB_TF = 48, WB_TE = 50, WB_DONE = 52 };

// A stretch of one sequence's key tiles, the work of a CTA between two sequence
// changes.
struct WeightRun {
    int b, nv;         // sequence; entries that some query token of it sees
    int lo, hi;        // key tiles of this run
    int z0, z1;        // entries this run zeroes (not counted: those no query token sees)
};

__device__ __forceinline__ int aw_visible(const WeightParams &p, int flat)
{
    const long long pos = p.q_pos ? p.q_pos[flat] : flat % p.Lq;
    const int nv = pf_visible(pos, p.m, p.W, p.e0 + p.Nc);
    return max(nv - p.e0, 0);
}

__device__ __forceinline__ int aw_tiles(const WeightParams &p, int nv)
{
    return ((p.idx ? p.K : nv) + kAwBM - 1) / kAwBM;
}

// Walks a CTA's runs (whole warp; every role walks the same ones).
struct WeightWalk {
    long long u, end;
    int b;
    const int *nvs, *cum;

    __device__ __forceinline__ WeightWalk(const WeightParams &p, const int *nv_, const int *cum_)
        : b(0), nvs(nv_), cum(cum_)
    {
        const long long total = p.counted ? cum[p.B] : (long long)p.B * p.tiles;
        if (total < (1 << 20)) {       // (a 64-bit division is a hundred instructions)
            u = (unsigned)total * blockIdx.x / gridDim.x;
            end = (unsigned)total * (blockIdx.x + 1) / gridDim.x;
        } else {
            u = total * blockIdx.x / gridDim.x;
            end = total * (blockIdx.x + 1) / gridDim.x;
        }
        if (p.counted && u < end) {
            // the sequence of tile u: the last one with cum <= u
            int lo = 0, hi = p.B - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (cum[mid] <= (int)u)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            b = lo;
        }
    }

    __device__ __forceinline__ bool next(const WeightParams &p, int lane, WeightRun &r)
    {
        if (u >= end)
            return false;
        r.z0 = r.z1 = 0;
        if (p.counted) {
            while (cum[b + 1] <= (int)u)
                ++b;
            r.b = b;
            r.nv = nvs[b];
            r.lo = (int)u - cum[b];
            r.hi = min(cum[b + 1], (int)end) - cum[b];
            u += r.hi - r.lo;
            return true;
        }
        // shares of full caches: a sequence's visible tiles are spread over its share
        r.b = u < (1ll << 31) ? (int)((unsigned)u / (unsigned)p.tiles) : (int)(u / p.tiles);
        const int a0 = (int)(u - (long long)r.b * p.tiles);
        const int a1 = (int)min((long long)p.tiles, a0 + (end - u));
        u += a1 - a0;
        int nv = 0;
        for (int t = lane; t < p.Lq; t += 32)
            nv = max(nv, aw_visible(p, r.b * p.Lq + t));
        r.nv = __reduce_max_sync(0xffffffffu, nv);
        if (p.idx) {                   // as many tiles as a full selection
            r.lo = a0;
            r.hi = a1;
            return true;
        }
        const long long T = aw_tiles(p, r.nv);
        r.lo = (int)(T * a0 / p.tiles);
        r.hi = (int)(T * a1 / p.tiles);
        if (!p.accumulate && !p.idx) {
            r.z0 = r.nv + (int)((long long)(p.Nc - r.nv) * a0 / p.tiles);
            r.z1 = r.nv + (int)((long long)(p.Nc - r.nv) * a1 / p.tiles);
        }
        return true;
    }
};

// S buffer of block i of a CTA's nt-th tile, and how often it was used before: a
// warpgroup's own buffer, or the four in turn.
__device__ __forceinline__ void aw_buffer(const WeightParams &p, uint32_t nt, int nblocks, int i, uint32_t &buf,
                                          uint32_t &round)
{
    static_assert(kAwSBufs == kAwWgs, "a buffer a warpgroup");
    if (p.split) {
        const uint32_t n = nt * nblocks + i;
        buf = n % kAwSBufs;
        round = n / kAwSBufs;
    } else {
        buf = nt % kAwWgs;
        round = nt / kAwWgs * nblocks + i;
    }
}

template <int D, bool STREAM>
__global__ void __launch_bounds__(kAwThreads, 1)
attn_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const WeightParams p)
{
    using SM = WeightSmem<D>;
    constexpr int NCB = D / 64;
    constexpr int KS_LOG2 = STREAM ? 1 : 2;      // K stages
    constexpr uint32_t nks = 1u << KS_LOG2;
    extern __shared__ __align__(1024) uint8_t aw_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(aw_smem_raw) + 1023) &
                                                ~(uintptr_t)1023);
    uint8_t *sQ = smem + SM::OFF_Q;
    uint8_t *sK = smem + SM::OFF_K + (kAwKStages - nks) * SM::K_BYTES;
    float *sLse = reinterpret_cast<float *>(smem + SM::OFF_COL);       // -lse, log2 units, per slot and column
    int *sNv = reinterpret_cast<int *>(smem + SM::OFF_COL + SM::NCOL * 4);
    float *sSum = reinterpret_cast<float *>(smem + SM::OFF_SUM);
    int *sSeq = reinterpret_cast<int *>(smem + SM::OFF_NV);
    int *sCum = reinterpret_cast<int *>(smem + SM::OFF_CUM);
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + SM::OFF_BAR);
    int *misc = reinterpret_cast<int *>(smem + SM::OFF_MISC);
    int *sMin = misc + 8;                                              // [16] least count of a slot's columns
    volatile int *abort_flag = misc + 1;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kAwQStages; ++s) {
            mbar_init(&bar[WB_QF + s], 1 + 32);    // the TMA copy, the lanes of the slot's column warp
            mbar_init(&bar[WB_QE + s], 1 + 4 * kAwWgs);   // the MMA, the epilogue warps
        }
        for (int s = 0; s < kAwKStages; ++s) {
            mbar_init(&bar[WB_KF + s], p.idx ? 128 : 1);
            mbar_init(&bar[WB_KE + s], 1);
        }
        for (int s = 0; s < kAwSBufs; ++s) {
            mbar_init(&bar[WB_SF + s], 1);
            mbar_init(&bar[WB_SE + s], p.split ? 4 * kAwWgs : 4);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar[WB_TF + s], 4 * (kAwWgs - 1));   // the other warpgroups' sums
            mbar_init(&bar[WB_TE + s], 4);
        }
        mbar_init(&bar[WB_DONE], 1);
        mbar_fence_init();
        misc[1] = 0;
    }
    for (int b = threadIdx.x; p.counted && b < p.B; b += kAwThreads)
        sSeq[b] = 0;
    if (warp == 17)
        tmem_alloc(reinterpret_cast<uint32_t *>(&misc[0]), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)misc[0];
    pdl_wait();      // launched as a programmatic dependent: the previous kernel's writes
    pdl_trigger();   // are visible from here on; the next kernel may start its launch
    const int tries = wait_tries();
    if (p.counted) {
        const int n = p.B * p.Lq;
#pragma unroll 4
        for (int i = threadIdx.x; i < n; i += kAwThreads) {
            const int nv = aw_visible(p, i);
            if (nv > 0)
                atomicMax(&sSeq[p.Lq == 1 ? i : i / p.Lq], nv);
        }
        __syncthreads();
        if (warp == 0) {
            int before = 0;
            for (int b0 = 0; b0 < p.B; b0 += 32) {
                const int b = b0 + lane;
                int t = b < p.B ? aw_tiles(p, sSeq[b]) : 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, t, o);
                    t += lane >= o ? x : 0;
                }
                if (b < p.B)
                    sCum[b + 1] = before + t;
                before += __shfl_sync(0xffffffffu, t, 31);
            }
            if (lane == 0)
                sCum[0] = 0;
        }
        __syncthreads();
    }

    const uint32_t qbytes = (uint32_t)p.NB * D * 2;
    const int nblocks = p.Hkv * p.ntt * p.nht;     // query blocks of a sequence
    auto wait = [&](int b, uint32_t parity) {      // whole warp
        return __all_sync(0xffffffffu, mbar_wait_short(&bar[b], parity, abort_flag, tries)) != 0;
    };
    WeightWalk walk(p, sSeq, sCum);
    WeightRun r;
    bool ok = true;
    uint32_t runs = 0;                             // runs with tiles so far
    // Query slots go round (streamed blocks): the next use's slot, and its fill's parity.
    uint32_t ring = 0, ring_par = 0;
    auto advance = [&]() {
        if (++ring == (uint32_t)p.nqs) {
            ring = 0;
            ring_par ^= 1;
        }
    };
    // The blocks of a sequence, by KV head, token tile and head tile (no divisions:
    // they would cost more than a block's other instructions).
    auto for_blocks = [&](auto f) {
        int i = 0;
        for (int h = 0; ok && h < p.Hkv; ++h)
            for (int tt = 0; ok && tt < p.ntt; ++tt)
                for (int ht = 0; ok && ht < p.nht; ++ht, ++i)
                    f(i, h, tt * p.tpt, ht * p.hpt, tt + ht == 0, tt == p.ntt - 1 && ht == p.nht - 1);
    };

    if (warp >= 16)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAwOtherRegs));
    // Without a selection two of the gather's warps write columns too.  A slot always has
    // the same warp: one that ran a fill ahead would take the parity of the fill before
    // for its own.
    const int ncw = p.idx ? 2 : 4;
    if (warp == 16 || (warp >= 18 && warp < 18 + ncw)) {
        // ============ query blocks: copies (warp 16), lse and counts (warps 18 on); K tiles (warp 16) ============
        uint32_t kc = 0, qc = 0;
        const uint32_t box_bytes = (uint32_t)p.hpt * p.tpt * D * 2;
        while (ok && walk.next(p, lane, r)) {
            for (int tile = r.lo; ok && tile < r.hi; ++tile) {
                const bool load_q = STREAM || tile == r.lo;
                if (!load_q && (warp >= 18 || p.idx))
                    break;
                for_blocks([&](int i, int h, int t0, int h0, bool first, bool) {
                    if (warp == 16 && first && !p.idx) {
                        const uint32_t st = kc & (nks - 1);
                        if (kc >= nks && !(ok = wait(WB_KE + st, ((kc >> KS_LOG2) - 1) & 1)))
                            return;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&bar[WB_KF + st], SM::K_BYTES);
                            for (int cb = 0; cb < NCB; ++cb)
                                tma_load_4d(sK + st * SM::K_BYTES + cb * kAwBM * 128, &tm_k, &bar[WB_KF + st],
                                            cb * 64, h, tile * kAwBM, r.b);
                        }
                        __syncwarp();
                        ++kc;
                    }
                    if (!load_q)
                        return;
                    const uint32_t st = STREAM ? ring : i, par = STREAM ? ring_par : runs & 1;
                    const bool used = STREAM ? qc >= (uint32_t)p.nqs : runs > 0;
                    if (warp >= 18 && (st & (ncw - 1)) != (uint32_t)(warp - 18)) {
                        ++qc;              // another warp's slot
                        advance();
                        return;
                    }
                    if (warp == 16) {
                        if (used && !(ok = wait(WB_QE + st, par ^ 1)))
                            return;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&bar[WB_QF + st], box_bytes);
                            for (int cb = 0; cb < NCB; ++cb)
                                tma_load_4d(sQ + st * qbytes + cb * p.NB * 128, &tm_q, &bar[WB_QF + st], cb * 64,
                                            h * p.g + h0, t0, r.b);
                        }
                        __syncwarp();
                    } else {
                        // up to four columns a lane, all loads before the slot's wait
                        float l[4];
                        int nv[4], least = INT_MAX;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int c = lane + 32 * k;
                            l[k] = 0.f;
                            nv[k] = 0;
                            if (c < p.hpt * p.tpt) {
                                const int dt = c / p.hpt, t = t0 + dt, hd = h0 + c - dt * p.hpt;
                                if (t < p.Lq && hd < p.g) {
                                    l[k] = p.lse[((size_t)r.b * p.Hq + h * p.g + hd) * p.Lq + t];
                                    nv[k] = p.Lq == 1 ? r.nv : aw_visible(p, r.b * p.Lq + t);
                                    least = min(least, nv[k]);
                                }
                            }
                        }
                        least = __reduce_min_sync(0xffffffffu, least);
                        if (used && !(ok = wait(WB_QE + st, par ^ 1)))
                            return;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int c = lane + 32 * k;
                            if (c < p.NB) {
                                sLse[st * p.NB + c] = -1.4426950408889634f * l[k];
                                sNv[st * p.NB + c] = nv[k];
                            }
                        }
                        if (lane == 0)
                            sMin[st] = least;
                        mbar_arrive(&bar[WB_QF + st]);
                    }
                    ++qc;
                    advance();
                });
            }
            if (r.hi > r.lo)
                ++runs;
        }
        if (warp == 16 && lane == 0) {
            // unwinding: wait for the last copies issued into every slot
            for (uint32_t c = (kc > nks ? kc - nks : 0); c < kc; ++c)
                drain_wait(&bar[WB_KF + (c & (nks - 1))], (c >> KS_LOG2) & 1);
            if (STREAM) {
                for (uint32_t c = (qc > (uint32_t)p.nqs ? qc - p.nqs : 0); c < qc; ++c)
                    drain_wait(&bar[WB_QF + c % p.nqs], (c / p.nqs) & 1);
            } else {
                for (uint32_t c = 0; c < qc && c < (uint32_t)nblocks; ++c)
                    drain_wait(&bar[WB_QF + c], ((qc - 1 - c) / nblocks) & 1);
            }
        }
    } else if (warp >= 20) {
        // ============================ selected rows: gather ============================
        if (p.idx) {
            constexpr int CH = D / 8;              // 16-byte chunks of a row
            constexpr int RPI = 128 / CH;          // rows a pass
            constexpr int N = kAwBM / RPI;
            const int pt = threadIdx.x - 20 * 32;
            const int c8 = pt % CH, rsub = pt / CH;
            const uint32_t dchunk = (c8 >> 3) * kAwBM * 128;
            uint32_t kc = 0;
            while (ok && walk.next(p, lane, r)) {
                for (int tile = r.lo; ok && tile < r.hi; ++tile) {
                    int src[N];
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const int slot = tile * kAwBM + i * RPI + rsub;
                        src[i] = slot < p.K ? __ldg(p.idx + (size_t)r.b * p.K + slot) : -1;
                    }
                    bool bad = false;
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        bad |= src[i] >= p.Nc;
                        src[i] = src[i] < r.nv ? src[i] : -1;
                    }
                    if (bad && c8 == 0)
                        set_error(HYB_ERR_DEVICE_BOUNDS);
                    for (int h = 0; h < p.Hkv; ++h) {
                        const uint32_t st = kc & (nks - 1);
                        if (kc >= nks && !(ok = wait(WB_KE + st, ((kc >> KS_LOG2) - 1) & 1)))
                            break;
                        const uint32_t dst = smem_u32(sK + st * SM::K_BYTES) + dchunk;
#pragma unroll
                        for (int i = 0; i < N; ++i)
                            cp_async_16(dst + sw128_offset(i * RPI + rsub, c8 & 7),
                                        p.kc + (((size_t)r.b * p.Nc + max(src[i], 0)) * p.Hkv + h) * D + c8 * 8,
                                        src[i] >= 0 ? 16u : 0u);
                        cp_async_mbar_arrive(&bar[WB_KF + st]);
                        mbar_arrive(&bar[WB_KF + st]);
                        ++kc;
                    }
                }
            }
            cp_async_wait_group<0>();
        }
    } else if (warp == 17) {
        // ================================ MMA issue ================================
        const uint32_t idesc = idesc_bf16(kAwBM, p.NB, false, false);
        const uint64_t dQ = sw128_desc(smem_u32(sQ), 16, 1024), dK = sw128_desc(smem_u32(sK), 16, 1024);
        uint32_t kc = 0, nt = 0;
        const bool leader = elect_one();
        while (ok && walk.next(p, lane, r)) {
            for (int tile = r.lo; ok && tile < r.hi; ++tile, ++nt) {
                for_blocks([&](int i, int, int, int, bool first, bool last) {
                    const uint32_t qs = STREAM ? ring : i, par = STREAM ? ring_par : runs & 1;
                    const uint32_t ks = kc & (nks - 1);
                    uint32_t buf, round;
                    aw_buffer(p, nt, nblocks, i, buf, round);
                    if (!(ok = wait(WB_QF + qs, par)))
                        return;
                    advance();
                    if (first) {
                        if (!(ok = wait(WB_KF + ks, (kc >> KS_LOG2) & 1)))
                            return;
                        if (p.idx)
                            fence_proxy_async_smem();   // rows written by cp.async, read by the MMA
                    }
                    if (round > 0 && !(ok = wait(WB_SE + buf, (round - 1) & 1)))
                        return;
                    tc_fence_after();
                    if (leader) {
                        // (addresses are the low bits of a descriptor, in 16-byte units)
                        const uint64_t da = dK + (ks * SM::K_BYTES >> 4), db = dQ + (qs * qbytes >> 4);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            mma_bf16_ss(tmem + buf * 128, da + (kk >> 2) * (kAwBM * 8) + (kk & 3) * 2,
                                        db + (kk >> 2) * (p.NB * 8) + (kk & 3) * 2, idesc, kk > 0 ? 1u : 0u);
                        }
                        mma_commit(&bar[WB_SF + buf]);
                        if (last)
                            mma_commit(&bar[WB_KE + ks]);
                        if (STREAM || tile == r.hi - 1)
                            mma_commit(&bar[WB_QE + qs]);
                    }
                    __syncwarp();
                    kc += last;
                });
            }
            if (r.hi > r.lo)
                ++runs;
        }
        if (leader)
            mma_commit(&bar[WB_DONE]);
        __syncwarp();
        drain_wait(&bar[WB_DONE], 0);
    } else if (warp < 4 * kAwWgs) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAwEpiRegs));
        // ============================ exponentials and sums ============================
        const int x = warp >> 2;
        const int quad = warp & 3;
        const int key = quad * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
        const uint64_t sc2 = f2(p.scale_log2, p.scale_log2);
        uint32_t nt = 0;                    // tiles so far
        if (p.counted && !p.accumulate && !p.idx) {
            // entries that no query token sees
            const int per = (p.Nc + kAwZero - 1) / kAwZero;
            for (int w = blockIdx.x; w < p.B * per; w += gridDim.x) {
                const int b = w / per, c = (w - b * per) * kAwZero, end = min(p.Nc, c + kAwZero);
                for (int j = max(sSeq[b], c) + (int)threadIdx.x; j < end; j += 128 * kAwWgs)
                    p.acc[(size_t)b * p.Nc + j] = 0.f;
            }
        }
        while (ok && walk.next(p, lane, r)) {
            for (int j = r.z0 + (int)threadIdx.x; j < r.z1; j += 128 * kAwWgs)
                p.acc[(size_t)r.b * p.Nc + j] = 0.f;
            for (int tile = r.lo; ok && tile < r.hi; ++tile, ++nt) {
                if (!p.split && (int)(nt % kAwWgs) != x)
                    continue;                            // another warpgroup's
                const int j = tile * kAwBM + key;        // entry, or slot of the selection
                const int key_at = p.idx ? 0 : j;        // every listed entry is seen
                int e = -1;
                if (p.idx && (!p.split || x == 0) && j < p.K)
                    e = __ldg(p.idx + (size_t)r.b * p.K + j);
                float tot = 0.f;
                for_blocks([&](int i, int, int t0, int h0, bool, bool) {
                    const uint32_t qs = STREAM ? ring : i, par = STREAM ? ring_par : runs & 1;
                    uint32_t buf, round;
                    aw_buffer(p, nt, nblocks, i, buf, round);
                    if (!(ok = wait(WB_QF + qs, par) && wait(WB_SF + buf, round & 1)))
                        return;
                    advance();
                    tc_fence_after();
                    // rows of this block: whole tokens, or the heads of a group's last tile
                    const int ncv = min(p.hpt, p.g - h0) * min(p.tpt, p.Lq - t0);
                    const bool full = p.idx || (tile + 1) * kAwBM <= sMin[qs];
                    const uint32_t tS = tl + buf * 128;
                    const float *nl = sLse + qs * p.NB;
                    const int *cn = sNv + qs * p.NB;
#pragma unroll 1
                    for (int c = p.split ? 32 * x : 0; c < ncv; c += p.split ? 32 * kAwWgs : 32) {
                        if (full && c + 32 <= ncv) {
                            float sv[32];
                            tmem_ld32(tS + c, sv);
                            tmem_ld_wait();
                            uint64_t s2[2] = {0ull, 0ull};
#pragma unroll
                            for (int q = 0; q < 32; q += 4) {
                                const ulonglong2 l2 = *reinterpret_cast<const ulonglong2 *>(nl + c + q);
                                float a0, a1, b0, b1;
                                f2_split(fma_f2(f2(sv[q], sv[q + 1]), sc2, l2.x), a0, a1);
                                f2_split(fma_f2(f2(sv[q + 2], sv[q + 3]), sc2, l2.y), b0, b1);
                                s2[0] = add_f2(s2[0], f2(ex2_approx(a0), ex2_approx(a1)));
                                s2[1] = add_f2(s2[1], f2(ex2_approx(b0), ex2_approx(b1)));
                            }
                            float a0, a1;
                            f2_split(add_f2(s2[0], s2[1]), a0, a1);
                            tot += a0 + a1;
                        } else {
                            // some columns are padding (count 0; from NB on there are none), or do
                            // not see every key of the tile
#pragma unroll 1
                            for (int c1 = c; c1 < min(c + 32, ncv); c1 += 16) {
                                float sv[16], s = 0.f;
                                tmem_ld16(tS + c1, sv);
                                tmem_ld_wait();
#pragma unroll
                                for (int q = 0; q < 16; q += 4) {
                                    const float4 l4 = *reinterpret_cast<const float4 *>(nl + c1 + q);
                                    const int4 n4 = *reinterpret_cast<const int4 *>(cn + c1 + q);
                                    const float l[4] = {l4.x, l4.y, l4.z, l4.w};
                                    const int nv[4] = {n4.x, n4.y, n4.z, n4.w};
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        const float e = ex2_approx(fmaf(sv[q + k], p.scale_log2, l[k]));
                                        s += key_at < nv[k] ? e : 0.f;
                                    }
                                }
                                tot += s;
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&bar[WB_SE + buf]);
                        if (STREAM)
                            mbar_arrive(&bar[WB_QE + qs]);   // this warp has read the slot's columns
                    }
                });
                if (!ok)
                    break;
                if (p.split) {
                    // the warpgroups' sums meet
                    const uint32_t tb = nt & 1, round = nt >> 1;
                    float *sums = sSum + tb * (kAwWgs - 1) * kAwBM + key;
                    if (x > 0) {
                        if (round > 0 && !(ok = wait(WB_TE + tb, (round - 1) & 1)))
                            break;
                        sums[(x - 1) * kAwBM] = tot;
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(&bar[WB_TF + tb]);
                        continue;
                    }
                    if (!(ok = wait(WB_TF + tb, round & 1)))
                        break;
#pragma unroll
                    for (int k = 0; k < kAwWgs - 1; ++k)
                        tot += sums[k * kAwBM];
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&bar[WB_TE + tb]);
                }
                if (p.idx) {
                    // an entry listed twice counts twice, whichever is added first
                    if (e >= 0 && e < r.nv)
                        atomicAdd(&p.acc[(size_t)r.b * p.Nc + e], tot);
                } else if (j < r.nv) {
                    float *a = &p.acc[(size_t)r.b * p.Nc + j];
                    *a = p.accumulate ? *a + tot : tot;
                }
            }
            if (ok && !STREAM && r.hi > r.lo) {
                // this warp has read the run's columns (it waits for them even where it
                // had no tile of the run, so that it never releases a slot a run ahead)
                for (int i = 0; ok && i < nblocks; ++i) {
                    ok = wait(WB_QF + i, runs & 1);
                    if (ok && lane == 0)
                        mbar_arrive(&bar[WB_QE + i]);
                }
            }
            if (r.hi > r.lo)
                ++runs;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc((uint32_t)misc[0], 512);
    }
}

__global__ void __launch_bounds__(256) attn_weights_zero_kernel(float *acc, long long n)
{
    pdl_wait();
    pdl_trigger();
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256)
        acc[i] = 0.f;
}

// Devices (below 64) on which a kernel's attributes are set, by d and by layout.
static std::atomic<unsigned long long> g_weights_ready[2][2];

template <int D>
static cudaError_t launch_weights_t(WeightParams &p, const void *q, const void *kc, cudaStream_t stream,
                                    int num_sms)
{
    using SM = WeightSmem<D>;
    const int slot = p.NB * D * 2;
    p.nqs = min(kAwQBytes / slot, kAwQStages);
    p.resident = (long long)p.Hkv * p.ntt * p.nht <= p.nqs;
    if (!p.resident)
        p.nqs = min(SM::Q_STREAM / slot, kAwQStages);
    p.split = !p.resident || (long long)p.B * p.tiles < 2LL * num_sms;
    CUtensorMap mq, mk;
    if (!make_map(&mq, q, D, p.Hq, p.Lq, p.B, p.hpt, p.tpt) ||
        !make_map(&mk, kc, D, p.Hkv, p.Nc, p.B, 1, kAwBM))
        return cudaErrorInvalidValue;
    const size_t ask = 1024 + SM::BYTES < 120 * 1024 ? 120 * 1024 : 1024 + SM::BYTES;
    auto kern = p.resident ? attn_weights_kernel<D, false> : attn_weights_kernel<D, true>;
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    std::atomic<unsigned long long> &ready = g_weights_ready[D == 128][!p.resident];
    if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ask);
        if (e == cudaSuccess)
            e = check_reg_split(kern, kAwThreads, 128 * kAwWgs, kAwEpiRegs, kAwOtherRegs);
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            ready.fetch_or(1ull << dev, std::memory_order_release);
    }
    if (p.idx && !p.accumulate) {
        const long long n = (long long)p.B * p.Nc;
        const long long blocks = (n + 1023) / 1024;
        e = launch_pdl(attn_weights_zero_kernel, dim3((unsigned)(blocks < num_sms * 8 ? blocks : num_sms * 8)),
                       dim3(256), 0, stream, p.acc, n);
        if (e != cudaSuccess)
            return e;
    }
    const long long tiles = (long long)p.B * p.tiles;
    const long long grid = tiles < num_sms ? tiles : num_sms;
    return launch_pdl(kern, dim3((unsigned)grid), dim3(kAwThreads), ask, stream, mq, mk, p);
}

cudaError_t launch_attn_weights(int B, int Lq, int Hq, int Hkv, int d, int Nc, int m, int W, int e0, int K,
                                float scale, const int32_t *q_pos, const void *q, const void *kc,
                                const float *lse, const int32_t *idx, float *acc, int accumulate,
                                cudaStream_t stream, int num_sms)
{
    WeightParams p = {};
    p.B = B;
    p.Lq = Lq;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.g = Hq / Hkv;
    p.Nc = Nc;
    p.m = m;
    p.W = W;
    p.e0 = e0;
    p.K = idx ? K : 0;
    p.hpt = p.g < 128 ? p.g : 128;
    p.tpt = 128 / p.hpt < Lq ? 128 / p.hpt : Lq;
    p.nht = (p.g + p.hpt - 1) / p.hpt;
    p.ntt = (Lq + p.tpt - 1) / p.tpt;
    p.NB = (p.hpt * p.tpt + 15) / 16 * 16;
    p.tiles = ((idx ? K : Nc) + kAwBM - 1) / kAwBM;
    // (with idx every sequence has the same number of tiles: shares are even as they are)
    p.counted = !idx && B <= kAwCounted && (long long)B * Lq <= kAwPositions && (long long)B * p.tiles < (1LL << 31);
    p.accumulate = accumulate;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.q_pos = q_pos;
    p.idx = idx;
    p.lse = lse;
    p.kc = static_cast<const __nv_bfloat16 *>(kc);
    p.acc = acc;
    return d == 128 ? launch_weights_t<128>(p, q, kc, stream, num_sms)
                    : launch_weights_t<64>(p, q, kc, stream, num_sms);
}

}  // namespace hyb
