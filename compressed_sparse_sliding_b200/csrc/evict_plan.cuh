// evict_plan.cuh -- how a selection is laid out over a cluster of CTAs per sequence.
// Plain host arithmetic, without CUDA: the tests compile it by itself.
#pragma once

namespace hyb {

constexpr int kEvThreads = 1024;
constexpr int kEvCluster = 16;          // CTAs of a sequence at most (over 8: opted in)
constexpr int kEvPortable = 8;          // ... wherever the device cannot place sixteen
constexpr int kEvKeysMax = 32;          // keys per thread held in registers

struct EvictPlan {
    int ranks;      // CTAs of a sequence
    int keys;       // keys per thread, in registers (a power of two); 0: slices read again from L2
    int slice;      // entries per CTA where keys is 0, whole 4-entry groups
};

// CTAs a sequence: more while SMs are free and a slice keeps two keys a thread, and
// as many as let the keys stay in registers.
inline EvictPlan evict_plan(int B, int Nc, int num_sms, int cluster)
{
    int ranks = 1;
    while (ranks < cluster && (long long)B * ranks * 2 <= num_sms && Nc / (ranks * 2) >= 2 * kEvThreads)
        ranks *= 2;
    while (ranks < cluster && Nc > ranks * kEvKeysMax * kEvThreads)
        ranks *= 2;
    const int per = (Nc + ranks - 1) / ranks;
    int keys = 1;
    while (keys < kEvKeysMax && keys * kEvThreads < per)
        keys *= 2;
    if (keys * kEvThreads < per) {
        keys = 0;
        ranks = kEvPortable;
    }
    return {ranks, keys, ((Nc + ranks - 1) / ranks + 3) & ~3};
}

}  // namespace hyb
