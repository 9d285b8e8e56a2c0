// Partition of a prompt attention: packed sequences into blocks of query tokens,
// longest first, blocks of many steps cut where that fills the GPU.
//
// A block is up to 256 query rows of one sequence and one key head: t =
// floor(128 / group) tokens per 128-row tile, with `group` query heads each, and
// two tiles.  It walks ceil(seen / 128) steps of 128 keys, `seen` being what its
// last token sees.  With S steps in all, times h_kv heads, over the GPU's P
// SMs, c = max(kMinSteps, ceil(S h_kv / P)) is an SM's share; a block of s > c
// steps is cut into ceil(s / c) parts of near-equal length whose partial results
// the combine joins.  So one long sequence with few heads fills the GPU, and a
// batch of prompts with many heads is not cut at all.
//
// One CTA: the bounds of up to 1024 sequences sit in shared memory, and the blocks
// are gone through three times (steps in all; how many segments have each length;
// their places, a counting sort).  The segments of a length come in no fixed order:
// which SM runs one has no influence on a result.
#include <cuda_runtime.h>

#include "mla_prefill.cuh"
#include "mla_schedule.cuh"
#include "mla_sm103.cuh"

namespace mla {
namespace {

constexpr int kThreads = 1024;
constexpr int kMinSteps = 8;     // of a part: below it the partial results cost more than the steps
constexpr int kLengths = 1024;   // lengths that the sort tells apart

struct Shared {
    long long warp[kThreads / 32];
    long long end[kThreads];     // blocks up to and with each sequence of the chunk
    int q[kThreads], lq[kThreads], k[kThreads], lk[kThreads];
    int count[kLengths];         // segments of each length; then their first place
    int slots, cuts, scan[kThreads / 32];
    unsigned long long steps;
};

// f(segment with all steps) for every block, the threads sharing the blocks of
// 1024 sequences at a time
template <typename F>
__device__ void each_block(const PrefillParams &p, Shared &sh, bool report, F f) {
    const int per = kPreTiles * pre_tile_tokens(p.group);
    for (int c0 = 0; c0 < p.batch; c0 += kThreads) {
        const int n = min(kThreads, p.batch - c0), b = c0 + threadIdx.x;
        // the bounds stay in shared memory where one chunk holds all sequences
        if (report || p.batch > kThreads) {
            int q = 0, lq = 0, k = 0, lk = 0;
            if ((int)threadIdx.x < n) {
                q = p.cu_q[b], k = p.cu_k[b];
                const int q1 = p.cu_q[b + 1], k1 = p.cu_k[b + 1];
                if (q < 0 || q1 < q || q1 > p.num_q || k < 0 || k1 < k || k1 > p.num_k) {
                    if (report) atomicOr(p.status, MLA_DEVERR_SEQLEN);
                    q = k = 0;
                } else {
                    lq = q1 - q, lk = k1 - k;
                }
            }
            sh.q[threadIdx.x] = q, sh.lq[threadIdx.x] = lq, sh.k[threadIdx.x] = k, sh.lk[threadIdx.x] = lk;
            long long total;
            const long long blocks = (lq + per - 1) / per;
            const long long before = block_exclusive_scan<kThreads>(blocks, sh.warp, &total);
            sh.end[threadIdx.x] = before + blocks;
            __syncthreads();
        }
        for (long long i = threadIdx.x; i < sh.end[n - 1]; i += kThreads) {
            int lo = 0, hi = n - 1;  // the first sequence whose blocks end behind i
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (sh.end[mid] > i) hi = mid;
                else lo = mid + 1;
            }
            const int first = (int)(i - (lo ? sh.end[lo - 1] : 0)) * per;
            PreSegment s;
            s.q0 = sh.q[lo] + first;
            s.tokens = min(per, sh.lq[lo] - first);
            s.k0 = sh.k[lo];
            s.keys = sh.lk[lo];
            s.seen = p.causal ? sh.lk[lo] - sh.lq[lo] + first + 1 : sh.lk[lo];
            s.step0 = 0;
            s.step1 = pre_steps(pre_seen(s, s.tokens - 1));
            s.slot = -1;
            f(s);
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kThreads) prefill_schedule_kernel(const PrefillParams p) {
    __shared__ Shared sh;
    if (threadIdx.x == 0) sm103::griddep_launch_dependents();
    sm103::griddep_wait();
    PreHeader *header = reinterpret_cast<PreHeader *>(p.metadata);
    PreSegment *segments = reinterpret_cast<PreSegment *>(header + 1);
    PreCut *cuts = reinterpret_cast<PreCut *>(segments + p.max_segments);
    for (int i = threadIdx.x; i < kLengths; i += kThreads) sh.count[i] = 0;
    if (threadIdx.x == 0) {
        sh.slots = sh.cuts = 0;
        sh.steps = 0;
    }
    __syncthreads();
    unsigned long long mine = 0;
    each_block(p, sh, true, [&](const PreSegment &s) { mine += s.step1; });
    if (mine) atomicAdd(&sh.steps, mine);
    __syncthreads();
    const unsigned long long share = (sh.steps * p.h_kv + p.sms - 1) / p.sms;
    const int most = share < kMinSteps ? kMinSteps : share > 0x7fffffff ? 0x7fffffff : (int)share;
    // parts of a block: the first `longer` of them have one step more than the others
    auto parts = [&](const PreSegment &s, int &shorter, int &longer) {
        const int n = s.step1 > most ? (s.step1 + most - 1) / most : 1;
        shorter = s.step1 / n;
        longer = s.step1 - shorter * n;
        return n;
    };
    // most steps first: bucket 0 holds the longest
    auto bucket = [](int steps) { return kLengths - 1 - min(steps, kLengths - 1); };
    each_block(p, sh, false, [&](const PreSegment &s) {
        int shorter, longer;
        const int n = parts(s, shorter, longer);
        if (longer) atomicAdd(&sh.count[bucket(shorter + 1)], longer);
        atomicAdd(&sh.count[bucket(shorter)], n - longer);
    });
    {
        int total;
        const int here = sh.count[threadIdx.x];
        const int first = block_exclusive_scan<kThreads>(here, sh.scan, &total);
        sh.count[threadIdx.x] = first;
        if (threadIdx.x == 0) header->segments = (int)min((long long)total, (long long)p.max_segments);
        __syncthreads();
    }
    each_block(p, sh, false, [&](PreSegment s) {
        int shorter, longer;
        const int n = parts(s, shorter, longer);
        int slot = -1;
        if (n > 1) {
            slot = atomicAdd(&sh.slots, n);
            const int at = atomicAdd(&sh.cuts, 1);
            if (at < p.max_slots) cuts[at] = {s.q0, s.tokens, slot, n};
        }
        int step = 0;
        for (int i = 0; i < n; ++i) {
            s.step0 = step;
            s.step1 = step += shorter + (i < longer);
            s.slot = n > 1 ? slot + i : -1;
            const int at = atomicAdd(&sh.count[bucket(s.step1 - s.step0)], 1);
            if (at < p.max_segments) segments[at] = s;
        }
    });
    if (threadIdx.x == 0) header->cuts = min(sh.cuts, p.max_slots);
}

}  // namespace

cudaError_t launch_prefill_schedule(const PrefillParams &p, cudaStream_t stream) {
    return launch_after(prefill_schedule_kernel, dim3(1), dim3(kThreads), 0, stream, p);
}

}  // namespace mla
