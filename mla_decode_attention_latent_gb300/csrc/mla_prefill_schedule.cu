// Partition of a prompt attention: packed sequences into blocks of query tokens,
// longest first, and some of them into parts.
//
// A block is up to 256 query rows of one sequence and one key head: t =
// floor(128 / group) tokens per 128-row tile, with `group` query heads each, and
// two tiles.  It walks ceil(seen / 128) steps of 128 keys, `seen` being what its
// last token sees.
//
// The items (segment, key head) go to the CTAs in rounds, longest first
// (pre_round_item).  A segment is a block, or a part of one: blocks of more than c
// steps are cut into ceil(steps / c) equal parts, whose partial results the combine
// joins.  32 values of c around an even share of the work are tried, and none: with n
// items of F + steps units each (F: an item's fixed cost), the last CTA is estimated to
// end at the larger of an even share of all units and, for the ceil(n / ctas) rounds,
// the longest item and a shortest one for every further round; a cut costs C for the
// combine, and has to gain an eighth.  So few rows over many keys fill the GPU, and a
// batch of prompts with many heads is not cut at all.  (Equal shares of a line of all
// items instead, each CTA beginning inside an item, kept three chunks behind long
// contexts as busy, 80 against 82 us, but 512 equal items took 258 us for 231: the heads
// of a moment then share no keys in L2.)
//
// One CTA.  Up to 1280 blocks, as many as there are where any is cut, are kept in shared
// memory; more are gone through twice.  The segments are put in order by counting how
// many have each length (a rank for each, a loop over all, took 1.4 us longer for 200
// blocks); the order of equal ones has no influence on a result.  12 prompts of 200 blocks take
// 4 us, 9 where cuts are looked for.
#include <cuda_runtime.h>

#include <mutex>

#include "mla_prefill.cuh"
#include "mla_schedule.cuh"
#include "mla_sm103.cuh"

namespace mla {
namespace {

constexpr int kFixed = 8;        // units of an item beside its steps (2 / 4 / 8 / 12: three chunks 86 / 86 / 84 / 84 us)
constexpr int kCombine = 3;      // units of the combine
constexpr int kLeastPart = 4;    // steps of a part
constexpr int kLengths = 1024;   // lengths that the counting sort tells apart
constexpr int kKept = 1280;      // blocks or segments kept in shared memory: as many as there are where any is cut
constexpr int kMany = 1024, kFew = 256;  // threads; few: for as many sequences and blocks, whose barriers cost less

template <int kThreads>
struct Shared {
    long long warp[kThreads / 32];
    long long end[kThreads];     // blocks up to and with each sequence of the chunk
    int q[kThreads], lq[kThreads], k[kThreads], lk[kThreads];
    int count[kLengths];         // blocks or segments of each length, longest first; then the next one's place
    int scan[kThreads / 32];
    int cost[32];                // estimates of the values of c
    int cuts, parts;
    PreSegment block[kKept];
    int first[kKept];            // segments before each block
    int length[kKept], owner[kKept];  // of each segment, and its block
};

// f(block, its index) for every block, the threads sharing the blocks of kThreads sequences at a time; their number
template <int kThreads, typename F>
__device__ long long each_block(const PrefillParams &p, Shared<kThreads> &sh, bool again, F f) {
    const int per = kPreTiles * pre_tile_tokens(p.group);
    long long base = 0;
    for (int c0 = 0; c0 < p.batch; c0 += kThreads) {
        const int n = min(kThreads, p.batch - c0), b = c0 + threadIdx.x;
        // the bounds stay in shared memory where one chunk holds all sequences
        if (!again || p.batch > kThreads) {
            int q = 0, lq = 0, k = 0, lk = 0;
            if ((int)threadIdx.x < n) {
                q = p.cu_q[b], k = p.cu_k[b];
                const int q1 = p.cu_q[b + 1], k1 = p.cu_k[b + 1];
                if (q < 0 || q1 < q || q1 > p.num_q || k < 0 || k1 < k || k1 > p.num_k) {
                    if (!again) atomicOr(p.status, MLA_DEVERR_SEQLEN);
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
            PreSegment x;
            x.q0 = sh.q[lo] + first;
            x.tokens = min(per, sh.lq[lo] - first);
            x.k0 = sh.k[lo];
            x.keys = sh.lk[lo];
            x.seen = p.causal ? sh.lk[lo] - sh.lq[lo] + first + 1 : sh.lk[lo];
            x.step0 = 0;
            x.step1 = pre_steps(pre_seen(x, x.tokens - 1));
            x.part = -1;
            f(x, base + i);
        }
        base += sh.end[n - 1];
        __syncthreads();
    }
    return base;
}

// parts of a block of `steps` for c = most; the first `longer` of them have one step more than the others
__device__ __forceinline__ int cut(int steps, int most, int &shorter, int &longer) {
    const int n = steps > most ? (int)(((unsigned)steps + most - 1) / (unsigned)most) : 1;
    shorter = (int)((unsigned)steps / (unsigned)n);
    longer = steps - shorter * n;
    return n;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) prefill_schedule_kernel(const PrefillParams p) {
    extern __shared__ __align__(16) char raw[];
    Shared<kThreads> &sh = *reinterpret_cast<Shared<kThreads> *>(raw);
    if (threadIdx.x == 0) sm103::griddep_launch_dependents();
    sm103::griddep_wait();
    const PreWork work(p.metadata, p.max_blocks, p.sms);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < kLengths; i += kThreads) sh.count[i] = 0;
    if (threadIdx.x == 0) {
        sh.cuts = sh.parts = 0;
    }
    __syncthreads();
    // places instead of numbers, from the longest on
    auto to_places = [&] {
        constexpr int kOwn = kLengths / kThreads;
        int here[kOwn], sum = 0, total;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) sum += here[i] = sh.count[threadIdx.x * kOwn + i];
        int at = block_exclusive_scan<kThreads>(sum, sh.scan, &total);
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            sh.count[threadIdx.x * kOwn + i] = at;
            at += here[i];
        }
        __syncthreads();
    };
    auto bucket = [](int steps) { return kLengths - 1 - min(steps, kLengths - 1); };
    long long steps = 0;  // of this thread's blocks
    const long long found = each_block(p, sh, false, [&](const PreSegment &x, long long i) {
        if (i < kKept) sh.block[i] = x;
        if constexpr (kThreads == kMany) atomicAdd(&sh.count[bucket(x.step1)], 1);
        steps += x.step1;
    });
    const int blocks = (int)min(found, (long long)p.max_blocks);
    if (kThreads == kMany && blocks > kKept) {
        to_places();
        each_block(p, sh, true, [&](const PreSegment &x, long long i) {
            const int at = atomicAdd(&sh.count[bucket(x.step1)], 1);
            if (at < blocks) work.segments[at] = x;
        });
        if (threadIdx.x == 0) *work.header = {blocks, 0, (int)p.causal, p.group, p.h_kv, {}};
        return;
    }
    int most = 0x7fffffff;  // c
    if (blocks > 0 && pre_may_cut(p.max_blocks, p.num_k, p.h_kv, p.sms) && kPreRounds * p.sms <= kKept) {
        long long all_steps;
        block_exclusive_scan<kThreads>(steps, sh.warp, &all_steps);
        // values of c, one per warp at a time: the last none, the others from a quarter to four times an even share
        const float share = (float)all_steps * p.h_kv / p.sms;
        auto value = [&](int w) { return w == 31 ? 0x7fffffff : max(kLeastPart, (int)ceilf(fminf(share * exp2f((float)w * (4.f / 30.f) - 2.f), 1e9f))); };
        for (int w = warp; w < 32; w += kThreads / 32) {
            const int c = value(w);
            int n = 0, parts = 0, longest = 0, shortest = 0x7fffffff;
            float units = 0.f;
            for (int i = lane; i < blocks; i += 32) {
                int shorter, longer;
                const int all = sh.block[i].step1, mine = cut(all, c, shorter, longer);
                n += mine;
                parts += mine > 1 ? mine : 0;
                units += (float)all;
                longest = max(longest, shorter + (longer > 0));
                shortest = min(shortest, shorter);
            }
#pragma unroll
            for (int off = 16; off; off >>= 1) units += __shfl_xor_sync(0xffffffffu, units, off);
            n = __reduce_add_sync(0xffffffffu, n);  // (c is at least a quarter of an even share: at most the blocks and four times the CTAs)
            parts = __reduce_add_sync(0xffffffffu, parts);
            longest = __reduce_max_sync(0xffffffffu, longest);
            shortest = __reduce_min_sync(0xffffffffu, shortest);
            const long long items = (long long)n * p.h_kv;
            const bool fits = items <= (long long)kPreRounds * p.sms && (long long)parts * p.h_kv <= pre_slots(p.sms);
            const float rounds = fits || c == 0x7fffffff ? ceilf((float)items / p.sms) : 0.f;
            const float even = (units + (float)kFixed * n) * p.h_kv / p.sms;
            const float end = fmaxf(even, longest + kFixed + (rounds - 1.f) * (shortest + kFixed)) + (parts ? kCombine : 0);
            if (lane == 0) sh.cost[w] = fits || c == 0x7fffffff ? (int)fminf(end, 5e7f) : 60000000;
        }
        __syncthreads();
        // the least of them, and whether it gains an eighth on not cutting
        const unsigned mine = (unsigned)sh.cost[lane] * 32 + lane, least = __reduce_min_sync(0xffffffffu, mine);
        if ((long long)(least / 32) * 8 < (long long)sh.cost[31] * 7) most = value(least % 32);
    }
    if constexpr (kThreads == kMany) {
        for (int i = threadIdx.x; i < kLengths; i += kThreads) sh.count[i] = 0;
    }
    // where each block's segments begin
    int segments = 0;
    for (int c0 = 0; c0 < blocks; c0 += kThreads) {
        const int i = c0 + threadIdx.x;
        int shorter = 0, longer = 0, n = 0;
        if (i < blocks) n = cut(sh.block[i].step1, most, shorter, longer);
        int total;
        const int first = segments + block_exclusive_scan<kThreads>(n, sh.scan, &total);
        if (i < blocks) sh.first[i] = first;
        if (n > 1) {
            const int part = atomicAdd(&sh.parts, n);  // (which slots a block has makes no difference)
            sh.block[i].part = part;
            work.cuts[atomicAdd(&sh.cuts, 1)] = {sh.block[i].q0, sh.block[i].tokens, part, n};
        }
        segments += total;
    }
    __syncthreads();
    // a thread per segment: its block and its part of it, then its place
    for (int at = threadIdx.x; at < segments; at += kThreads) {
        int i = 0, hi = blocks;  // first[i] <= at < first[i + 1]
        while (hi - i > 1) {
            const int mid = (i + hi) >> 1;
            if (sh.first[mid] <= at) i = mid;
            else hi = mid;
        }
        int shorter, longer;
        cut(sh.block[i].step1, most, shorter, longer);
        const int mine = shorter + (at - sh.first[i] < longer);
        sh.length[at] = mine;
        sh.owner[at] = i;
        atomicAdd(&sh.count[bucket(mine)], 1);
    }
    __syncthreads();
    to_places();
    for (int at = threadIdx.x; at < segments; at += kThreads) {
        const int i = sh.owner[at], mine = sh.length[at], k = at - sh.first[i];
        PreSegment x = sh.block[i];
        int shorter, longer;
        const int n = cut(x.step1, most, shorter, longer);
        x.step0 = k * shorter + min(k, longer);
        x.step1 = x.step0 + mine;
        x.part = n > 1 ? x.part + k : -1;
        work.segments[atomicAdd(&sh.count[bucket(mine)], 1)] = x;
    }
    if (threadIdx.x == 0) *work.header = {segments, sh.cuts, (int)p.causal, p.group, p.h_kv, {}};
}

template <int kThreads>
cudaError_t launch(const PrefillParams &p, cudaStream_t stream) {
    constexpr int kMaxDevices = 64;
    static std::mutex mutex;
    static bool ready[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mutex);
        if (!ready[dev]) {
            e = cudaFuncSetAttribute(prefill_schedule_kernel<kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared<kThreads>));
            if (e != cudaSuccess) return e;
            ready[dev] = true;
        }
    }
    return launch_after(prefill_schedule_kernel<kThreads>, dim3(1), dim3(kThreads), sizeof(Shared<kThreads>), stream, p);
}

}  // namespace

cudaError_t launch_prefill_schedule(const PrefillParams &p, cudaStream_t stream) {
    const bool few = p.batch <= kFew && p.max_blocks <= kFew;
    return few ? launch<kFew>(p, stream) : launch<kMany>(p, stream);
}

}  // namespace mla
