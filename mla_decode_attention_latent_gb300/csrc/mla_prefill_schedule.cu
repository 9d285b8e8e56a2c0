// Partition of a prompt attention: packed sequences into blocks of query tokens,
// longest first, and the items (block, key head) onto the CTAs.
//
// A block is up to 256 query rows of one sequence and one key head: t =
// floor(128 / group) tokens per 128-row tile, with `group` query heads each, and
// two tiles.  It walks ceil(seen / 128) steps of 128 keys, `seen` being what its
// last token sees.  Two ways to share the items, of which the one is taken that is
// estimated to end first (the line where it gains an eighth: 512 equal items of 152 CTAs
// lose 7 % on it):
//   rounds  whole items, in rounds over the CTAs (pre_round_item)
//   line    the items one behind the other, each taking F + steps units (F: its fixed
//           cost), cut into equal shares; a unit inside an item's first F moves to its
//           start.  Items that a share ends in are cut along their keys, and the
//           combine (cost C) joins the partial results
// Rounds suit many items: nothing is cut and the heads of a moment are few.  The line
// suits few rows over many keys, and counts that leave most CTAs idle in a last round.
//
// One CTA.  The bounds of up to 1024 sequences sit in shared memory, and the blocks
// are gone through twice (how many have each length; their places, a counting sort).
// Where the line may be taken the sort is stable, so that the same call always cuts the
// same items; in rounds the order of equal blocks has no influence on a result.
#include <cuda_runtime.h>

#include "mla_prefill.cuh"
#include "mla_schedule.cuh"
#include "mla_sm103.cuh"

namespace mla {
namespace {

constexpr int kThreads = 1024;
constexpr int kFixed = 2;        // units of an item beside its steps
constexpr int kCombine = 3;      // units of the combine
constexpr int kLeastShare = 6;   // units of a share on the line
constexpr int kLengths = 1024;   // lengths that the sort tells apart
constexpr int kStable = 1280;    // blocks that are sorted stably: as many as a line can have, and more

struct Shared {
    long long warp[kThreads / 32];
    long long end[kThreads];     // blocks up to and with each sequence of the chunk
    int q[kThreads], lq[kThreads], k[kThreads], lk[kThreads];
    int count[kLengths];         // blocks of each length; then their first place
    int scan[kThreads / 32];
    int longest, cuts;
    PrePlace place[kThreads / 4 + 1];
    short bucket[kStable];       // of each block
    long long units[kStable + 1];  // on the line before each block
};

// f(block, its index) for every block, the threads sharing the blocks of 1024 sequences at a time
template <typename F>
__device__ void each_block(const PrefillParams &p, Shared &sh, bool report, F f) {
    const int per = kPreTiles * pre_tile_tokens(p.group);
    long long base = 0;
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
            PreBlock x;
            x.q0 = sh.q[lo] + first;
            x.tokens = min(per, sh.lq[lo] - first);
            x.k0 = sh.k[lo];
            x.keys = sh.lk[lo];
            x.seen = p.causal ? sh.lk[lo] - sh.lq[lo] + first + 1 : sh.lk[lo];
            x.steps = pre_steps(pre_seen(x, x.tokens - 1));
            x.pad[0] = x.pad[1] = 0;
            f(x, base + i);
        }
        base += sh.end[n - 1];
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kThreads) prefill_schedule_kernel(const PrefillParams p) {
    __shared__ Shared sh;
    static_assert(kStable >= kPreRounds * 160 && kThreads / 4 >= 160, "multiprocessors");
    if (threadIdx.x == 0) sm103::griddep_launch_dependents();
    sm103::griddep_wait();
    const PreWork work(p.metadata, p.max_blocks, p.sms);
    for (int i = threadIdx.x; i < kLengths; i += kThreads) sh.count[i] = 0;
    if (threadIdx.x == 0) sh.longest = sh.cuts = 0;
    __syncthreads();
    // most steps first: bucket 0 holds the longest
    auto bucket = [](int steps) { return kLengths - 1 - min(steps, kLengths - 1); };
    long long steps = 0;
    each_block(p, sh, true, [&](const PreBlock &x, long long i) {
        atomicAdd(&sh.count[bucket(x.steps)], 1);
        if (i < kStable) sh.bucket[i] = (short)bucket(x.steps);
        steps += x.steps;
    });
    int blocks;
    {
        const int here = sh.count[threadIdx.x];
        const int first = block_exclusive_scan<kThreads>(here, sh.scan, &blocks);
        sh.count[threadIdx.x] = first;
        blocks = (int)min((long long)blocks, (long long)p.max_blocks);
    }
    long long all;
    block_exclusive_scan<kThreads>(steps, sh.warp, &all);  // its barriers publish the places
    const bool stable = blocks <= kStable;
    each_block(p, sh, false, [&](const PreBlock &x, long long i) {
        const int mine = bucket(x.steps);
        int at;
        if (stable) {
            at = sh.count[mine];
            for (int k = 0; k < i; ++k) at += sh.bucket[k] == mine;
        } else {
            at = atomicAdd(&sh.count[mine], 1);
        }
        if (at < blocks) work.blocks[at] = x;
    });
    __syncthreads();
    // when the last CTA ends, in units
    const long long items = (long long)blocks * p.h_kv, units = (all + (long long)kFixed * blocks) * p.h_kv;
    const long long share = max((units + p.sms - 1) / p.sms, (long long)kLeastShare);
    bool line = false;
    if (items > 0 && pre_line(p.max_blocks, p.h_kv, p.sms)) {
        if ((int)threadIdx.x < p.sms) {
            long long mine = 0;
            int block, head;
            for (int round = 0; pre_round_item(round, threadIdx.x, p.sms, blocks, p.h_kv, p.head_chunk, block, head); ++round)
                mine += kFixed + work.blocks[block].steps;
            atomicMax(&sh.longest, (int)min(mine, 0x7fffffffll));
        }
        __syncthreads();
        line = (share + kFixed + kCombine) * 8 < (long long)sh.longest * 7;
    }
    if (threadIdx.x == 0) {
        work.header->blocks = blocks;
        work.header->line = line;
        work.header->cuts = 0;
    }
    if (!line) return;
    // where every CTA begins
    long long before = 0;
    for (int c0 = 0; c0 < blocks; c0 += kThreads) {
        const int b = c0 + threadIdx.x;
        const long long each = b < blocks ? (long long)(kFixed + work.blocks[b].steps) * p.h_kv : 0;
        long long total;
        const long long first = before + block_exclusive_scan<kThreads>(each, sh.warp, &total);
        if (b < blocks) sh.units[b] = first;
        before += total;
    }
    if (threadIdx.x == 0) sh.units[blocks] = before;
    __syncthreads();
    const int cta = threadIdx.x;
    if (cta <= p.sms) {
        PrePlace place = {blocks, 0, 0, 0};
        const long long unit = cta * share;
        if (cta < p.sms && unit < before) {
            int lo = 0, hi = blocks;  // units[lo] <= unit < units[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (sh.units[mid] <= unit) lo = mid;
                else hi = mid;
            }
            const long long each = (sh.units[lo + 1] - sh.units[lo]) / p.h_kv, in = unit - sh.units[lo];
            place.block = lo;
            place.head = (int)(in / each);
            place.step = (int)max(0ll, in - place.head * each - kFixed);
        }
        sh.place[cta] = work.places[cta] = place;
    }
    __syncthreads();
    // a cut item: the first CTA that begins inside it
    if (cta > 0 && cta < p.sms && sh.place[cta].step > 0) {
        const PrePlace here = sh.place[cta], left = sh.place[cta - 1];
        const bool same = left.block == here.block && left.head == here.head;
        if (!(same && left.step > 0)) {
            int n = 2;
            for (int next = cta + 1; next < p.sms && sh.place[next].block == here.block && sh.place[next].head == here.head && sh.place[next].step > 0; ++next) ++n;
            // the part before it is the last item of the CTA on its left, or all that one has
            const int at = atomicAdd(&sh.cuts, 1);
            work.cuts[at] = {here.block, here.head, 2 * (cta - 1) + (same ? 0 : 1), cta, n, {0, 0, 0}};
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) work.header->cuts = sh.cuts;
}

}  // namespace

cudaError_t launch_prefill_schedule(const PrefillParams &p, cudaStream_t stream) {
    return launch_after(prefill_schedule_kernel, dim3(1), dim3(kThreads), 0, stream, p);
}

}  // namespace mla
