// Pages of requests: block tables, positions and slots of a step's new rows, and
// the pages of finished requests back to the free list.
//
// Sequence b holds len_b rows in have_b = ceil(len_b / 64) pages and gets n_b =
// cu_rows[b + 1] - cu_rows[b] more, so it needs
//   need_b = ceil((len_b + n_b) / 64) - have_b
// new pages.  The free list is a stack of num_free pages; page k of the step is
// free_pages[num_free - 1 - k].  Sequences are taken in order: b is served when
// need_b = 0 or need_0 + .. + need_b <= num_free, and its pages are the ones
// behind the need of those before it.  (A sequence that needs pages and is served
// has only served ones before it among those that need any, so the pages of a step
// are the top of the stack without gaps.)  Row r of sequence b is at position
// p = len_b + r - cu_rows[b], in slot 64 * page + p % 64.
//
// Bounds that descend, leave the rows or begin before the end of an earlier sequence
// (of those with 0 <= lo <= hi <= num_rows) belong to nobody.  A chunk of sequences that has
// any takes, in place of such a bound, the largest end before it: bounds that ascend, in
// which every other sequence keeps its own rows and each row is some chunk's.
//
// Everything follows from prefix sums of the need, which every CTA computes for
// itself, so nothing is exchanged between CTAs: the page of a position is an
// entry of the table as it was (have_b and below) or an entry of the free list.
// One cluster of up to 16 CTAs runs the call: the words that are read by all and
// may be updated in place (the lengths, the count of free pages) are written
// behind a cluster barrier, so one launch does it and no workspace is kept.
// Bound by latency: a chunk's lengths and bounds, its scan, one page id per row.  64 sequences
// of one row each take 4.6 us, 48 prompts of up to 4096 rows (83,794) 8.5, and 12.4 on 8 CTAs.
#include <cuda_runtime.h>

#include <mutex>

#include "mla_internal.h"
#include "mla_schedule.cuh"
#include "mla_sm103.cuh"

namespace mla {
namespace {

constexpr int kThreads = 1024;  // also the sequences of a chunk
constexpr int kFewThreads = 128;  // of a call with few sequences and rows, whose barriers cost less
constexpr int kPortableCtas = 8, kMostCtas = 16;  // of a cluster
constexpr int kRun = 4;         // consecutive rows of a thread: one search, and mostly one page
constexpr int kRunsInFlight = 2;

template <int kThreads>
struct AssignShared {
    long long warp[kThreads / 32];
    int cu[kThreads + 1];     // ascending
    int len[kThreads];        // rows before the step; -1: not served
    long long first[kThreads];  // pages that earlier sequences need
    int taken;                // pages taken so far
};

// Bounds that ascend in sh.cu, the largest end before it in place of a senseless one; whether this thread's is one.
// Out of line: a call without any does not fetch it.
template <int kThreads>
__device__ __noinline__ bool ascending_bounds(AssignShared<kThreads> &sh, int n, int covered, int lo, int hi, int64_t num_rows) {
    const int tid = threadIdx.x;
    const bool bad = lo < 0 || hi < lo || hi > num_rows;
    int end = bad || tid >= n ? 0 : hi;  // the largest up to each sequence, by doubling distances
    for (int off = 1; off < kThreads; off <<= 1) {
        sh.len[tid] = end;
        __syncthreads();
        if (tid >= off) end = max(end, sh.len[tid - off]);
        __syncthreads();
    }
    sh.len[tid] = end;
    __syncthreads();
    const int earlier = tid ? max(covered, sh.len[tid - 1]) : covered;
    if (tid < n && (bad || lo < earlier)) sh.cu[tid] = earlier;
    if (tid == n - 1) sh.cu[n] = max(covered, end);
    return bad || lo < earlier;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) assign_pages_kernel(const AssignPagesParams p, bool wide) {
    __shared__ AssignShared<kThreads> sh;
    sm103::griddep_wait();
    const int tid = threadIdx.x;
    const int cta = blockIdx.x, ctas = gridDim.x;  // one cluster
    int left = *p.num_free;
    if (left < 0 || left > p.max_free) {
        if (tid == 0) atomicOr(p.status, MLA_DEVERR_SEQLEN);
        left = left < 0 ? 0 : (int)p.max_free;
    }
    const long long cap = (long long)p.max_blocks * kPage;
    long long before = 0;  // pages needed by the chunks so far
    int covered = 0;       // rows of the chunks so far
    if (tid == 0) sh.taken = 0;
    for (int c0 = 0; c0 < p.batch; c0 += kThreads) {
        const int n = min(kThreads, p.batch - c0), b = c0 + tid;
        int len = 0, count = 0, need = 0, lo = 0, hi = 0;
        bool bad = false;
        if (tid < n) {
            lo = p.cu_rows[b], hi = p.cu_rows[b + 1];
            sh.cu[tid] = lo;
            if (tid == n - 1) sh.cu[n] = hi;
            len = p.seqlens[b];
            bad = lo < 0 || hi < lo || hi > p.num_rows;
        }
        // (a sequence's need is below 2^25; a senseless bound counts above all of them)
        const bool odd = bad || (tid == 0 && lo < covered);
        auto need_pages = [&] {
            count = bad ? 0 : hi - lo;
            bad = bad || len < 0 || (long long)len + count > cap;
            need = bad ? 0 : pages_of(len + count) - pages_of(len);
            return (long long)need;
        };
        long long total, earlier_need = block_exclusive_scan<kThreads>(need_pages() + (odd ? 1ll << 40 : 0), sh.warp, &total);
        if (total >> 40) {
            bad = ascending_bounds(sh, n, covered, lo, hi, p.num_rows) || tid >= n;
            earlier_need = block_exclusive_scan<kThreads>(need_pages(), sh.warp, &total);
        }
        const long long first = before + earlier_need;
        if (tid < n && bad) atomicOr(p.status, MLA_DEVERR_SEQLEN);
        const bool served = tid < n && !bad && (need == 0 || first + need <= left);
        if (tid < n) {
            sh.len[tid] = served ? len : -1;
            sh.first[tid] = first;
        }
        // those that are served of those that need any are the first ones: the last one's end
        if (served && need > 0) atomicMax(&sh.taken, (int)(first + need));
        __syncthreads();
        // every CTA has the chunk's lengths before one of them changes them
        sm103::cluster_arrive();
        // new table entries: a thread per page of the chunk's need
        const long long most = min(before + total, (long long)left);
        for (long long k = before + (long long)cta * kThreads + tid; k < most; k += (long long)ctas * kThreads) {
            int i = 0, hi = n;  // the last i with first[i] <= k: the one that needs page k
            while (hi - i > 1) {
                const int mid = (i + hi) >> 1;
                if (sh.first[mid] <= k) i = mid;
                else hi = mid;
            }
            if (sh.len[i] >= 0) p.block_table[(size_t)(c0 + i) * p.max_blocks + pages_of(sh.len[i]) + (k - sh.first[i])] = p.free_pages[left - 1 - k];
        }
        // the chunk's rows (and those before the first sequence and behind the last)
        const long long r0 = covered, r1 = c0 + n == p.batch ? p.num_rows : sh.cu[n];
        covered = sh.cu[n];
        const long long stride = (long long)ctas * kThreads * kRun;
        for (long long r = (r0 & ~(long long)(kRun - 1)) + ((long long)cta * kThreads + tid) * kRun; r < r1; r += stride * kRunsInFlight) {
            int pos[kRunsInFlight][kRun], page[kRunsInFlight][kRun];
            bool live[kRunsInFlight][kRun];
#pragma unroll
            for (int k = 0; k < kRunsInFlight; ++k) {
                const long long row0 = r + k * stride;
                int i = 0, hi = n;  // the last i with cu[i] <= the run's first row
                while (hi - i > 1) {
                    const int mid = (i + hi) >> 1;
                    if (sh.cu[mid] <= row0) i = mid;
                    else hi = mid;
                }
                const int32_t *from[kRun];
#pragma unroll
                for (int e = 0; e < kRun; ++e) {
                    const long long row = row0 + e;
                    while (i + 1 < n && sh.cu[i + 1] <= row) ++i;
                    const int l = sh.len[i];
                    live[k][e] = row >= r0 && row < r1 && l >= 0 && row >= sh.cu[i] && row < sh.cu[i + 1];
                    pos[k][e] = live[k][e] ? l + (int)(row - sh.cu[i]) : 0;
                    const int c = pos[k][e] / kPage, have = pages_of(l);
                    from[e] = !live[k][e] ? p.num_free  // (any word that can be read)
                              : c < have ? p.block_table + (size_t)(c0 + i) * p.max_blocks + c : p.free_pages + (left - 1 - (sh.first[i] + c - have));
                }
#pragma unroll
                for (int e = 0; e < kRun; ++e) page[k][e] = *from[e];  // together under way
            }
#pragma unroll
            for (int k = 0; k < kRunsInFlight; ++k) {
                const long long row0 = r + k * stride;
                if (row0 >= r1) continue;
                int64_t slot[kRun];
#pragma unroll
                for (int e = 0; e < kRun; ++e) {
                    if (live[k][e] && page[k][e] < 0) atomicOr(p.status, MLA_DEVERR_BLOCK_ID);
                    slot[e] = live[k][e] && page[k][e] >= 0 ? (int64_t)page[k][e] * kPage + pos[k][e] % kPage : -1;
                }
                if (wide && row0 >= r0 && row0 + kRun <= r1) {
                    if (p.positions) *reinterpret_cast<int4 *>(p.positions + row0) = make_int4(pos[k][0], pos[k][1], pos[k][2], pos[k][3]);
                    if (p.slots) {
                        longlong2 *dst = reinterpret_cast<longlong2 *>(p.slots + row0);
                        dst[0] = make_longlong2(slot[0], slot[1]);
                        dst[1] = make_longlong2(slot[2], slot[3]);
                    }
                    continue;
                }
#pragma unroll
                for (int e = 0; e < kRun; ++e) {
                    const long long row = row0 + e;
                    if (row < r0 || row >= r1) continue;
                    if (p.positions) p.positions[row] = pos[k][e];
                    if (p.slots) p.slots[row] = slot[e];
                }
            }
        }
        sm103::cluster_wait();
        if (cta == 0 && tid < n) p.new_seqlens[b] = served ? len + count : (len < 0 ? 0 : len);
        before += total;
        __syncthreads();  // the chunk in shared memory is used up
    }
    // behind the last chunk's barrier every CTA has read the count
    if (cta == 0 && tid == 0) *p.num_free_out = left - sh.taken;
}

// Pages of finished sequences onto the stack, in the order of the sequences and
// of their pages; one CTA, a warp per sequence.  An entry that is no page is reported and not pushed.
// Bound by latency: 64 sequences of which none has finished take 2.4 us, of which 6 of up to 64
// pages have 3.5, and 64 of them 5.2; of up to 2048 pages (66,985 in all) 64.
struct ReleaseShared {
    long long warp[kThreads / 32];
    int count[kThreads];
    long long first[kThreads];
};

__global__ void __launch_bounds__(kThreads) release_pages_kernel(const ReleasePagesParams p) {
    __shared__ ReleaseShared sh;
    sm103::griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int left = *p.num_free;
    if (left < 0 || left > p.max_free) {
        if (tid == 0) atomicOr(p.status, MLA_DEVERR_SEQLEN);
        left = left < 0 ? 0 : (int)p.max_free;
    }
    long long top = left;
    for (int c0 = 0; c0 < p.batch; c0 += kThreads) {
        const int n = min(kThreads, p.batch - c0);
        // entries to push of each sequence
        for (int i = warp; i < n; i += kThreads / 32) {
            const int b = c0 + i;
            int count = 0;
            if (p.finished[b] != 0) {
                int len = p.seqlens[b];
                const long long cap = (long long)p.max_blocks * kPage;
                if (len < 0 || len > cap) {
                    if (lane == 0) atomicOr(p.status, MLA_DEVERR_SEQLEN);
                    len = len < 0 ? 0 : (int)cap;
                }
                const int pages = pages_of(len);
                for (int c = 0; c < pages; c += 32) {
                    const bool in = c + lane < pages;
                    const int id = in ? p.block_table[(size_t)b * p.max_blocks + c + lane] : 0;
                    const bool good = in && id >= 0 && id < p.num_blocks;
                    if (in && !good) atomicOr(p.status, MLA_DEVERR_BLOCK_ID);
                    count += __popc(__ballot_sync(0xffffffffu, good));
                }
            }
            if (lane == 0) sh.count[i] = count;
        }
        __syncthreads();
        long long total;
        const long long first = block_exclusive_scan<kThreads>((long long)(tid < n ? sh.count[tid] : 0), sh.warp, &total);
        if (tid < n) sh.first[tid] = top + first;
        __syncthreads();
        for (int i = warp; i < n; i += kThreads / 32) {
            const int b = c0 + i;
            if (p.finished[b] == 0) continue;
            const int len = p.seqlens[b];
            const long long cap = (long long)p.max_blocks * kPage;
            const int pages = pages_of(len < 0 ? 0 : len > cap ? (int)cap : len);
            long long at = sh.first[i];
            for (int c = 0; c < pages; c += 32) {
                const bool in = c + lane < pages;
                int32_t *entry = p.block_table + (size_t)b * p.max_blocks + c + lane;
                const int id = in ? *entry : 0;
                const bool good = in && id >= 0 && id < p.num_blocks;
                const unsigned mask = __ballot_sync(0xffffffffu, good);
                const long long to = at + __popc(mask & ((1u << lane) - 1u));
                if (good) {
                    if (to < p.max_free) p.free_pages[to] = id;
                    else atomicOr(p.status, MLA_DEVERR_SEQLEN);
                }
                if (in) *entry = -1;
                at += __popc(mask);
            }
            __syncwarp();
            if (lane == 0) p.seqlens[b] = 0;
        }
        top += total;
        __syncthreads();
    }
    if (tid == 0) *p.num_free = (int)min(top, (long long)p.max_free);
}

}  // namespace

// CTAs of the cluster of a call with many rows: 16 where the device takes such a cluster, or 8, which all do
static cudaError_t many_ctas(int *ctas) {
    constexpr int kMaxDevices = 64;
    static std::mutex mutex;
    static int known[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mutex);
    if (!known[dev]) {
        e = cudaFuncSetAttribute(assign_pages_kernel<kThreads>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kMostCtas);
        cfg.blockDim = dim3(kThreads);
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = kMostCtas;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        e = cudaOccupancyMaxActiveClusters(&clusters, assign_pages_kernel<kThreads>, &cfg);
        if (e != cudaSuccess) return e;
        known[dev] = clusters > 0 ? kMostCtas : kPortableCtas;
    }
    *ctas = known[dev];
    return cudaSuccess;
}

cudaError_t launch_assign_pages(const AssignPagesParams &p, cudaStream_t stream) {
    const bool few = p.num_rows <= 4 * kFewThreads * kRun && p.batch <= kFewThreads;
    int ctas = few || p.num_rows <= kThreads * kRun ? 1 : kPortableCtas;
    if (p.num_rows > kPortableCtas * kThreads * kRun) {
        const cudaError_t e = many_ctas(&ctas);
        if (e != cudaSuccess) return e;
    }
    // whole runs are stored at once where the outputs allow it
    const bool wide = ((reinterpret_cast<uintptr_t>(p.positions) | reinterpret_cast<uintptr_t>(p.slots)) & 15) == 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(few ? kFewThreads : kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return few ? cudaLaunchKernelEx(&cfg, assign_pages_kernel<kFewThreads>, p, wide) : cudaLaunchKernelEx(&cfg, assign_pages_kernel<kThreads>, p, wide);
}

cudaError_t launch_release_pages(const ReleasePagesParams &p, cudaStream_t stream) {
    return launch_after(release_pages_kernel, dim3(1), dim3(kThreads), 0, stream, p);
}

}  // namespace mla
