// The work partition, as a routine of one CTA: see mla_schedule.cu for what it
// computes.  The scheduler kernel runs it over sequences or row tiles; the page
// selection runs it beside the selection, over the lengths it will leave.
#pragma once

#include "mla_internal.h"

namespace mla {

__device__ __forceinline__ int pages_of(int t) { return t <= 0 ? 0 : t / kPage + (t % kPage != 0); }

// Exclusive prefix sum over the block; *total receives the block total.
template <int kSchedThreads, typename T>
__device__ T block_exclusive_scan(T v, T *s_warp, T *total) {
    constexpr int kWarps = kSchedThreads / 32;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) s_warp[w] = x;
    __syncthreads();
    if (w == 0) {
        T y = lane < kWarps ? s_warp[lane] : T(0);
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const T z = __shfl_up_sync(0xffffffffu, y, off);
            if (lane >= off) y += z;
        }
        if (lane < kWarps) s_warp[lane] = y;
    }
    __syncthreads();
    const T base = w > 0 ? s_warp[w - 1] : T(0);
    *total = s_warp[kWarps - 1];
    __syncthreads();  // s_warp may be reused right after
    return base + x - v;
}

// One CTA.  Thread t owns the contiguous chunk of sequences
// [t * chunk, (t + 1) * chunk); a scan of the chunk costs gives every chunk's
// first unit, so a unit is located by a binary search over the chunks and a
// short walk inside one.
// `seqlens[i]` is the length of entry i.  kWhole: a batch of at most one entry
// per part may also get one part each, whole, where that is estimated no slower:
// the line's grid cuts entries whose lengths differ a little, and each cut costs a
// segment and the combine.
template <int kSchedThreads>
struct ScheduleShared {
    long long start[kSchedThreads + 1];  // first unit of every chunk; [kSchedThreads] = total
    long long warp64[kSchedThreads / 32];
    int warp32[kSchedThreads / 32];
    int pages[kSchedThreads];            // with one entry per thread: its pages, so that none is looked up again
};

template <bool kWhole, int kSchedThreads, typename Entries>
__device__ void schedule_body(ScheduleShared<kSchedThreads> &sh, const Entries &seqlens, int batch, int num_parts,
                              int fixed_cost, int combine_cost, int32_t *__restrict__ metadata,
                              int32_t *__restrict__ num_splits, unsigned int *status) {
    long long *s_start = sh.start, *s_warp64 = sh.warp64;
    int *s_warp32 = sh.warp32;
    const int chunk = (batch + kSchedThreads - 1) / kSchedThreads;
    const int i0 = min(threadIdx.x * chunk, batch), i1 = min(i0 + chunk, batch);
    long long cost = 0;
    bool bad = false;
    for (int i = i0; i < i1; ++i) {
        const int t = seqlens[i];
        bad |= t < 0;
        cost += pages_of(t) + fixed_cost;
        if (chunk == 1) sh.pages[i] = pages_of(t);
    }
    auto entry_pages = [&](int i) { return chunk == 1 ? sh.pages[i] : pages_of(seqlens[i]); };
    if (bad) atomicOr(status, MLA_DEVERR_SEQLEN);
    long long total;
    const long long first_unit = block_exclusive_scan<kSchedThreads>(cost, s_warp64, &total);
    s_start[threadIdx.x] = first_unit;
    if (threadIdx.x == 0) s_start[kSchedThreads] = total;

    // how many parts get work: all of them, or one per sequence when the
    // batch is smaller and that is estimated to finish sooner.  A candidate
    // with quota q costs q, plus F + C when a part would start strictly
    // inside some sequence's pages (a multiple of q in (S_b + F, S_{b+1})).
    // (quotients of a line below 2^31 units, which 64-bit division is five times slower at)
    const bool narrow = total < 0x7fffffffll - num_parts - fixed_cost;
    auto div = [&](long long a, long long b) {
        return narrow ? (long long)((unsigned)a / (unsigned)b) : a / b;
    };
    const long long q_all = (total + num_parts - 1) / num_parts;  // total >= batch * F > 0
    const long long q_seq = (total + batch - 1) / batch;
    bool cut_all = false, cut_seq = false;
    if (batch < num_parts) {
        long long u = first_unit;
        for (int i = i0; i < i1; ++i) {
            const int n = entry_pages(i);
            const long long next = u + n + fixed_cost;
            if (n > 0) {
                cut_all |= div(next - 1, q_all) > div(u + fixed_cost, q_all);
                cut_seq |= div(next - 1, q_seq) > div(u + fixed_cost, q_seq);
            }
            u = next;
        }
    }
    cut_all = __syncthreads_or(cut_all);
    cut_seq = __syncthreads_or(cut_seq);
    const long long est_all = q_all + (cut_all ? fixed_cost + combine_cost : 0);
    const long long est_seq = q_seq + (cut_seq ? fixed_cost + combine_cost : 0);
    const long long quota = (batch < num_parts && est_seq < est_all) ? q_seq : q_all;

    if constexpr (kWhole) {
        if (batch <= num_parts) {
            int longest = 0;
            for (int i = i0; i < i1; ++i) longest = max(longest, entry_pages(i));
            longest = __reduce_max_sync(0xffffffffu, longest);
            if ((threadIdx.x & 31) == 0) s_warp32[threadIdx.x >> 5] = longest;
            __syncthreads();
            for (int w = 0; w < kSchedThreads / 32; ++w) longest = max(longest, s_warp32[w]);
            if (longest + fixed_cost <= (est_seq < est_all ? est_seq : est_all)) {
                for (int p = threadIdx.x; p < num_parts; p += kSchedThreads) {
                    const int b = min(p, batch), next = min(p + 1, batch);
                    int32_t *row = metadata + (size_t)p * kMdInts;
                    row[0] = b;
                    row[2] = next;
                    row[1] = row[3] = row[4] = row[5] = row[6] = row[7] = 0;
                }
                for (int i = threadIdx.x; i <= batch; i += kSchedThreads) num_splits[i] = i;
                return;
            }
            __syncthreads();  // s_warp32 is used again
        }
    }

    // cursor of unit x: sequence b, page, and S_b
    auto cursor = [&](long long x, int &b, int &pg, long long &sb) {
        if (x >= total) {
            b = batch;
            pg = 0;
            sb = total;
            return;
        }
        int lo = 0, hi = kSchedThreads;  // s_start[lo] <= x < s_start[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_start[mid] <= x) lo = mid;
            else hi = mid;
        }
        long long u = s_start[lo];
        int i = lo * chunk;
        while (true) {
            const long long c = entry_pages(i) + fixed_cost;
            if (x < u + c) break;
            u += c;
            ++i;
        }
        b = i;
        sb = u;
        const long long off = x - u;
        pg = off <= fixed_cost ? 0 : (int)(off - fixed_cost);
    };

    for (int p = threadIdx.x; p < num_parts; p += kSchedThreads) {
        int b0, pg0, b1 = batch, pg1 = 0;
        long long s0, s1;
        cursor((long long)p * quota, b0, pg0, s0);
        if (p + 1 < num_parts) cursor((long long)(p + 1) * quota, b1, pg1, s1);
        // parts touching b0 before p: the one holding its page 0, then every
        // part that started inside its pages (the first at floor((S + F) / Q) + 1)
        const int split0 = pg0 > 0 ? (int)(p - div(s0 + fixed_cost, quota)) : 0;
        int32_t *row = metadata + (size_t)p * kMdInts;  // 4-byte alignment is all the caller promises
        row[0] = b0;
        row[1] = pg0;
        row[2] = b1;
        row[3] = pg1;
        row[4] = split0;
        row[5] = 0;
        row[6] = 0;
        row[7] = 0;
    }

    // parts touching sequence b: 1 + the part starts strictly inside its pages
    int segs = 0;
    {
        long long u = first_unit;
        for (int i = i0; i < i1; ++i) {
            const int n = entry_pages(i);
            const long long next = u + n + fixed_cost;
            segs += 1 + (n > 0 ? (int)(div(next - 1, quota) - div(u + fixed_cost, quota)) : 0);
            u = next;
        }
    }
    int all;
    int run = block_exclusive_scan<kSchedThreads>(segs, s_warp32, &all);
    {
        long long u = first_unit;
        for (int i = i0; i < i1; ++i) {
            const int n = entry_pages(i);
            const long long next = u + n + fixed_cost;
            run += 1 + (n > 0 ? (int)(div(next - 1, quota) - div(u + fixed_cost, quota)) : 0);
            num_splits[i + 1] = run;
            u = next;
        }
    }
    if (threadIdx.x == 0) num_splits[0] = 0;
}

}  // namespace mla
