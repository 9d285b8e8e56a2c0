// Walk of a ragged list of pages by a fixed grid.
//
// Sequence i contributes `count` pages from page `first` on (both computed on
// the device from the lengths, which the host does not know).  All pages of
// all sequences form one list; CTA `cta` takes entries cta, cta + stride, ...
// Sequences are taken in chunks of kThreads: a prefix sum of the chunk's counts
// in shared memory, then a binary search per entry.  Every thread of the CTA
// calls next() together and gets the same answer; what the callers do between
// two calls may run ahead of one another only up to the barriers inside.
#pragma once

#include <stdint.h>

#include "mla_internal.h"

namespace mla {

// length of a sequence on the device: negative ones count as 0 and ones past
// the table as its capacity, and both set a status bit
__device__ __forceinline__ int clamp_len(int t, int max_blocks, unsigned int *status) {
    const int cap = max_blocks * kPage;
    if (t < 0 || t > cap) {
        atomicOr(status, MLA_DEVERR_SEQLEN);
        return t < 0 ? 0 : cap;
    }
    return t;
}

template <int kThreads>
class PageWalk {
public:
    struct Shared {
        long long end[kThreads];  // inclusive prefix sums of the chunk's counts
        int first[kThreads];
        long long warp[kThreads / 32];
    };

    __device__ PageWalk(Shared &s, int batch, long long cta, long long stride)
        : s_(s), batch_(batch), at_(cta), stride_(stride) {}

    // The next entry of this CTA: sequence b, page pg; false when there is none.
    template <typename Range>
    __device__ bool next(Range range, int &b, int &pg) {
        while (true) {
            if (chunk_ >= 0) {
                const int n = min(kThreads, batch_ - chunk_);
                if (at_ < base_ + s_.end[n - 1]) {
                    int lo = 0, hi = n - 1;  // the first i with at_ < base_ + end[i]
                    while (lo < hi) {
                        const int mid = (lo + hi) >> 1;
                        if (at_ < base_ + s_.end[mid]) hi = mid;
                        else lo = mid + 1;
                    }
                    b = chunk_ + lo;
                    pg = s_.first[lo] + (int)(at_ - base_ - (lo ? s_.end[lo - 1] : 0));
                    at_ += stride_;
                    __syncthreads();  // the caller's shared memory of the entry before is free
                    return true;
                }
                base_ += s_.end[n - 1];
                __syncthreads();  // every thread has read the chunk
                chunk_ += kThreads;
            } else {
                chunk_ = 0;
            }
            if (chunk_ >= batch_) return false;
            const int i = chunk_ + (int)threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
            int first = 0, count = 0;
            if (i < batch_) range(i, first, count);
            long long x = count;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, x, off);
                if (lane >= off) x += y;
            }
            if (lane == 31) s_.warp[warp] = x;
            __syncthreads();
            for (int w = 0; w < warp; ++w) x += s_.warp[w];
            s_.end[threadIdx.x] = x;
            s_.first[threadIdx.x] = first;
            __syncthreads();
        }
    }

private:
    Shared &s_;
    int batch_;
    long long at_, stride_, base_ = 0;
    int chunk_ = -1;
};

}  // namespace mla
