// Page selection: which topk pages of its sequence each query token attends to.
//
// Every cached page has a key (mla_page_keys.cu): int8 codes key[c] and a scale.
// Query token i of sequence b, head h:
//   s_h   = max_c |q[c]| / 127 (1 for a head of zeros),  qi[c] = rint(q[c] / s_h)
//   score(page) = scale_page * max_h (s_h * sum_c qi[c] key[c])
// Each integer dot product is at most 576 * 127^2 < 2^24, exact in int32 and in
// fp32 alike, and the maximum does not depend on its order, so a score has one
// value, whatever computes it; ties go to the lowest page.  A NaN score (a query
// or a page mean that is not finite) ranks above every number.
//
// Of the token's ceil(L / 64) visible pages (L: its causal length) the first
// `sink` and the last `local` are always taken, the rest by score; a token with
// at most topk pages takes them all.  The chosen pages, ascending, form a block
// table of their own: only the last visible page can be partial, and it is
// always chosen, so the dense decode runs on (sel_table, sel_lens) as it is.
#include <cuda_runtime.h>

#include "mla_internal.h"
#include "mla_page_walk.cuh"
#include "mla_schedule.cuh"
#include "mla_sm103.cuh"

namespace mla {
namespace {

// visible length of query token i of a sequence of length T
__device__ __forceinline__ int token_len(const SelectParams &p, int T, int i) {
    const int L = p.causal ? T - p.s_q + i + 1 : T;
    return L < 0 ? 0 : L;
}

// ---------------------------------------------------------------- selection
constexpr int kSelectThreads = 256;

// scores as unsigned integers of the same order; -0 as 0, NaN on top
__device__ __forceinline__ uint32_t rank_of(float s) {
    if (s != s) return 0xffffffffu;
    const uint32_t u = __float_as_uint(s + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Lengths that the selection leaves, as entries of the decode's work line (one
// per query token and row tile): they follow from the sequence lengths alone.
struct SelectedLengths {
    SelectParams p;
    int tiles;
    __device__ __forceinline__ int operator[](int e) const {
        const int t = e / tiles, b = t / p.s_q;
        const int T = min(max(p.seqlens[b], 0), p.max_blocks * kPage);
        const int L = token_len(p, T, t - b * p.s_q), n = pages_of(L), taken = min(n, p.topk);
        return taken ? (taken - 1) * kPage + (L - (n - 1) * kPage) : 0;
    }
};

// CTA 0 computes the decode's work partition meanwhile (mla_schedule.cu); then
// one CTA per query token: a radix search (8 bits a pass) for the rank of the
// last page taken by score, then one pass over the pages in order that writes
// the taken ones at their place.
__global__ void __launch_bounds__(kSelectThreads) select_pages_kernel(const SelectParams p) {
    __shared__ ScheduleShared<kSelectThreads> s_sched;
    __shared__ int s_hist[256];
    __shared__ int s_warp[kSelectThreads / 32];
    __shared__ int s_pick[2];
    sm103::griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // (letting the split-KV launch start its prologue meanwhile measured 4-5 us
    // slower on 64 tokens: its CTAs take the SMs before the selection's last ones)
    if (blockIdx.x == 0) {
        const int tiles = (p.h_q + MLA_TILE_ROWS - 1) / MLA_TILE_ROWS;
        schedule_body<true>(s_sched, SelectedLengths{p, tiles}, p.batch * p.s_q * tiles, p.num_parts, kFixedCost, kCombineCost,
                      p.metadata, p.num_splits, p.status);
        return;
    }
    const int t = blockIdx.x - 1, b = t / p.s_q, tok = t % p.s_q;
    const int L = token_len(p, clamp_len(p.seqlens[b], p.max_blocks, p.status), tok);
    const int n = pages_of(L);
    const int32_t *table = p.block_table + (size_t)b * p.max_blocks;
    const float *score = p.scores + (size_t)t * p.max_blocks;
    int32_t *sel = p.sel_table + (size_t)t * p.topk, *out = p.pages + (size_t)t * p.topk;
    const int taken = min(n, p.topk);
    if (tid == 0) p.sel_lens[t] = taken ? (taken - 1) * kPage + (L - (n - 1) * kPage) : 0;
    for (int i = taken + tid; i < p.topk; i += kSelectThreads) {
        sel[i] = 0;
        out[i] = -1;
    }
    if (n <= p.topk) {
        for (int i = tid; i < n; i += kSelectThreads) {
            sel[i] = table[i];
            out[i] = i;
        }
        return;
    }
    // pages [lo, hi) compete for `want` places
    const int lo = p.sink, hi = n - p.local;
    int want = p.topk - p.sink - p.local;
    uint32_t prefix = 0, mask = 0;
    for (int shift = 24; shift >= 0 && want > 0; shift -= 8) {
        s_hist[tid] = 0;
        __syncthreads();
        for (int i = lo + tid; i < hi; i += kSelectThreads) {
            const uint32_t r = rank_of(score[i]);
            if ((r & mask) == prefix) atomicAdd(&s_hist[(r >> shift) & 255], 1);
        }
        __syncthreads();
        // bin `tid` counted from the top: how many lie in higher bins
        const int mine = s_hist[255 - tid];
        int above = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, above, off);
            if (lane >= off) above += y;
        }
        if (lane == 31) s_warp[warp] = above;
        __syncthreads();
        for (int w = 0; w < warp; ++w) above += s_warp[w];
        above -= mine;
        if (above < want && above + mine >= want) {
            s_pick[0] = 255 - tid;
            s_pick[1] = want - above;
        }
        __syncthreads();
        prefix |= (uint32_t)s_pick[0] << shift;
        mask |= 255u << shift;
        want = s_pick[1];
        __syncthreads();
    }
    // `want` pages of rank `prefix` are taken, the first ones in order
    const bool by_score = p.topk > p.sink + p.local;
    int done = 0, ties = 0;  // pages taken and ties seen so far
    for (int i0 = 0; i0 < n; i0 += kSelectThreads) {
        const int i = i0 + tid;
        bool take = false, tie = false;
        if (i < n) {
            if (i < lo || i >= hi) {
                take = true;
            } else if (by_score) {
                const uint32_t r = rank_of(score[i]);
                take = r > prefix;
                tie = r == prefix;
            }
        }
        const uint32_t below = (1u << lane) - 1u;
        const uint32_t bt = __ballot_sync(0xffffffffu, tie);
        if (lane == 0) s_warp[warp] = __popc(bt);
        __syncthreads();
        int before = ties + __popc(bt & below);
        for (int w = 0; w < kSelectThreads / 32; ++w) {
            if (w < warp) before += s_warp[w];
            ties += s_warp[w];
        }
        if (tie && before < want) take = true;
        __syncthreads();
        const uint32_t bk = __ballot_sync(0xffffffffu, take);
        if (lane == 0) s_warp[warp] = __popc(bk);
        __syncthreads();
        int at = done + __popc(bk & below);
        for (int w = 0; w < kSelectThreads / 32; ++w) {
            if (w < warp) at += s_warp[w];
            done += s_warp[w];
        }
        if (take && at < p.topk) {
            sel[at] = table[i];
            out[at] = i;
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_select_pages(const SelectParams &p, cudaStream_t stream) {
    return launch_after(select_pages_kernel, dim3((unsigned)(p.batch * p.s_q) + 1), dim3(kSelectThreads), 0, stream, p);
}

}  // namespace mla
