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

#include <mutex>

#include "mla_internal.h"
#include "mla_page_walk.cuh"
#include "mla_sm103.cuh"

namespace mla {
namespace {

constexpr int kScoreThreads = 128;  // one page per thread
constexpr int kHeadChunk = 128;     // heads whose codes sit in shared memory together

// visible length of query token i of a sequence of length T
__device__ __forceinline__ int token_len(const SelectParams &p, int T, int i) {
    const int L = p.causal ? T - p.s_q + i + 1 : T;
    return L < 0 ? 0 : L;
}

__device__ __forceinline__ int pages_of(int len) { return len / kPage + (len % kPage != 0); }

// Scores of 128 pages per step: thread t holds the 144 words of page t's key
// and walks the heads' codes in shared memory (the same word for every thread).
template <int D>
__global__ void __launch_bounds__(kScoreThreads) page_scores_kernel(const SelectParams p) {
    constexpr int kWords = D / 4;
    extern __shared__ uint4 s_q4[];  // [kHeadChunk][D] codes
    __shared__ float s_unit[kHeadChunk];
    __shared__ int s_bad;
    __shared__ PageWalk<kScoreThreads>::Shared s_walk;
    sm103::griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    PageWalk<kScoreThreads> walk(s_walk, p.batch, blockIdx.x, gridDim.x);
    int b, unit;
    while (walk.next(
        [&](int i, int &first, int &count) {
            const int n = pages_of(clamp_len(p.seqlens[i], p.max_blocks, p.status));
            first = 0;
            count = n > p.topk ? p.s_q * ((n + kScoreThreads - 1) / kScoreThreads) : 0;
        },
        b, unit)) {
        const int T = min(p.seqlens[b], p.max_blocks * kPage);
        const int tiles = (pages_of(T) + kScoreThreads - 1) / kScoreThreads;
        const int tok = unit / tiles, tile = unit % tiles;
        const int n = pages_of(token_len(p, T, tok));
        const int page = tile * kScoreThreads + tid;
        float scale = 0.f;
        uint4 key[kWords / 4];
#pragma unroll
        for (int w = 0; w < kWords / 4; ++w) key[w] = make_uint4(0, 0, 0, 0);
        if (page < n) {
            const int blk = p.block_table[(size_t)b * p.max_blocks + page];
            if (blk < 0 || (int64_t)blk >= p.num_blocks) {
                atomicOr(p.status, MLA_DEVERR_BLOCK_ID);
            } else {
                scale = p.scales[blk];
                const uint4 *src = reinterpret_cast<const uint4 *>(p.keys + (size_t)blk * D);
#pragma unroll
                for (int w = 0; w < kWords / 4; ++w) key[w] = src[w];
            }
        }
        if (tid == 0) s_bad = 0;
        float best = -__uint_as_float(0x7f800000u);
        for (int h0 = 0; h0 < p.h_q; h0 += kHeadChunk) {
            const int heads = min(kHeadChunk, p.h_q - h0);
            __syncthreads();
            for (int h = warp; h < heads; h += kScoreThreads / 32) {
                const uint32_t *src = reinterpret_cast<const uint32_t *>(
                    p.q + (((size_t)b * p.s_q + tok) * p.h_q + h0 + h) * D);
                uint32_t x[D / 64], top = 0;
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    x[j] = src[lane + 32 * j];
                    top = max(top, max((x[j] << 16) & 0x7fffffffu, x[j] & 0x7fff0000u));
                }
                top = __reduce_max_sync(0xffffffffu, top);
                const bool finite = top < 0x7f800000u;
                const float u = top ? __uint_as_float(top) / 127.f : 1.f;
                char2 *dst = reinterpret_cast<char2 *>(reinterpret_cast<int8_t *>(s_q4) + (size_t)h * D);
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    char2 c = make_char2(0, 0);
                    if (finite)
                        c = make_char2((signed char)__float2int_rn(__uint_as_float(x[j] << 16) / u),
                                       (signed char)__float2int_rn(__uint_as_float(x[j] & 0xffff0000u) / u));
                    dst[lane + 32 * j] = c;
                }
                if (lane == 0) {
                    s_unit[h] = u;
                    if (!finite) s_bad = 1;
                }
            }
            __syncthreads();
            for (int h = 0; h < heads; ++h) {
                const uint4 *qh = s_q4 + h * (kWords / 4);
                int dot[4] = {0, 0, 0, 0};
#pragma unroll
                for (int w = 0; w < kWords / 4; ++w) {
                    const uint4 c = qh[w];
                    dot[0] = __dp4a((int)c.x, (int)key[w].x, dot[0]);
                    dot[1] = __dp4a((int)c.y, (int)key[w].y, dot[1]);
                    dot[2] = __dp4a((int)c.z, (int)key[w].z, dot[2]);
                    dot[3] = __dp4a((int)c.w, (int)key[w].w, dot[3]);
                }
                best = fmaxf(best, __fmul_rn(s_unit[h], (float)(dot[0] + dot[1] + dot[2] + dot[3])));
            }
        }
        if (page < n) {
            const float s = s_bad ? __uint_as_float(0x7fffffffu) : __fmul_rn(best, scale);
            p.scores[((size_t)b * p.s_q + tok) * p.max_blocks + page] = s;
        }
    }
}

// ---------------------------------------------------------------- selection
constexpr int kSelectThreads = 256;

// scores as unsigned integers of the same order; -0 as 0, NaN on top
__device__ __forceinline__ uint32_t rank_of(float s) {
    if (s != s) return 0xffffffffu;
    const uint32_t u = __float_as_uint(s + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// One CTA per query token: a radix search (8 bits a pass) for the rank of the
// last page taken by score, then one pass over the pages in order that writes
// the taken ones at their place.
__global__ void __launch_bounds__(kSelectThreads) select_pages_kernel(const SelectParams p) {
    __shared__ int s_hist[256];
    __shared__ int s_warp[kSelectThreads / 32];
    __shared__ int s_pick[2];
    sm103::griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t = blockIdx.x, b = t / p.s_q, tok = t % p.s_q;
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
    int done = 0, ties = 0;  // pages taken and ties seen before this round
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

constexpr int kMaxDevices = 64;
bool g_ready[kMaxDevices] = {};
std::mutex g_ready_mutex;

template <int D>
constexpr size_t score_smem() { return (size_t)kHeadChunk * D; }

}  // namespace

cudaError_t launch_select_pages(const SelectParams &p, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(g_ready_mutex);
        if (!g_ready[dev]) {
            e = cudaFuncSetAttribute(page_scores_kernel<kDqk>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)score_smem<kDqk>());
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(page_scores_kernel<kDv>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)score_smem<kDv>());
            if (e != cudaSuccess) return e;
            g_ready[dev] = true;
        }
    }
    if ((e = device_sm_count(&sms)) != cudaSuccess) return e;
    if (p.max_blocks > p.topk) {
        const long long most = (long long)p.batch * p.s_q * ((p.max_blocks + kScoreThreads - 1) / kScoreThreads);
        const unsigned grid = (unsigned)(most < 2LL * sms ? most : 2LL * sms);
        e = p.d == kDqk ? launch_after(page_scores_kernel<kDqk>, dim3(grid), dim3(kScoreThreads), score_smem<kDqk>(), stream, p)
                        : launch_after(page_scores_kernel<kDv>, dim3(grid), dim3(kScoreThreads), score_smem<kDv>(), stream, p);
        if (e != cudaSuccess) return e;
    }
    return launch_after(select_pages_kernel, dim3((unsigned)(p.batch * p.s_q)), dim3(kSelectThreads), 0, stream, p);
}

}  // namespace mla
