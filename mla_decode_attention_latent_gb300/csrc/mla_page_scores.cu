// Scores of cached pages against query tokens, on the tensor cores.
//
//   score(page) = scale_page * max_h (u_h * <qi_h, key_page>)
// (mla_select_pages.cu has the definition).  The integer product runs as an
// f16 MMA: codes of -127 .. 127 are f16 values, every product and partial sum
// is an integer below 576 * 127^2 < 2^24, so the fp32 accumulator is exact and
// the result is the integer whatever the order.
//
// A work unit is 128 pages of one query token: D[page][head] = keys (A, 128 x d)
// times the token's quantised heads (B, up to 128 x d, kept in shared memory
// while consecutive units share the token).  Pages are the rows of D, so a
// thread reads the products of its page out of its TMEM lane and the maximum
// over the heads needs no exchange but between the two threads that share a
// page's heads.  The keys arrive as int8 (580 bytes a page: reading them is
// the bound for 128 heads) and are widened to f16 on their way into the
// swizzled operand: all of a unit's loads are in registers one unit ahead, 64 dims
// at a time go through four 16 KB stages that the MMAs free.  The heads' codes
// come from a small kernel in front.
// Work is cut into contiguous ranges of units, one per CTA.
#include <cuda_runtime.h>

#include <mutex>

#include "mla_internal.h"
#include "mla_page_walk.cuh"
#include "mla_schedule.cuh"
#include "mla_sm103.cuh"

namespace mla {
namespace {

using namespace sm103;

constexpr int kScoreThreads = 256;
constexpr int kTilePages = 128;               // rows of an MMA = TMEM lanes
constexpr int kHeadChunk = 128;               // heads of an MMA
constexpr int kStages = 4;
constexpr uint32_t kTileBytes = 128 * 128;    // 128 rows of 64 f16
constexpr uint32_t kTmemCols = 128;

template <int D>
struct ScoreSmem {
    static constexpr int kChunks = D / 64;
    static constexpr uint32_t q = 0;                                  // [chunk][head][64] f16, 128-byte swizzle
    static constexpr uint32_t a = q + kChunks * kTileBytes;           // [stage][page][64] f16
    static constexpr uint32_t unit = a + kStages * kTileBytes;        // [head] u_h
    static constexpr uint32_t best = unit + kHeadChunk * 4;           // [page] maximum of the upper heads
    static constexpr uint32_t bars = best + kTilePages * 4;           // stage barriers, done barrier
    static constexpr uint32_t tmem = bars + (kStages + 1) * 8;
    static constexpr uint32_t bad = tmem + 4;                         // the token holds a NaN or an infinity
    static constexpr uint32_t first = bad + 4;                        // the CTA's first unit: {sequence, unit in it}
    static constexpr uint32_t scan = (first + 8 + 15) & ~15u;         // [9] long long
    static constexpr uint32_t total = scan + 9 * 8;
};

// int8 codes (four per word) to f16 values: a byte b + 128 in the low bits of
// 1024 (0x6400) is the f16 number 1024 + 128 + b
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    w ^= 0x80808080u;
    lo = f16x2_sub(__byte_perm(w, 0x64646464u, 0x4140), 0x64806480u);
    hi = f16x2_sub(__byte_perm(w, 0x64646464u, 0x4342), 0x64806480u);
}

struct UnitAt {
    int b, tok, tile, tiles, n, T;
};

// Query heads to codes: u_h = max |q| / 127 (NaN for a head that is not finite,
// whose codes are 0), qi = rint(q / u_h).  One warp per head, so that the tokens'
// heads are quantised once, on all SMs, and not again by every CTA that scores
// pages for the token (which cost 7 us per token and CTA).
constexpr int kQuantWarps = 8;
template <int D>
__global__ void __launch_bounds__(kQuantWarps * 32) quantise_heads_kernel(const SelectParams p) {
    griddep_wait();
    // the scores may be launched now: what they read before they wait for this
    // kernel was complete when this kernel began
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * kQuantWarps + (threadIdx.x >> 5);
    if (row >= (long long)p.batch * p.s_q * p.h_q) return;
    constexpr int kPieces = D / 8;
    const uint4 *src = reinterpret_cast<const uint4 *>(p.q + row * D);
    uint4 x[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) x[j] = lane + 32 * j < kPieces ? src[lane + 32 * j] : make_uint4(0, 0, 0, 0);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max((w[e] << 16) & 0x7fffffffu, w[e] & 0x7fff0000u));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    const bool finite = top < 0x7f800000u;
    const float u = !finite ? __uint_as_float(0x7fffffffu) : top ? __uint_as_float(top) / 127.f : 1.f;
    uint2 *dst = reinterpret_cast<uint2 *>(p.q_codes + row * D);
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        if (lane + 32 * j >= kPieces) continue;
        const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
        uint32_t c[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            c[2 * e] = finite ? (uint32_t)__float2int_rn(__uint_as_float(w[e] << 16) / u) & 255u : 0u;
            c[2 * e + 1] = finite ? (uint32_t)__float2int_rn(__uint_as_float(w[e] & 0xffff0000u) / u) & 255u : 0u;
        }
        dst[lane + 32 * j] = make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24, c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
    }
    if (lane == 0) p.q_units[row] = u;
}

template <int D>
__global__ void __launch_bounds__(kScoreThreads, 1) page_scores_kernel(const SelectParams p) {
    using S = ScoreSmem<D>;
    constexpr int kChunks = S::kChunks;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t base_s = smem_u32(base);
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + S::bars);
    float *s_unit = reinterpret_cast<float *>(base + S::unit), *s_best = reinterpret_cast<float *>(base + S::best);
    volatile int *s_bad = reinterpret_cast<volatile int *>(base + S::bad);
    int *s_first = reinterpret_cast<int *>(base + S::first);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = tid & 127, half = tid >> 7;  // the thread's page, and its half of every 64 dims and of the heads

    if (tid == 0) {
        for (int i = 0; i <= kStages; ++i) mbar_init(bars + i, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(reinterpret_cast<uint32_t *>(base + S::tmem), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<uint32_t *>(base + S::tmem);
    // Up to the wait below, this reads only inputs of the call: the kernel
    // before it on the stream (quantise_heads_kernel) lets this one start only
    // after its own wait, when everything that wrote those inputs is complete.

    // sequence i's units; its pages and those of its tokens
    auto pages = [&](int i) { return pages_of(clamp_len(p.seqlens[i], p.max_blocks, p.status)); };
    auto units = [&](int i) -> long long {
        const int n = pages(i);
        return n > p.topk ? (long long)p.s_q * ((n + kTilePages - 1) / kTilePages) : 0;
    };
    // this CTA's range of all units, and where it starts
    const int chunk = (p.batch + kScoreThreads - 1) / kScoreThreads;
    const int i0 = min(tid * chunk, p.batch), i1 = min(i0 + chunk, p.batch);
    long long mine = 0, total;
    for (int i = i0; i < i1; ++i) mine += units(i);
    long long at = block_exclusive_scan<kScoreThreads>(mine, reinterpret_cast<long long *>(base + S::scan), &total);
    const long long share = (total + gridDim.x - 1) / gridDim.x;
    const long long u0 = share * blockIdx.x, u1 = min(u0 + share, total);
    if (u0 >= at && u0 < at + mine) {
        for (int i = i0; i < i1; ++i) {
            const long long c = units(i);
            if (u0 < at + c) {
                s_first[0] = i;
                s_first[1] = (int)(u0 - at);
                break;
            }
            at += c;
        }
    }
    __syncthreads();
    const int todo = u1 > u0 ? (int)(u1 - u0) : 0;

    auto load_seq = [&](UnitAt &u) {
        u.T = min(p.seqlens[u.b], p.max_blocks * kPage);
        u.tiles = (pages_of(u.T) + kTilePages - 1) / kTilePages;
    };
    auto set_token = [&](UnitAt &u) {
        const int L = p.causal ? u.T - p.s_q + u.tok + 1 : u.T;
        u.n = pages_of(L);
    };
    auto advance = [&](UnitAt &u) {
        if (++u.tile < u.tiles) return;
        u.tile = 0;
        if (++u.tok == p.s_q) {
            u.tok = 0;
            do ++u.b;
            while (u.b < p.batch && units(u.b) == 0);
            if (u.b >= p.batch) return;
            load_seq(u);
        }
        set_token(u);
    };
    // the thread's part of its page's key, 32 bytes of every 64 dims, and the scale
    uint4 key[kChunks][2];
    float scale = 0.f;
    auto load_keys = [&](const UnitAt &u) {
        const int page = u.tile * kTilePages + row;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) key[c][0] = key[c][1] = make_uint4(0, 0, 0, 0);
        scale = 0.f;
        if (page < u.n) {
            const int blk = p.block_table[(size_t)u.b * p.max_blocks + page];
            if (blk < 0 || (int64_t)blk >= p.num_blocks) {
                atomicOr(p.status, MLA_DEVERR_BLOCK_ID);
            } else {
                const uint4 *src = reinterpret_cast<const uint4 *>(p.keys + (size_t)blk * D) + 2 * half;
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    key[c][0] = __ldg(src + 4 * c);
                    key[c][1] = __ldg(src + 4 * c + 1);
                }
                scale = __ldg(p.scales + blk);
            }
        }
    };
    // codes of heads h0 .. h0 + heads - 1 of a token, widened into shared memory
    auto load_heads = [&](const UnitAt &u, int h0, int heads) {
        constexpr int kPieces = D / 16;  // 16-code pieces of a row
        constexpr int kItems = 128 * kPieces / kScoreThreads;
        const size_t first = ((size_t)u.b * p.s_q + u.tok) * p.h_q + h0;
        if (tid == 0 && h0 == 0) *s_bad = 0;
        uint4 x[kItems];
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int item = tid + i * kScoreThreads;
            x[i] = item < heads * kPieces ? reinterpret_cast<const uint4 *>(p.q_codes + first * D)[item] : make_uint4(0, 0, 0, 0);
        }
        const float un = tid < heads ? p.q_units[first + tid] : 1.f;
        __syncthreads();
        if (tid < heads) {
            s_unit[tid] = un;
            if (un != un) *s_bad = 1;
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int item = tid + i * kScoreThreads, h = item / kPieces, piece = 2 * (item - h * kPieces);
            uint32_t w[8];
            widen4(x[i].x, w[0], w[1]);
            widen4(x[i].y, w[2], w[3]);
            widen4(x[i].z, w[4], w[5]);
            widen4(x[i].w, w[6], w[7]);
            const uint32_t dst = base_s + S::q + (uint32_t)(piece >> 3) * kTileBytes + 128u * (uint32_t)h;
            sts128(dst + 16u * (uint32_t)((piece & 7) ^ (h & 7)), w[0], w[1], w[2], w[3]);
            sts128(dst + 16u * (uint32_t)(((piece & 7) + 1) ^ (h & 7)), w[4], w[5], w[6], w[7]);
        }
    };

    UnitAt u{};
    if (todo > 0) {
        u.b = s_first[0];
        load_seq(u);
        u.tok = s_first[1] / u.tiles;
        u.tile = s_first[1] - u.tok * u.tiles;
        set_token(u);
        load_keys(u);
    }
    griddep_wait();  // the heads' codes; writes to memory start behind it too
    int held_b = -1, held_tok = -1, held_h = -1;  // whose heads are in shared memory
    uint32_t fill = 0, done = 0;                  // chunks staged, products finished
    bool ok = true;
    for (int k = 0; k < todo && ok; ++k) {
        float best = -__uint_as_float(0x7f800000u);
        const float my_scale = scale;
        UnitAt next = u;
        if (k + 1 < todo) advance(next);
        for (int h0 = 0; h0 < p.h_q && ok; h0 += kHeadChunk) {
            const int heads = min(kHeadChunk, p.h_q - h0);
            if (held_b != u.b || held_tok != u.tok || held_h != h0) {
                load_heads(u, h0, heads);  // (the products of the heads before are finished)
                held_b = u.b;
                held_tok = u.tok;
                held_h = h0;
            }
            const uint32_t idesc = idesc_f16(kTilePages, (heads + 15) & ~15, false, false);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const uint32_t st = fill % kStages;
                if (ok) ok = mbar_wait(bars + st, ((fill / kStages) & 1) ^ 1, p.status);
                const uint32_t dst = base_s + S::a + st * kTileBytes + 128u * (uint32_t)row;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint4 x = key[c][j];
                    uint32_t w[8];
                    widen4(x.x, w[0], w[1]);
                    widen4(x.y, w[2], w[3]);
                    widen4(x.z, w[4], w[5]);
                    widen4(x.w, w[6], w[7]);
                    const uint32_t piece = 4u * (uint32_t)half + 2u * (uint32_t)j;
                    sts128(dst + 16u * (piece ^ (uint32_t)(row & 7)), w[0], w[1], w[2], w[3]);
                    sts128(dst + 16u * ((piece + 1) ^ (uint32_t)(row & 7)), w[4], w[5], w[6], w[7]);
                }
                fence_proxy_async_smem();
                ok = __syncthreads_and(ok) != 0;
                if (tid == 0 && ok) {
                    tc_fence_after();
                    const uint64_t ad = desc_sw128(base_s + S::a + st * kTileBytes, 16, 1024);
                    const uint64_t bd = desc_sw128(base_s + S::q + c * kTileBytes, 16, 1024);
#pragma unroll
                    for (int s = 0; s < 4; ++s) mma_ss(tmem, ad + 2 * s, bd + 2 * s, idesc, c > 0 || s > 0);
                    mma_commit(bars + st);
                    if (c == kChunks - 1) mma_commit(bars + kStages);
                }
                ++fill;
            }
            // the next unit's keys travel while the products finish and are read
            if (k + 1 < todo && h0 + kHeadChunk >= p.h_q) load_keys(next);
            if (ok) ok = mbar_wait(bars + kStages, done & 1, p.status);
            ok = __syncthreads_and(ok) != 0;
            if (!ok) break;
            ++done;
            tc_fence_after();
            const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
#pragma unroll
            for (int c0 = 0; c0 < 64; c0 += 32) {
                const int col = 64 * half + c0;
                if (col < heads) {
                    uint32_t v[32];
                    tmem_ld32(lanes + (uint32_t)col, v);
                    tmem_wait_ld();
                    if (col + 32 <= heads) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) best = fmaxf(best, __fmul_rn(s_unit[col + j], __uint_as_float(v[j])));
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (col + j < heads) best = fmaxf(best, __fmul_rn(s_unit[col + j], __uint_as_float(v[j])));
                    }
                }
            }
            tc_fence_before();
            __syncthreads();  // the accumulator and the heads may be replaced
            tc_fence_after();
        }
        if (!ok) break;
        if (half) s_best[row] = best;
        const bool bad = *s_bad != 0;
        __syncthreads();
        const int page = u.tile * kTilePages + row;
        if (!half && page < u.n) {
            best = fmaxf(best, s_best[row]);
            p.scores[((size_t)u.b * p.s_q + u.tok) * p.max_blocks + page] =
                bad ? __uint_as_float(0x7fffffffu) : __fmul_rn(best, my_scale);
        }
        u = next;
    }
    // the last products have finished (they were waited for); a wait that gave up
    // leaves at most what this CTA staged, which its own barriers still count
    if (!ok && tid == 0)
        for (uint32_t f = fill > (uint32_t)kStages ? fill - kStages : 0; f < fill; ++f)
            mbar_wait(bars + f % kStages, (f / kStages) & 1, p.status);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

constexpr int kMaxDevices = 64;
bool g_ready[kMaxDevices] = {};
std::mutex g_ready_mutex;

template <int D>
constexpr size_t score_smem() { return ScoreSmem<D>::total + 1024; }
static_assert(score_smem<kDqk>() <= 232448, "shared memory per CTA");

}  // namespace

cudaError_t launch_page_scores(const SelectParams &p, cudaStream_t stream) {
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
    const long long most = (long long)p.batch * p.s_q * ((p.max_blocks + kTilePages - 1) / kTilePages);
    const unsigned grid = (unsigned)(most < sms ? most : sms);
    const long long rows = (long long)p.batch * p.s_q * p.h_q;
    const dim3 qgrid((unsigned)((rows + kQuantWarps - 1) / kQuantWarps)), qblock(kQuantWarps * 32);
    e = p.d == kDqk ? launch_after(quantise_heads_kernel<kDqk>, qgrid, qblock, 0, stream, p)
                    : launch_after(quantise_heads_kernel<kDv>, qgrid, qblock, 0, stream, p);
    if (e != cudaSuccess) return e;
    return p.d == kDqk ? launch_after(page_scores_kernel<kDqk>, dim3(grid), dim3(kScoreThreads), score_smem<kDqk>(), stream, p)
                       : launch_after(page_scores_kernel<kDv>, dim3(grid), dim3(kScoreThreads), score_smem<kDv>(), stream, p);
}

}  // namespace mla
