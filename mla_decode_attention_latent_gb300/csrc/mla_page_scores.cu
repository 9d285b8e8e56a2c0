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

constexpr int kScoreThreads = 256;            // 8 warps that stage keys and read products
constexpr int kCtaThreads = kScoreThreads + 32;  // and one that issues the MMAs
constexpr int kTilePages = 128;               // rows of an MMA = TMEM lanes
constexpr int kHeadChunk = 128;               // heads of an MMA
constexpr int kStages = 4;
constexpr uint32_t kTileBytes = 128 * 128;    // 128 rows of 64 f16
constexpr uint32_t kTmemCols = 256;           // two accumulators

template <int D>
struct ScoreSmem {
    static constexpr int kChunks = D / 64;
    static constexpr uint32_t q = 0;                                  // [chunk][head][64] f16, 128-byte swizzle
    static constexpr uint32_t a = q + kChunks * kTileBytes;           // [stage][page][64] f16
    static constexpr uint32_t unit = a + kStages * kTileBytes;        // [head] u_h
    static constexpr uint32_t best = unit + kHeadChunk * 4;           // [page] maximum of the upper heads
    static constexpr uint32_t bars = best + kTilePages * 4;           // B_* below
    static constexpr uint32_t tmem = bars + (2 * kStages + 4) * 8;
    static constexpr uint32_t bad = tmem + 4;                         // the token holds a NaN or an infinity
    static constexpr uint32_t first = bad + 4;                        // the CTA's first unit: {sequence, unit in it}
    static constexpr uint32_t scan = (first + 8 + 15) & ~15u;         // [9] long long
    static constexpr uint32_t total = scan + (kCtaThreads / 32) * 8;
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

// barriers: stage staged (256 arrivals) / free (commit), accumulator finished
// (commit) / read (256 arrivals)
enum { B_FULL = 0, B_EMPTY = kStages, B_DONE = 2 * kStages, B_READ = 2 * kStages + 2, B_ALL = 2 * kStages + 4 };

// The MMA issuer (one thread): for every job, the chunks in order.  A wait
// that gave up leaves `ok` false; the loops go on without waiting or issuing, so
// that every thread reaches the kernel's end.
template <int D>
__device__ void score_issuer(const SelectParams &p, uint32_t base_s, uint64_t *bars, uint32_t tmem, long long jobs) {
    using S = ScoreSmem<D>;
    uint32_t fill = 0;
    bool ok = true;
    const int passes = (p.h_q + kHeadChunk - 1) / kHeadChunk;
    for (long long j = 0; j < jobs; ++j) {
        const int heads = min(kHeadChunk, p.h_q - (int)(j % passes) * kHeadChunk);
        const uint32_t idesc = idesc_f16(kTilePages, (heads + 15) & ~15, false, false);
        const uint32_t buf = (uint32_t)(j & 1), d = tmem + buf * 128;
        if (ok) ok = mbar_wait(bars + B_READ + buf, (uint32_t)((j >> 1) & 1) ^ 1u, p.status);
        tc_fence_after();
        for (int c = 0; c < S::kChunks; ++c, ++fill) {
            const uint32_t st = fill % kStages;
            if (ok) ok = mbar_wait(bars + B_FULL + st, (fill / kStages) & 1, p.status);
            if (!ok) continue;
            const uint64_t ad = desc_sw128(base_s + S::a + st * kTileBytes, 16, 1024);
            const uint64_t bd = desc_sw128(base_s + S::q + c * kTileBytes, 16, 1024);
#pragma unroll
            for (int s = 0; s < 4; ++s) mma_ss(d, ad + 2 * s, bd + 2 * s, idesc, c > 0 || s > 0);
            mma_commit(bars + B_EMPTY + st);
            if (c == S::kChunks - 1) mma_commit(bars + B_DONE + buf);
        }
    }
    // everything issued has finished before the tensor memory goes (after a wait
    // that gave up, long ago: MMAs take microseconds, the limit is seconds)
    if (ok && jobs > 0) mbar_wait(bars + B_DONE + (uint32_t)((jobs - 1) & 1), (uint32_t)(((jobs - 1) >> 1) & 1), p.status);
}

template <int D>
__global__ void __launch_bounds__(kCtaThreads, 1) page_scores_kernel(const SelectParams p) {
    using S = ScoreSmem<D>;
    constexpr int kChunks = S::kChunks;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t base_s = smem_u32(base);
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + S::bars);
    float *s_unit = reinterpret_cast<float *>(base + S::unit), *s_best = reinterpret_cast<float *>(base + S::best);
    volatile int *s_bad = reinterpret_cast<volatile int *>(base + S::bad);
    int *s_first = reinterpret_cast<int *>(base + S::first);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int row = tid & 127, half = (tid >> 7) & 1;  // the thread's page, and its half of the heads

    if (tid == 0) {
        for (int i = 0; i < B_ALL; ++i)
            mbar_init(bars + i, (i >= B_EMPTY && i < B_READ) ? 1 : kScoreThreads);
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
    const int chunk = (p.batch + kCtaThreads - 1) / kCtaThreads;
    const int i0 = min(tid * chunk, p.batch), i1 = min(i0 + chunk, p.batch);
    long long mine = 0, total;
    for (int i = i0; i < i1; ++i) mine += units(i);
    long long at = block_exclusive_scan<kCtaThreads>(mine, reinterpret_cast<long long *>(base + S::scan), &total);
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
    // The thread's part of the unit's keys: of every 64 dims, 16 bytes of rows
    // srow and srow + 64 (four neighbouring lanes read 64 contiguous bytes); and
    // the scale of its own page.  A page that is not there reads block 0's key
    // (its score goes nowhere, or, for a bad block id, is any number).  The block
    // ids are looked up a unit ahead of the keys, and the keys a unit ahead of
    // their use, so that no load waits for another.
    const int srow = (tid & 255) >> 2, quarter = tid & 3;
    uint4 key[kChunks][2];
    float scale = 0.f;
    struct Blocks {
        int s0, s1, own;
    };
    auto block_of = [&](const UnitAt &u, int r) {
        const int page = u.tile * kTilePages + r;
        return page < u.n ? __ldg(p.block_table + (size_t)u.b * p.max_blocks + page) : 0;
    };
    auto look_up = [&](const UnitAt &u) { return Blocks{block_of(u, srow), block_of(u, srow + 64), block_of(u, row)}; };
    auto safe = [&](int blk) { return blk < 0 || (int64_t)blk >= p.num_blocks ? 0 : blk; };
    auto key_row = [&](int blk) { return reinterpret_cast<const uint4 *>(p.keys + (size_t)safe(blk) * D) + quarter; };
    auto load_scale = [&](int own) {
        if (own < 0 || (int64_t)own >= p.num_blocks) atomicOr(p.status, MLA_DEVERR_BLOCK_ID);
        scale = __ldg(p.scales + safe(own));
    };
    // codes of heads h0 .. h0 + heads - 1 of a token, widened into shared memory
    auto load_heads = [&](const UnitAt &u, int h0, int heads) {
        constexpr int kPieces = D / 16;  // 16-code pieces of a row
        constexpr int kItems = 128 * kPieces / kScoreThreads, kBatch = kItems / 2;  // loads in flight: half of them
        static_assert(kItems % 2 == 0, "two batches");
        const size_t first = ((size_t)u.b * p.s_q + u.tok) * p.h_q + h0;
        if (tid == 0 && h0 == 0) *s_bad = 0;
        const float un = tid < heads ? p.q_units[first + tid] : 1.f;
        named_bar_sync(1, kScoreThreads);  // s_bad is cleared, and what the heads before left is read
        if (tid < kHeadChunk) {
            // a product with NaN never is the maximum: the columns behind the heads drop out
            s_unit[tid] = tid < heads ? un : __uint_as_float(0x7fffffffu);
            if (un != un) *s_bad = 1;
        }
#pragma unroll 1
        for (int i0 = 0; i0 < kItems; i0 += kBatch) {
            uint4 x[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int item = tid + (i0 + i) * kScoreThreads;
                x[i] = item < heads * kPieces ? reinterpret_cast<const uint4 *>(p.q_codes + first * D)[item]
                                              : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int item = tid + (i0 + i) * kScoreThreads, h = item / kPieces, piece = 2 * (item - h * kPieces);
                uint32_t w[8];
                widen4(x[i].x, w[0], w[1]);
                widen4(x[i].y, w[2], w[3]);
                widen4(x[i].z, w[4], w[5]);
                widen4(x[i].w, w[6], w[7]);
                const uint32_t dst = base_s + S::q + (uint32_t)(piece >> 3) * kTileBytes + 128u * (uint32_t)h;
                sts128(dst + 16u * (uint32_t)((piece & 7) ^ (h & 7)), w[0], w[1], w[2], w[3]);
                sts128(dst + 16u * (uint32_t)(((piece & 7) + 1) ^ (h & 7)), w[4], w[5], w[6], w[7]);
            }
        }
    };

    const int passes = (p.h_q + kHeadChunk - 1) / kHeadChunk;  // jobs of a unit: its heads, 128 at a time
    if (warp == kScoreThreads / 32) {
        if (elect_one_lane()) score_issuer<D>(p, base_s, bars, tmem, (long long)todo * passes);
    } else {
        UnitAt u{};
        if (todo > 0) {
            u.b = s_first[0];
            load_seq(u);
            u.tok = s_first[1] / u.tiles;
            u.tile = s_first[1] - u.tok * u.tiles;
            set_token(u);
            const Blocks b = look_up(u);
            const uint4 *s0 = key_row(b.s0), *s1 = key_row(b.s1);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                key[c][0] = __ldg(s0 + 4 * c);
                key[c][1] = __ldg(s1 + 4 * c);
            }
            load_scale(b.own);
        }
        // the unit after this one, and its block ids
        UnitAt next = u;
        Blocks next_blocks{0, 0, 0};
        if (todo > 1) {
            advance(next);
            next_blocks = look_up(next);
        }
        griddep_wait();  // the heads' codes; the scores are written behind it too
        bool ok = true;
        float best = -__uint_as_float(0x7f800000u);
        // The products of job j are read after job j + 1 is staged, or before the
        // heads are replaced: `late` is what that needs.
        struct Late {
            int heads = 0;        // 0: nothing to read
            bool last = false;    // the unit's last heads: its scores are complete
            long long job = 0;
            float scale = 0.f;
            float *out = nullptr;
        } late;
        auto read_products = [&] {
            if (late.heads == 0) return;
            const uint32_t buf = (uint32_t)(late.job & 1);
            if (ok) ok = mbar_wait(bars + B_DONE + buf, (uint32_t)((late.job >> 1) & 1), p.status);
            tc_fence_after();
            const uint32_t lanes = tmem + buf * 128 + ((uint32_t)(32 * (warp & 3)) << 16);
#pragma unroll
            for (int c0 = 0; c0 < 64; c0 += 32) {
                const int col = 64 * half + c0;
                if (col < late.heads) {
                    uint32_t v[32];
                    tmem_ld32(lanes + (uint32_t)col, v);
                    tmem_wait_ld();
                    const uint32_t un = base_s + S::unit + 4u * (uint32_t)col;
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const uint4 w = lds128(un + 4 * j);
                        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            best = fmaxf(best, __fmul_rn(__uint_as_float(ws[e]), __uint_as_float(v[j + e])));
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(bars + B_READ + buf);
            if (late.last) {
                if (half) s_best[row] = best;
                const bool bad = *s_bad != 0;
                named_bar_sync(1, kScoreThreads);
                if (!half && late.out) {
                    best = fmaxf(best, s_best[row]);
                    *late.out = bad ? __uint_as_float(0x7fffffffu) : __fmul_rn(best, late.scale);
                }
                named_bar_sync(1, kScoreThreads);  // s_best may be written again
                best = -__uint_as_float(0x7f800000u);
            }
            late.heads = 0;
        };
        int held_b = -1, held_tok = -1, held_h = -1;  // whose heads are in shared memory
        uint32_t fill = 0;
        long long job = 0;
        for (int k = 0; k < todo; ++k) {
            const int page = u.tile * kTilePages + row;
            const float my_scale = scale;
            UnitAt after = next;
            Blocks after_blocks{0, 0, 0};
            for (int h0 = 0; h0 < p.h_q; h0 += kHeadChunk, ++job) {
                const int heads = min(kHeadChunk, p.h_q - h0);
                if (held_b != u.b || held_tok != u.tok || held_h != h0) {
                    read_products();  // waits for the products that use the heads in place
                    load_heads(u, h0, heads);
                    held_b = u.b;
                    held_tok = u.tok;
                    held_h = h0;
                }
                // with a unit's last heads the next unit's keys replace its own piece by
                // piece: their loads spread over the staging (all at once behind it
                // they queue up: 36.5 us for 64 tokens of 1024 pages and 128 heads, now MEASURED)
                const bool ahead = h0 + kHeadChunk >= p.h_q && k + 1 < todo;
                const uint4 *s0 = key_row(next_blocks.s0), *s1 = key_row(next_blocks.s1);
#pragma unroll
                for (int c = 0; c < kChunks; ++c, ++fill) {
                    const uint32_t st = fill % kStages;
                    if (ok) ok = mbar_wait(bars + B_EMPTY + st, ((fill / kStages) & 1) ^ 1, p.status);
                    const uint32_t dst = base_s + S::a + st * kTileBytes + 128u * (uint32_t)srow;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint4 x = key[c][j];
                        uint32_t w[8];
                        widen4(x.x, w[0], w[1]);
                        widen4(x.y, w[2], w[3]);
                        widen4(x.z, w[4], w[5]);
                        widen4(x.w, w[6], w[7]);
                        const uint32_t piece = 2u * (uint32_t)quarter, at = dst + 64u * 128u * (uint32_t)j;
                        sts128(at + 16u * (piece ^ (uint32_t)(srow & 7)), w[0], w[1], w[2], w[3]);
                        sts128(at + 16u * ((piece + 1) ^ (uint32_t)(srow & 7)), w[4], w[5], w[6], w[7]);
                    }
                    fence_proxy_async_smem();  // these and the heads, before the MMAs that the arrival lets go
                    mbar_arrive(bars + B_FULL + st);
                    if (ahead) {
                        key[c][0] = __ldg(s0 + 4 * c);
                        key[c][1] = __ldg(s1 + 4 * c);
                    }
                }
                if (ahead) {
                    load_scale(next_blocks.own);
                    if (k + 2 < todo) {
                        advance(after);
                        after_blocks = look_up(after);
                    }
                }
                read_products();
                late.heads = heads;
                late.last = h0 + kHeadChunk >= p.h_q;
                late.job = job;
                late.scale = my_scale;
                late.out = page < u.n ? p.scores + ((size_t)u.b * p.s_q + u.tok) * p.max_blocks + page : nullptr;
            }
            u = next;
            next = after;
            next_blocks = after_blocks;
        }
        read_products();
    }
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
    return p.d == kDqk ? launch_after(page_scores_kernel<kDqk>, dim3(grid), dim3(kCtaThreads), score_smem<kDqk>(), stream, p)
                       : launch_after(page_scores_kernel<kDv>, dim3(grid), dim3(kCtaThreads), score_smem<kDv>(), stream, p);
}

}  // namespace mla
