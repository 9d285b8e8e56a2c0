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
// page's heads.  The keys arrive as int8 (580 bytes a page) through asynchronous
// copies that run up to six chunks of 64 dims ahead, and are widened to f16 on
// their way into tensor memory, where A is read from: through shared memory the
// staging, the MMAs' reads of both operands and the copies share its bandwidth.
// The heads' codes come from a small kernel in front.
// Work is cut into contiguous ranges of units, one per CTA.  A unit holds one token
// whatever its heads and however many tokens share its pages: the right size for one
// token of 128 heads, while s_q tokens widen the same keys s_q times (16 sequences of
// up to 256 pages and four tokens: 14 us) and 16 heads fill an eighth of an MMA.
//
// Measured on GB300, 64 tokens x 1024 pages x 128 heads (38 MB of keys and 9.7 GFLOP: 6
// us for either): 155 us on one issuing thread among the staging ones, 36.6 with
// its own warp and products read late, 30.8 with the next unit's loads spread over
// the staging, 26.5 by asynchronous copies, 24.2 with A in tensor memory.  What is left
// per CTA: 6 us until the first keys and heads are there, four units of 3.5 us, of
// which the widening threads' own work is 2.5.  A second issuer, each with half the
// dims, changed nothing while A was in shared memory; now there is no room for its sums.
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
constexpr int kStages = 4;                    // widened chunks of 64 dims (in tensor memory), and
constexpr int kRaw = 3;                       // chunks of codes on their way, of each half of the warps
constexpr uint32_t kTileBytes = 128 * 128;    // 128 rows of 64 f16
constexpr uint32_t kRawBytes = 128 * 64;
constexpr uint32_t kTmemCols = 512;           // two accumulators of 128 columns, then (kStageCol) the stages of 32
constexpr uint32_t kStageCol = 256;

template <int D>
struct ScoreSmem {
    static constexpr int kChunks = D / 64;
    static constexpr uint32_t q = 0;                                  // [chunk][head][64] f16, 128-byte swizzle
    static constexpr uint32_t raw = q + kChunks * kTileBytes;         // [warp][slot][page of the warp] 64 codes
    static constexpr uint32_t unit = raw + 2 * kRaw * kRawBytes;      // [head] u_h
    static constexpr uint32_t best = unit + kHeadChunk * 4;           // [unit parity][page] maximum of the upper heads
    static constexpr uint32_t bars = best + 2 * kTilePages * 4;       // B_* below
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
// pages for the token (which cost 7 us per token and CTA).  64 x 128 heads: 8.6 us
// with divisions, 6.4 without.
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
    // x / u without the division: with inv = 1 / u correctly rounded, q = x inv and
    // the fused remainder r = x - q u, q + r inv is the correctly rounded quotient
    // (Markstein's theorem; u = m / 127 for an 8-bit m never has the all-ones
    // significand that it excludes: m is 127 times a power of two, or 1/254 of it off)
    const float inv = 1.f / u;
    const uint64_t inv2 = f2_pack(inv, inv), minus_u2 = f2_pack(-u, -u);
    uint2 *dst = reinterpret_cast<uint2 *>(p.q_codes + row * D);
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        if (lane + 32 * j >= kPieces) continue;
        const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
        uint32_t c[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float a = __uint_as_float(w[e] << 16), b = __uint_as_float(w[e] & 0xffff0000u);
            if (u < 0x1p-100f) {  // the remainder and the reciprocal would leave the normal range
                a /= u;
                b /= u;
            } else {
                const uint64_t x2 = f2_pack(a, b), q2 = f2_fma(x2, inv2, f2_pack(0.f, 0.f));
                f2_unpack(f2_fma(f2_fma(q2, minus_u2, x2), inv2, q2), a, b);
            }
            c[2 * e] = finite ? (uint32_t)__float2int_rn(a) & 255u : 0u;
            c[2 * e + 1] = finite ? (uint32_t)__float2int_rn(b) & 255u : 0u;
        }
        dst[lane + 32 * j] = make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24, c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
    }
    if (lane == 0) p.q_units[row] = u;
}

// barriers: stage staged (128 arrivals) / free (commit), accumulator finished
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
            tc_fence_after();
            const uint64_t bd = desc_sw128(base_s + S::q + c * kTileBytes, 16, 1024);
#pragma unroll
            for (int s = 0; s < 4; ++s) mma_ts(d, tmem + kStageCol + 32 * st + 8 * s, bd + 2 * s, idesc, c > 0 || s > 0);
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
            mbar_init(bars + i, i < B_EMPTY ? kScoreThreads / 2 : i < B_READ ? 1 : kScoreThreads);
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
    // The two halves of the warps widen every other chunk: a warp 64 dims of its 32
    // pages, a page per lane.  It copies them kRaw of its chunks ahead and across
    // units, so that the loads never wait for one another and no warp for another's.
    // Four neighbouring lanes copy one page's 64 bytes, pages first + lane / 4 and 8, 16
    // and 24 behind it.  A page that is not there reads block 0's key (its score goes
    // nowhere, or, for a bad block id, is any number).  The block ids are looked up a
    // unit ahead of the copies.
    const int lane = tid & 31, srow = (row & ~31) + (lane >> 2);
    const int passes = (p.h_q + kHeadChunk - 1) / kHeadChunk;  // jobs of a unit: its heads, 128 at a time
    struct Blocks {
        int s[4], own;
    };
    auto block_of = [&](const UnitAt &u, int r) {
        const int page = u.tile * kTilePages + r;
        return page < u.n ? __ldg(p.block_table + (size_t)u.b * p.max_blocks + page) : 0;
    };
    auto look_up = [&](const UnitAt &u) { return Blocks{{block_of(u, srow), block_of(u, srow + 8), block_of(u, srow + 16), block_of(u, srow + 24)}, block_of(u, row)}; };
    auto safe = [&](int blk) { return blk < 0 || (int64_t)blk >= p.num_blocks ? 0 : blk; };
    auto key_row = [&](int blk) { return reinterpret_cast<const uint4 *>(p.keys + (size_t)safe(blk) * D) + (lane & 3); };
    const uint32_t raw_s = base_s + S::raw + (uint32_t)(warp & 7) * (kRaw * 2048u);  // (16-byte piece q of page r at q ^ (r / 2 & 3))
    struct Feed {
        int left = 0;               // units to come, this one included
        UnitAt u{}, next{};         // and the one behind it, whose block ids are known
        Blocks blocks{};
        const uint4 *s[4] = {};
        float scale = 0.f;          // of the thread's own page of u
        int pass = 0, c = 0;
        uint32_t slot = 0;
    } feed;
    auto feed_unit = [&](const Blocks &b) {
#pragma unroll
        for (int i = 0; i < 4; ++i) feed.s[i] = key_row(b.s[i]);
        if (b.own < 0 || (int64_t)b.own >= p.num_blocks) atomicOr(p.status, MLA_DEVERR_BLOCK_ID);
        feed.scale = __ldg(p.scales + safe(b.own));
        feed.next = feed.u;
        if (feed.left > 1) {
            advance(feed.next);
            feed.blocks = look_up(feed.next);
        }
    };
    // one chunk (an empty group behind the last, which keeps the count)
    auto feed_chunk = [&] {
        if (feed.left > 0) {
            const uint32_t dst = raw_s + feed.slot * 2048u + 64u * (uint32_t)(lane >> 2) + 16u * (uint32_t)((lane ^ (lane >> 3)) & 3);
#pragma unroll
            for (int i = 0; i < 4; ++i) cp_async16(dst + 512u * i, feed.s[i] + 4 * feed.c);
            if (++feed.slot == kRaw) feed.slot = 0;
            if ((feed.c += 2) >= kChunks) {
                feed.c -= kChunks;
                if (++feed.pass == passes) {
                    feed.pass = 0;
                    if (--feed.left > 0) {
                        feed.u = feed.next;
                        feed_unit(feed.blocks);
                    }
                }
            }
        }
        cp_async_commit();
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
        fence_proxy_async_smem();
        named_bar_sync(1, kScoreThreads);  // all of it, before the MMAs that the next arrivals let go
    };

    if (warp == kScoreThreads / 32) {
        if (elect_one_lane()) score_issuer<D>(p, base_s, bars, tmem, (long long)todo * passes);
    } else {
        if (todo > 0) {
            UnitAt u{};
            u.b = s_first[0];
            load_seq(u);
            u.tok = s_first[1] / u.tiles;
            u.tile = s_first[1] - u.tok * u.tiles;
            set_token(u);
            feed.left = todo;
            feed.c = half;
            feed.u = u;
            feed_unit(look_up(u));
        }
#pragma unroll 1
        for (int i = 0; i < kRaw; ++i) feed_chunk();
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
        int units_read = 0;
        auto read_products = [&] {
            if (late.heads == 0) return;
            const uint32_t buf = (uint32_t)(late.job & 1);
            if (ok) ok = mbar_wait(bars + B_DONE + buf, (uint32_t)((late.job >> 1) & 1), p.status);
            __syncwarp();
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
                float *other = s_best + (units_read++ & 1) * kTilePages + row;  // (its last reader met a barrier since)
                if (half) *other = best;
                const bool bad = *s_bad != 0;
                named_bar_sync(1, kScoreThreads);
                if (!half && late.out) {
                    best = fmaxf(best, *other);
                    *late.out = bad ? __uint_as_float(0x7fffffffu) : __fmul_rn(best, late.scale);
                }
                best = -__uint_as_float(0x7f800000u);
            }
            late.heads = 0;
        };
        int held_b = -1, held_tok = -1, held_h = -1;  // whose heads are in shared memory
        uint32_t fill = 0, slot = 0;
        long long job = 0;
        for (int k = 0; k < todo; ++k) {
            static_assert(2 * kRaw < kChunks && kStages % 2 == 0, "the feed is less than a unit ahead");
            const UnitAt u = feed.u;
            const int page = u.tile * kTilePages + row;
            const float my_scale = feed.scale;
            for (int h0 = 0; h0 < p.h_q; h0 += kHeadChunk, ++job) {
                const int heads = min(kHeadChunk, p.h_q - h0);
                if (held_b != u.b || held_tok != u.tok || held_h != h0) {
                    read_products();  // waits for the products that use the heads in place
                    load_heads(u, h0, heads);
                    held_b = u.b;
                    held_tok = u.tok;
                    held_h = h0;
                }
#pragma unroll 1
                for (int c = 0; c < kChunks; ++c, ++fill) {
                    if ((int)(fill & 1) != half) continue;  // the other half's chunk
                    const uint32_t st = fill % kStages;
                    cp_async_wait<kRaw - 1>();
                    __syncwarp();  // every lane's copies
                    const uint32_t src = raw_s + slot * 2048u + 64u * (uint32_t)lane;
                    uint32_t w[32];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 x = lds128(src + 16u * (uint32_t)(j ^ ((lane >> 1) & 3)));
                        widen4(x.x, w[8 * j], w[8 * j + 1]);
                        widen4(x.y, w[8 * j + 2], w[8 * j + 3]);
                        widen4(x.z, w[8 * j + 4], w[8 * j + 5]);
                        widen4(x.w, w[8 * j + 6], w[8 * j + 7]);
                    }
                    if (++slot == kRaw) slot = 0;
                    if (ok) ok = mbar_wait(bars + B_EMPTY + st, ((fill / kStages) & 1) ^ 1, p.status);
                    __syncwarp();
                    tc_fence_after();
                    tmem_st32(tmem + kStageCol + 32 * st + ((uint32_t)(32 * (warp & 3)) << 16), w);
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(bars + B_FULL + st);
                    feed_chunk();  // into the slot that the warp has just read
                }
                read_products();
                late.heads = heads;
                late.last = h0 + kHeadChunk >= p.h_q;
                late.job = job;
                late.scale = my_scale;
                late.out = page < u.n ? p.scores + ((size_t)u.b * p.s_q + u.tok) * p.max_blocks + page : nullptr;
            }
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
