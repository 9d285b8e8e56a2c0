// Page keys: one int8 row and one fp32 scale that stand for the 64 cached rows
// of a page in the page-selecting decode (mla_select_pages.cu).
//
// For a page with n rows inside its sequence:
//   mean[c] = (sum over its rows of k[c]) / n        fp32, absent rows as 0,
//             summed as a balanced tree over the row index (neighbours first)
//   scale   = max_c |mean[c]| / 127                  (1 for a mean of zeros, else 2^-149 at least)
//   key[c]  = rint(mean[c] / scale)                  -127 .. 127: limited, since a subnormal
//             scale has few bits and the quotient may round to 128
// The order of the sums and the roundings (IEEE fp32 throughout) are part of
// the definition, so a page's key has one value however it is computed.  A page
// whose mean is not finite gets zero codes and a NaN scale (its score is then
// NaN, which the selection ranks above every number).
//
// Only the pages that positions [starts[b], seqlens[b]) touch are computed: a
// decoding step updates one or two pages per sequence.  The host does not know
// the lengths, so a fixed grid walks the list of touched pages: every CTA
// prefix-sums the sequences' page counts in shared memory and takes every
// gridDim.x-th page.  Within a page each thread owns one 16-byte column piece of
// a run of consecutive rows (16 bf16 rows, 8 e4m3 rows), all its loads in
// flight together, and the next page's behind them; the runs' sums are the lower levels of the tree and the
// shared-memory join its upper levels.  One pass over the bytes: the bf16 form is bound by
// HBM (6.1 TB/s on 262,144 tokens); the e4m3 form reaches 4.0 TB/s on 524,288, with 54 % of
// the issue slots used (widening, scaling and adding every code) between its barriers.
#include <cuda_runtime.h>

#include "mla_internal.h"
#include "mla_page_walk.cuh"
#include "mla_sm103.cuh"

namespace mla {
namespace {

constexpr int kKeyThreads = 288;
// CTAs of an SM: the e4m3 form's loads take half the registers (64 x 8192 tokens: 77.5 us
// with 3, 81.8 with 2; bf16, 32 x 8192 tokens: 60.1 with 3, 49.5 with 2, 6.1 TB/s)
constexpr int key_ctas(bool e4m3) { return e4m3 ? 3 : 2; }

template <int D, bool E4M3>
__global__ void __launch_bounds__(kKeyThreads, key_ctas(E4M3)) page_keys_kernel(const PageKeysParams p) {
    constexpr int kCols = E4M3 ? 16 : 8;              // columns of one 16-byte piece
    constexpr int kPieces = D / kCols;                // 72 / 64 (bf16), 36 (e4m3)
    constexpr int kRuns = E4M3 ? 8 : 4;               // runs of consecutive rows
    constexpr int kRun = kPage / kRuns;               // rows of a run
    static_assert(kPieces * kRuns <= kKeyThreads, "one thread per piece and run");
    __shared__ float s_part[kRuns][D];
    __shared__ float s_max[kKeyThreads / 32];
    __shared__ PageWalk<kKeyThreads>::Shared s_walk;
    sm103::griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int piece = tid % kPieces, run = tid / kPieces;

    PageWalk<kKeyThreads> walk(s_walk, p.batch, blockIdx.x, gridDim.x);
    // A page ahead of the one whose loads are in flight: its block id travels
    // while they do, and its own loads start as soon as the sums have freed the
    // registers, before the CTA meets at its barriers.
    struct Entry {
        bool valid = false;
        int blk = -1, n = 0;
    };
    auto next_entry = [&] {
        Entry e;
        int b, pg;
        e.valid = walk.next(
            [&](int i, int &first, int &count) {
                const int T = clamp_len(p.seqlens[i], p.max_blocks, p.status);
                int t0 = p.starts ? p.starts[i] : 0;
                if (t0 < 0) t0 = 0;
                first = t0 / kPage;
                count = max(0, (T + kPage - 1) / kPage - first);
            },
            b, pg);
        if (e.valid) {
            e.blk = p.block_table[(size_t)b * p.max_blocks + pg];
            e.n = min(kPage, min(p.seqlens[b], p.max_blocks * kPage) - pg * kPage);
        }
        return e;
    };
    uint4 x[kRun];
    float c[E4M3 ? kRun : 1];
    auto load = [&](Entry &e) {
        if (!e.valid) return;
        if (e.blk < 0 || (int64_t)e.blk >= p.num_blocks) {
            if (tid == 0) atomicOr(p.status, MLA_DEVERR_BLOCK_ID);
            e.blk = -1;
            e.n = 0;
        }
        if (run >= kRuns) return;
        const char *page = static_cast<const char *>(p.cache) +
                           (size_t)max(e.blk, 0) * (E4M3 ? MLA_FP8_PAGE_BYTES(kDqk) : kPage * D * 2);
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const int row = run * kRun + i;
            x[i] = row < e.n ? reinterpret_cast<const uint4 *>(page)[row * kPieces + piece] : make_uint4(0, 0, 0, 0);
            if constexpr (E4M3) c[i] = row < e.n ? reinterpret_cast<const float *>(page + kPage * kDqk)[row] : 0.f;
        }
    };
    Entry cur = next_entry(), nxt;
    if (cur.valid) nxt = next_entry();
    load(cur);
    while (cur.valid) {
        const int n = cur.n, blk = cur.blk;
        if (run < kRuns) {
            float v[kCols];
            if constexpr (E4M3) {
#pragma unroll
                for (int w = 0; w < 8; ++w) {  // two columns at a time
                    uint64_t s2[kRun];
#pragma unroll
                    for (int i = 0; i < kRun; ++i) {
                        const uint32_t word = (w >> 1) == 0 ? x[i].x : (w >> 1) == 1 ? x[i].y : (w >> 1) == 2 ? x[i].z : x[i].w;
                        float a, b;
                        sm103::f16x2_to_f32(sm103::e4m3x2_to_f16x2((w & 1) ? word >> 16 : word), a, b);
                        // (an absent row's codes and scale are 0)
                        s2[i] = sm103::f2_fma(sm103::f2_pack(a, b), sm103::f2_pack(c[i], c[i]), sm103::f2_pack(0.f, 0.f));
                    }
#pragma unroll
                    for (int s = 1; s < kRun; s *= 2)
#pragma unroll
                        for (int i = 0; i < kRun; i += 2 * s) s2[i] = sm103::f2_add(s2[i], s2[i + s]);
                    sm103::f2_unpack(s2[0], v[2 * w], v[2 * w + 1]);
                }
            } else {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint64_t s2[kRun];
#pragma unroll
                    for (int i = 0; i < kRun; ++i) {
                        const uint32_t word = w == 0 ? x[i].x : w == 1 ? x[i].y : w == 2 ? x[i].z : x[i].w;
                        s2[i] = sm103::f2_pack(__uint_as_float(word << 16), __uint_as_float(word & 0xffff0000u));
                    }
#pragma unroll
                    for (int s = 1; s < kRun; s *= 2)
#pragma unroll
                        for (int i = 0; i < kRun; i += 2 * s) s2[i] = sm103::f2_add(s2[i], s2[i + s]);
                    sm103::f2_unpack(s2[0], v[2 * w], v[2 * w + 1]);
                }
            }
#pragma unroll
            for (int j = 0; j < kCols; j += 4)
                *reinterpret_cast<float4 *>(&s_part[run][piece * kCols + j]) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
        load(nxt);
        Entry after;
        if (nxt.valid) after = next_entry();
        __syncthreads();
        // columns 2 tid, 2 tid + 1: the tree's upper levels and the mean
        float m0 = 0.f, m1 = 0.f;
        if (2 * tid < D) {
            float2 u[kRuns];
#pragma unroll
            for (int g = 0; g < kRuns; ++g) u[g] = *reinterpret_cast<const float2 *>(&s_part[g][2 * tid]);
#pragma unroll
            for (int s = 1; s < kRuns; s *= 2)
#pragma unroll
                for (int g = 0; g < kRuns; g += 2 * s) {
                    u[g].x = __fadd_rn(u[g].x, u[g + s].x);
                    u[g].y = __fadd_rn(u[g].y, u[g + s].y);
                }
            m0 = u[0].x / (float)max(n, 1);
            m1 = u[0].y / (float)max(n, 1);
        }
        // magnitude bits order as magnitudes do, with infinities and NaN on top
        uint32_t top = max(__float_as_uint(m0) & 0x7fffffffu, __float_as_uint(m1) & 0x7fffffffu);
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) s_max[warp] = __uint_as_float(top);
        __syncthreads();
        top = 0;
#pragma unroll
        for (int i = 0; i < kKeyThreads / 32; ++i) top = max(top, __float_as_uint(s_max[i]));
        const bool finite = top < 0x7f800000u;
        const float scale = !finite ? __uint_as_float(0x7fffffffu) : top ? fmaxf(__uint_as_float(top) / 127.f, 0x1p-149f) : 1.f;
        if (blk >= 0 && 2 * tid < D) {
            char2 k = make_char2(0, 0);
            const auto code = [&](float m) { return (signed char)__float2int_rn(fminf(fmaxf(m / scale, -127.f), 127.f)); };
            if (finite) k = make_char2(code(m0), code(m1));
            reinterpret_cast<char2 *>(p.keys + (size_t)blk * D)[tid] = k;
        }
        if (blk >= 0 && tid == 0) p.scales[blk] = scale;
        cur = nxt;
        nxt = after;
    }
}

}  // namespace

cudaError_t launch_page_keys(const PageKeysParams &p, int d, bool e4m3, cudaStream_t stream) {
    int sms = 0;
    cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    const long long most = (long long)p.batch * p.max_blocks;
    const long long at_once = (long long)key_ctas(e4m3) * sms;
    const unsigned grid = (unsigned)(most < at_once ? most : at_once);
    void (*kernel)(PageKeysParams) =
        e4m3 ? page_keys_kernel<kDqk, true> : d == kDqk ? page_keys_kernel<kDqk, false> : page_keys_kernel<kDv, false>;
    return launch_after(kernel, dim3(grid), dim3(kKeyThreads), 0, stream, p);
}

}  // namespace mla
