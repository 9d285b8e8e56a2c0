// Cache rows: writing tokens' rows into the paged latent cache and reading
// them back, for bf16 pages and for packed e4m3 pages with per-token scales
// (layouts in include/mla_decode.h).
//
// Row r of the ragged input belongs to sequence b with cu_rows[b] <= r <
// cu_rows[b + 1] (or b = r / rows_per_seq), sits at position
// p = starts[b] + r - cu_rows[b], and lives in row p % 64 of page
// block_table[b][p / 64].
//   write, e4m3:  c = max |x| / 448 (1 for a row of zeros), code = e4m3(x / c)
//   read, e4m3:   x = bf16(c * code)
// Both quotients are IEEE divisions in fp32, so a row's codes have one value.
//
// A warp takes two consecutive rows as one list of 8-value pieces (2 x 72, or
// 2 x 64 for d = 512), so that few lanes idle behind the 72 pieces of a row.  Every access is
// a contiguous run within a row, all of a lane's loads are in flight together, a
// row's maximum is one warp reduction and the rows never leave the registers: one
// pass over the bytes, bound by HBM on prompts and by the launch on single tokens.
// Measured on GB300, 131,072 / 262,144 rows (e4m3 write / read): one row per warp 52.1 / 87.1 us,
// two 46.1 / 74.0, four 45.7 / 71.8, but 64 rows (a decoding step) 2.3 / 3.0 / 4.3 us.  Two reach,
// on 262,144 rows, 6.7 TB/s in the bf16 copies, 6.2 in the e4m3 read and 5.5 in the e4m3
// write, whose instructions (the quotients) fill 67 % of the issue slots.
#include <cuda_runtime.h>

#include "mla_internal.h"
#include "mla_sm103.cuh"

namespace mla {
namespace {

constexpr int kRowWarps = 8;

// Sequence of row r: the number of entries of cu[1 .. batch] that are <= r, by
// a 32-way search of the whole warp; batch when r lies behind the last
// sequence, -1 when it lies before the first.
__device__ __forceinline__ int find_sequence(const int32_t *__restrict__ cu, int batch, int64_t r, int lane) {
    int lo = 0, len = batch;
    while (len > 0) {
        const int step = (len + 31) >> 5;
        const int first = lane * step;
        const bool below = first < len && cu[1 + lo + min(first + step, len) - 1] <= r;
        const int full = __popc(__ballot_sync(0xffffffffu, below)) * step;  // entries known to be <= r
        if (full >= len) {
            lo += len;
            len = 0;
        } else {
            lo += full;
            len = min(step, len - full) - 1;  // the block's last entry is > r
        }
    }
    return (lo < batch && cu[lo] > r) ? -1 : lo;
}

// Places of rows r0 .. r0 + R - 1: lane i < R learns that row r0 + i is cached at
// row `off` of block `blk`, or blk = -1 when it belongs to no sequence or its place
// does not exist (the latter sets a status bit).  Neighbouring rows mostly share a
// sequence, so a search is made once per sequence.
template <int R>
__device__ __forceinline__ void locate(const CacheRowsParams &p, int64_t r0, int lane, int64_t &blk, int &off) {
    int b = 0;
    int64_t i = 0;
    if (p.cu_rows) {
        int at = find_sequence(p.cu_rows, p.batch, r0, lane);
        int64_t end = at >= 0 && at < p.batch ? p.cu_rows[at + 1] : -1;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int64_t r = r0 + k;
            if (k > 0 && at < p.batch && r >= end) {
                at = find_sequence(p.cu_rows, p.batch, r, lane);
                end = at >= 0 && at < p.batch ? p.cu_rows[at + 1] : -1;
            }
            if (lane == k) b = at;
        }
        if (b >= p.batch) b = -1;
        if (lane < R && b >= 0) i = r0 + lane - p.cu_rows[b];
    } else {
        b = (int)((r0 + lane) / p.rows_per_seq);
        i = r0 + lane - (int64_t)b * p.rows_per_seq;
    }
    blk = -1;
    off = 0;
    if (lane >= R || r0 + lane >= p.num_rows || b < 0 || b >= p.batch) return;
    const int64_t pos = (int64_t)p.starts[b] + i;
    if (pos < 0 || pos >= (int64_t)p.max_blocks * kPage) {
        atomicOr(p.status, MLA_DEVERR_SEQLEN);
        return;
    }
    const int id = p.block_table[(size_t)b * p.max_blocks + pos / kPage];
    if (id < 0 || (int64_t)id >= p.num_blocks) {
        atomicOr(p.status, MLA_DEVERR_BLOCK_ID);
        return;
    }
    blk = id;
    off = (int)(pos % kPage);
}

constexpr int kRows = 2;  // rows of a warp
// 16-byte pieces of the outside rows that a warp's lanes go through
template <int kPieces>
constexpr int items() { return (kRows * kPieces + 31) / 32; }

// piece `piece` of the outside row r: 8 bf16 values of its latent or RoPE part
__device__ __forceinline__ uint4 *outside(const CacheRowsParams &p, int64_t r, int piece) {
    return piece < 64 ? reinterpret_cast<uint4 *>(p.latent + r * p.latent_stride) + piece
                      : reinterpret_cast<uint4 *>(p.rope + r * p.rope_stride) + (piece - 64);
}

// bf16 pages, both directions
template <int D, bool kWrite>
__global__ void __launch_bounds__(kRowWarps * 32) copy_rows_kernel(const CacheRowsParams p) {
    constexpr int kPieces = D / 8, kItems = items<kPieces>();
    sm103::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t r0 = ((int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5)) * kRows;
    if (r0 >= p.num_rows) return;
    uint4 x[kItems];
    if constexpr (kWrite) {
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int item = lane + 32 * j, row = item / kPieces, piece = item - row * kPieces;
            if (row < kRows && r0 + row < p.num_rows) x[j] = *outside(p, r0 + row, piece);
        }
    }
    int64_t blk;
    int off;
    locate<kRows>(p, r0, lane, blk, off);
    const long long base = blk < 0 ? -1ll : (blk * kPage + off) * kPieces;
    long long at[kItems];
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        const int item = lane + 32 * j, row = item / kPieces, piece = item - row * kPieces;
        const long long first = __shfl_sync(0xffffffffu, base, row & 31);
        at[j] = first < 0 || row >= kRows ? -1ll : first + piece;
    }
    uint4 *cache = static_cast<uint4 *>(p.cache);
    if constexpr (!kWrite) {
#pragma unroll
        for (int j = 0; j < kItems; ++j)
            if (at[j] >= 0) x[j] = cache[at[j]];
    }
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        const int item = lane + 32 * j, row = item / kPieces, piece = item - row * kPieces;
        if (at[j] < 0) continue;
        if constexpr (kWrite) cache[at[j]] = x[j];
        else *outside(p, r0 + row, piece) = x[j];
    }
}

// The codes of 8 values with scale c, e4m3(x / c), by the division.
__device__ __noinline__ uint2 divide8(uint4 x, float c) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t code[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        code[i] = sm103::pack_e4m3x2(__uint_as_float(w[i] << 16) / c + 0.f, __uint_as_float(w[i] & 0xffff0000u) / c + 0.f);
    return make_uint2(code[0] | (code[1] << 16), code[2] | (code[3] << 16));
}

// The same without it: with inv the correctly rounded reciprocal of c,
// q = x inv, r = x - q c (exact in one fused operation) and q + r inv is the
// correctly rounded quotient (Markstein's theorem; c = m / 448 for an 8-bit m
// never has the all-ones significand that it excludes).  Two values per
// instruction.  A zero's code is +0.
__device__ __forceinline__ uint2 quantise8(uint4 x, uint64_t inv2, uint64_t minus_c2) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    const uint64_t zero2 = sm103::f2_pack(0.f, 0.f);
    uint32_t code[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t v = sm103::f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        const uint64_t q = sm103::f2_fma(v, inv2, zero2), r = sm103::f2_fma(q, minus_c2, v);
        float a, b;
        sm103::f2_unpack(sm103::f2_fma(r, inv2, q), a, b);
        code[i] = sm103::pack_e4m3x2(a, b);
    }
    return make_uint2(code[0] | (code[1] << 16), code[2] | (code[3] << 16));
}

__global__ void __launch_bounds__(kRowWarps * 32) write_rows_e4m3_kernel(const CacheRowsParams p) {
    constexpr int kPieces = kDqk / 8, kItems = items<kPieces>();
    sm103::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t r0 = ((int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5)) * kRows;
    if (r0 >= p.num_rows) return;
    uint4 x[kItems];
    // largest magnitude bits of a piece's even and odd values: they order as
    // magnitudes do, infinities and NaN on top
    uint32_t top[kItems];
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        const int item = lane + 32 * j, row = item / kPieces, piece = item - row * kPieces;
        x[j] = row < kRows && r0 + row < p.num_rows ? *outside(p, r0 + row, piece) : make_uint4(0, 0, 0, 0);
    }
    int64_t blk;
    int off;
    locate<kRows>(p, r0, lane, blk, off);
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
        top[j] = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu), __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
    }
    float scale[kRows], inv[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        uint32_t t = 0;
#pragma unroll
        for (int j = 0; j < kItems; ++j)
            if (32 * j / kPieces <= k && (32 * j + 31) / kPieces >= k)  // the pieces that may be of row k
                t = __vmaxu2(t, (lane + 32 * j) / kPieces == k ? top[j] : 0u);
        t = __reduce_max_sync(0xffffffffu, max(t >> 16, t & 0xffffu)) << 16;
        scale[k] = t >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : t ? __uint_as_float(t) / 448.f : 1.f;
        inv[k] = 1.f / scale[k];
    }
    uint8_t *page = static_cast<uint8_t *>(p.cache) + (size_t)(blk < 0 ? 0 : blk) * MLA_FP8_PAGE_BYTES(kDqk);
    if (lane < kRows && blk >= 0) {
        float c = scale[0];
#pragma unroll
        for (int k = 1; k < kRows; ++k)
            if (lane == k) c = scale[k];
        if (!(c < (float)MLA_FP8_SCALE_LIMIT)) atomicOr(p.status, MLA_DEVERR_SCALE);
        reinterpret_cast<float *>(page + kPage * kDqk)[off] = c;
    }
    const unsigned long long base = blk < 0 ? 0ull : (unsigned long long)(page + off * kDqk);
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        const int item = lane + 32 * j, row = item / kPieces, piece = item - row * kPieces;
        const unsigned long long dst = __shfl_sync(0xffffffffu, base, row & 31);
        const int k0 = 32 * j / kPieces, k1 = k0 + 1 < kRows ? k0 + 1 : k0;  // the rows that a lane's piece may be of
        const float c = row != k0 ? scale[k1] : scale[k0], in = row != k0 ? inv[k1] : inv[k0];
        if (dst && row < kRows) {
            // below 2^-100 the remainder and the reciprocal leave the normal range
            const uint2 code = c < 0x1p-100f ? divide8(x[j], c) : quantise8(x[j], sm103::f2_pack(in, in), sm103::f2_pack(-c, -c));
            reinterpret_cast<uint2 *>(dst)[piece] = code;
        }
    }
}

__device__ __forceinline__ uint4 dequantise8(uint32_t lo, uint32_t hi, float c) {
    const uint32_t code[4] = {lo, lo >> 16, hi, hi >> 16};
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        sm103::f16x2_to_f32(sm103::e4m3x2_to_f16x2(code[i]), a, b);
        out[i] = sm103::pack_bf16(c * a, c * b);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

__global__ void __launch_bounds__(kRowWarps * 32) read_rows_e4m3_kernel(const CacheRowsParams p) {
    constexpr int kPieces = kDqk / 8, kItems = items<kPieces>();
    sm103::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t r0 = ((int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5)) * kRows;
    if (r0 >= p.num_rows) return;
    int64_t blk;
    int off;
    locate<kRows>(p, r0, lane, blk, off);
    const uint8_t *page = static_cast<const uint8_t *>(p.cache) + (size_t)(blk < 0 ? 0 : blk) * MLA_FP8_PAGE_BYTES(kDqk);
    const unsigned long long base = blk < 0 ? 0ull : (unsigned long long)(page + off * kDqk);
    float c = 0.f;
    if (lane < kRows && blk >= 0) c = reinterpret_cast<const float *>(page + kPage * kDqk)[off];
    uint2 x[kItems];
    bool on[kItems];
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        const int item = lane + 32 * j, row = item / kPieces, piece = item - row * kPieces;
        const unsigned long long src = __shfl_sync(0xffffffffu, base, row & 31);
        on[j] = src != 0 && row < kRows;
        if (on[j]) x[j] = reinterpret_cast<const uint2 *>(src)[piece];
    }
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        const int item = lane + 32 * j, row = item / kPieces, piece = item - row * kPieces;
        const float s = __shfl_sync(0xffffffffu, c, row & 31);
        if (on[j]) *outside(p, r0 + row, piece) = dequantise8(x[j].x, x[j].y, s);
    }
}

}  // namespace

cudaError_t launch_cache_rows(const CacheRowsParams &p, int d, bool e4m3, bool write, cudaStream_t stream) {
    const int per_cta = kRowWarps * kRows;
    const unsigned grid = (unsigned)((p.num_rows + per_cta - 1) / per_cta);
    void (*kernel)(CacheRowsParams) =
        e4m3 ? (write ? write_rows_e4m3_kernel : read_rows_e4m3_kernel)
             : (d == kDqk ? (write ? copy_rows_kernel<kDqk, true> : copy_rows_kernel<kDqk, false>)
                          : (write ? copy_rows_kernel<kDv, true> : copy_rows_kernel<kDv, false>));
    return launch_after(kernel, dim3(grid), dim3(kRowWarps * 32), 0, stream, p);
}

}  // namespace mla
