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
// One warp per row: 72 (d = 576) or 64 (d = 512) 16-byte pieces of 8 bf16
// values, pieces lane, lane + 32 from the latent part and 64 + lane from the
// RoPE part, so that every access of a warp is a contiguous run.  The row's
// maximum is one warp reduction and the row never leaves the registers: one
// pass over the bytes, bound by HBM on prompts and by the launch on single
// tokens.
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

// Where row r lives; false when it belongs to no sequence or its place does
// not exist (the latter sets a status bit).
__device__ __forceinline__ bool locate(const CacheRowsParams &p, int64_t r, int lane, int64_t &blk, int &off) {
    int b;
    int64_t i;
    if (p.cu_rows) {
        b = find_sequence(p.cu_rows, p.batch, r, lane);
        if (b < 0 || b >= p.batch) return false;
        i = r - p.cu_rows[b];
    } else {
        b = (int)(r / p.rows_per_seq);
        i = r - (int64_t)b * p.rows_per_seq;
    }
    const int64_t pos = (int64_t)p.starts[b] + i;
    if (pos < 0 || pos >= (int64_t)p.max_blocks * kPage) {
        if (lane == 0) atomicOr(p.status, MLA_DEVERR_SEQLEN);
        return false;
    }
    const int id = p.block_table[(size_t)b * p.max_blocks + pos / kPage];
    if (id < 0 || (int64_t)id >= p.num_blocks) {
        if (lane == 0) atomicOr(p.status, MLA_DEVERR_BLOCK_ID);
        return false;
    }
    blk = id;
    off = (int)(pos % kPage);
    return true;
}

template <int D>
__global__ void __launch_bounds__(kRowWarps * 32) write_rows_kernel(const CacheRowsParams p) {
    sm103::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    if (r >= p.num_rows) return;
    const uint4 *src = reinterpret_cast<const uint4 *>(p.latent + r * p.latent_stride);
    const uint4 a = src[lane], b = src[lane + 32];
    uint4 c = make_uint4(0, 0, 0, 0);
    if (D > kDv && lane < 8) c = reinterpret_cast<const uint4 *>(p.rope + r * p.rope_stride)[lane];
    int64_t blk;
    int off;
    if (!locate(p, r, lane, blk, off)) return;
    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.cache) + (blk * kPage + off) * D);
    dst[lane] = a;
    dst[lane + 32] = b;
    if (D > kDv && lane < 8) dst[64 + lane] = c;
}

__device__ __forceinline__ void unpack8(uint4 x, float (&v)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint2 quantise8(const float (&v)[8], float c) {
    uint2 r;
    r.x = sm103::pack_e4m3x2(v[0] / c, v[1] / c) | (sm103::pack_e4m3x2(v[2] / c, v[3] / c) << 16);
    r.y = sm103::pack_e4m3x2(v[4] / c, v[5] / c) | (sm103::pack_e4m3x2(v[6] / c, v[7] / c) << 16);
    return r;
}

__global__ void __launch_bounds__(kRowWarps * 32) write_rows_e4m3_kernel(const CacheRowsParams p) {
    sm103::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    if (r >= p.num_rows) return;
    const uint4 *src = reinterpret_cast<const uint4 *>(p.latent + r * p.latent_stride);
    float x[3][8];
    unpack8(src[lane], x[0]);
    unpack8(src[lane + 32], x[1]);
    unpack8(lane < 8 ? reinterpret_cast<const uint4 *>(p.rope + r * p.rope_stride)[lane] : make_uint4(0, 0, 0, 0), x[2]);
    int64_t blk;
    int off;
    if (!locate(p, r, lane, blk, off)) return;
    // the maximum over magnitude bits, which order as the values do with
    // infinities and NaN on top
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[i][j]) & 0x7fffffffu);
    top = __reduce_max_sync(0xffffffffu, top);
    const bool finite = top < 0x7f800000u;
    const float c = !finite ? __uint_as_float(0x7fffffffu) : top ? __uint_as_float(top) / 448.f : 1.f;
    if (!(c < (float)MLA_FP8_SCALE_LIMIT) && lane == 0) atomicOr(p.status, MLA_DEVERR_SCALE);
    uint8_t *page = static_cast<uint8_t *>(p.cache) + (size_t)blk * MLA_FP8_PAGE_BYTES(kDqk);
    uint2 *dst = reinterpret_cast<uint2 *>(page + off * kDqk);
    dst[lane] = quantise8(x[0], c);
    dst[lane + 32] = quantise8(x[1], c);
    if (lane < 8) dst[64 + lane] = quantise8(x[2], c);
    if (lane == 0) reinterpret_cast<float *>(page + kPage * kDqk)[off] = c;
}

template <int D>
__global__ void __launch_bounds__(kRowWarps * 32) read_rows_kernel(const CacheRowsParams p) {
    sm103::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    if (r >= p.num_rows) return;
    int64_t blk;
    int off;
    if (!locate(p, r, lane, blk, off)) return;
    const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.cache) + (blk * kPage + off) * D);
    const uint4 a = src[lane], b = src[lane + 32];
    uint4 c = make_uint4(0, 0, 0, 0);
    if (D > kDv && lane < 8) c = src[64 + lane];
    uint4 *dst = reinterpret_cast<uint4 *>(p.latent + r * p.latent_stride);
    dst[lane] = a;
    dst[lane + 32] = b;
    if (D > kDv && lane < 8) reinterpret_cast<uint4 *>(p.rope + r * p.rope_stride)[lane] = c;
}

__device__ __forceinline__ uint4 dequantise8(uint2 x, float c) {
    float v[8];
    sm103::f16x2_to_f32(sm103::e4m3x2_to_f16x2(x.x), v[0], v[1]);
    sm103::f16x2_to_f32(sm103::e4m3x2_to_f16x2(x.x >> 16), v[2], v[3]);
    sm103::f16x2_to_f32(sm103::e4m3x2_to_f16x2(x.y), v[4], v[5]);
    sm103::f16x2_to_f32(sm103::e4m3x2_to_f16x2(x.y >> 16), v[6], v[7]);
    return make_uint4(sm103::pack_bf16(c * v[0], c * v[1]), sm103::pack_bf16(c * v[2], c * v[3]),
                      sm103::pack_bf16(c * v[4], c * v[5]), sm103::pack_bf16(c * v[6], c * v[7]));
}

__global__ void __launch_bounds__(kRowWarps * 32) read_rows_e4m3_kernel(const CacheRowsParams p) {
    sm103::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    if (r >= p.num_rows) return;
    int64_t blk;
    int off;
    if (!locate(p, r, lane, blk, off)) return;
    const uint8_t *page = static_cast<const uint8_t *>(p.cache) + (size_t)blk * MLA_FP8_PAGE_BYTES(kDqk);
    const uint2 *src = reinterpret_cast<const uint2 *>(page + off * kDqk);
    const float s = reinterpret_cast<const float *>(page + kPage * kDqk)[off];
    const uint2 a = src[lane], b = src[lane + 32];
    uint2 c = make_uint2(0, 0);
    if (lane < 8) c = src[64 + lane];
    uint4 *dst = reinterpret_cast<uint4 *>(p.latent + r * p.latent_stride);
    dst[lane] = dequantise8(a, s);
    dst[lane + 32] = dequantise8(b, s);
    if (lane < 8) reinterpret_cast<uint4 *>(p.rope + r * p.rope_stride)[lane] = dequantise8(c, s);
}

}  // namespace

cudaError_t launch_cache_rows(const CacheRowsParams &p, int d, bool e4m3, bool write, cudaStream_t stream) {
    const unsigned grid = (unsigned)((p.num_rows + kRowWarps - 1) / kRowWarps);
    void (*kernel)(CacheRowsParams) =
        e4m3 ? (write ? write_rows_e4m3_kernel : read_rows_e4m3_kernel)
             : (d == kDqk ? (write ? write_rows_kernel<kDqk> : read_rows_kernel<kDqk>)
                          : (write ? write_rows_kernel<kDv> : read_rows_kernel<kDv>));
    return launch_after(kernel, dim3(grid), dim3(kRowWarps * 32), 0, stream, p);
}

}  // namespace mla
