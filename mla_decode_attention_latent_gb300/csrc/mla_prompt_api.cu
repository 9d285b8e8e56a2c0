// C ABI of the prompt path: pages of requests, norms and rotations, rows placed
// into the cache.  See include/mla_decode.h for each contract.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cmath>

#include "mla_internal.h"

namespace mla {
namespace {

struct Range {
    explicit Range(const char *name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int result(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA; }

constexpr int kMaxHeadDim = 576;
constexpr int kMaxRopeDim = 256;

// a strided row of bf16 values that is read or written in 16-byte pieces
bool rows_ok(const void *ptr, int64_t stride, int64_t width, bool written) {
    return aligned16(ptr) && stride >= (written ? width : 0) && stride % 8 == 0;
}

bool real(float x) { return x - x == 0.f; }

int place_rows(const void *latent, int64_t latent_stride, const void *k_rope, int64_t k_rope_stride, int64_t num_rows,
               const void *weight, float eps, const int32_t *positions, const int64_t *turns, int interleaved, float rope_scale,
               const int64_t *slots, void *cache, int64_t num_blocks, int d, void *latent_out, int64_t latent_out_stride,
               void *k_rope_out, int64_t k_rope_out_stride, bool e4m3, struct CUstream_st *stream) {
    if (!cache || num_blocks < 1 || num_rows < 0 || d < 1 || !aligned16(cache) || !aligned16(weight)) return MLA_ERR_INVALID_ARG;
    if (d != kDqk && (e4m3 || d != kDv)) return MLA_ERR_UNSUPPORTED;
    if (num_rows > 0x7fffffffLL || num_blocks > 0x7fffffffLL) return MLA_ERR_UNSUPPORTED;
    const bool rope = d > kDv;
    if (num_rows > 0 && (!latent || !slots || (rope && (!k_rope || !positions || !turns)))) return MLA_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !real(eps) || (rope && !real(rope_scale))) return MLA_ERR_INVALID_ARG;
    if (!rows_ok(latent, latent_stride, kDv, false) || (rope && !rows_ok(k_rope, k_rope_stride, kDqk - kDv, false)))
        return MLA_ERR_INVALID_ARG;
    if (latent_out && !rows_ok(latent_out, latent_out_stride, kDv, true)) return MLA_ERR_INVALID_ARG;
    if (k_rope_out && (!rope || !rows_ok(k_rope_out, k_rope_out_stride, kDqk - kDv, true))) return MLA_ERR_INVALID_ARG;
    if (num_rows == 0) return MLA_OK;
    Range range("mla_norm_rope_cache_write");
    PlaceRowsParams p{};
    p.latent = static_cast<const uint16_t *>(latent);
    p.latent_stride = latent_stride;
    p.k_rope = static_cast<const uint16_t *>(k_rope);
    p.k_rope_stride = k_rope_stride;
    p.num_rows = num_rows;
    p.weight = static_cast<const uint16_t *>(weight);
    p.eps = eps;
    p.rope = {positions, turns, kDqk - kDv, interleaved != 0, rope_scale};
    p.slots = slots;
    p.cache = cache;
    p.num_blocks = num_blocks;
    p.latent_out = static_cast<uint16_t *>(latent_out);
    p.latent_out_stride = latent_out_stride;
    p.k_rope_out = static_cast<uint16_t *>(k_rope_out);
    p.k_rope_out_stride = k_rope_out_stride;
    if (status_address(&p.status) != MLA_OK) return MLA_ERR_CUDA;
    return result(launch_place_rows(p, d, e4m3, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

int mla_assign_pages(const int32_t *cache_seqlens, const int32_t *cu_rows, int batch, int64_t num_rows, int32_t *block_table,
                     int max_blocks_per_seq, const int32_t *free_pages, int64_t max_free, const int32_t *num_free,
                     int32_t *num_free_out, int32_t *new_seqlens, int32_t *positions, int64_t *slots,
                     struct CUstream_st *stream) {
    if (!cache_seqlens || !cu_rows || !block_table || !free_pages || !num_free || !num_free_out || !new_seqlens)
        return MLA_ERR_INVALID_ARG;
    if (batch < 1 || num_rows < 0 || max_blocks_per_seq < 1 || max_free < 1) return MLA_ERR_INVALID_ARG;
    if ((long long)max_blocks_per_seq * kPage > 0x7fffffffLL) return MLA_ERR_INVALID_ARG;
    if (num_rows > 0x7fffffffLL || max_free > 0x7fffffffLL) return MLA_ERR_UNSUPPORTED;
    Range range("mla_assign_pages");
    AssignPagesParams p{};
    p.seqlens = cache_seqlens;
    p.cu_rows = cu_rows;
    p.batch = batch;
    p.num_rows = num_rows;
    p.block_table = block_table;
    p.max_blocks = max_blocks_per_seq;
    p.free_pages = free_pages;
    p.max_free = max_free;
    p.num_free = num_free;
    p.num_free_out = num_free_out;
    p.new_seqlens = new_seqlens;
    p.positions = positions;
    p.slots = slots;
    if (status_address(&p.status) != MLA_OK) return MLA_ERR_CUDA;
    return result(launch_assign_pages(p, reinterpret_cast<cudaStream_t>(stream)));
}

int mla_release_pages(int32_t *cache_seqlens, const int32_t *finished, int batch, int32_t *block_table, int max_blocks_per_seq,
                      int64_t num_blocks, int32_t *free_pages, int64_t max_free, int32_t *num_free, struct CUstream_st *stream) {
    if (!cache_seqlens || !finished || !block_table || !free_pages || !num_free) return MLA_ERR_INVALID_ARG;
    if (batch < 1 || max_blocks_per_seq < 1 || num_blocks < 1 || max_free < 1) return MLA_ERR_INVALID_ARG;
    if ((long long)max_blocks_per_seq * kPage > 0x7fffffffLL) return MLA_ERR_INVALID_ARG;
    if (max_free > 0x7fffffffLL) return MLA_ERR_UNSUPPORTED;
    Range range("mla_release_pages");
    ReleasePagesParams p{};
    p.seqlens = cache_seqlens;
    p.finished = finished;
    p.batch = batch;
    p.block_table = block_table;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.free_pages = free_pages;
    p.max_free = max_free;
    p.num_free = num_free;
    if (status_address(&p.status) != MLA_OK) return MLA_ERR_CUDA;
    return result(launch_release_pages(p, reinterpret_cast<cudaStream_t>(stream)));
}

int mla_rope_turns(int rope_dim, double base, double factor, int original_positions, double fast_turns, double slow_turns,
                   int64_t *turns) {
    if (!turns || rope_dim < 2 || rope_dim % 2 || original_positions < 0) return MLA_ERR_INVALID_ARG;
    if (!(base > 1.0) || !(factor >= 1.0) || !std::isfinite(base) || !std::isfinite(factor)) return MLA_ERR_INVALID_ARG;
    if (original_positions > 0 && (!(slow_turns > 0.0) || !(fast_turns >= slow_turns) || !std::isfinite(fast_turns)))
        return MLA_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925286766559;
    auto pair = [&](double t) { return rope_dim * std::log(original_positions / (two_pi * t)) / (2.0 * std::log(base)); };
    double lo = 0.0, span = 1.0;
    if (original_positions > 0) {
        lo = std::fmax(0.0, std::floor(pair(fast_turns)));
        span = std::fmax(std::fmin(rope_dim - 1.0, std::ceil(pair(slow_turns))) - lo, 0.001);
    }
    for (int i = 0; i < rope_dim / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rope_dim);
        const double r = original_positions > 0 ? std::fmin(1.0, std::fmax(0.0, (i - lo) / span)) : 1.0;
        // below 2^62: a frequency is at most one radian
        turns[i] = std::llround((f / factor * r + f * (1.0 - r)) / two_pi * 0x1p64);
    }
    return MLA_OK;
}

int mla_norm_rope(const void *x, int64_t x_token_stride, int64_t x_head_stride, int64_t num_tokens, int heads, int d,
                  const void *weight, float eps, const int32_t *positions, const int64_t *turns, int rope_dim, int interleaved,
                  float rope_scale, void *out, int64_t out_token_stride, int64_t out_head_stride, struct CUstream_st *stream) {
    if (num_tokens < 0 || heads < 1 || d < 1 || rope_dim < 0) return MLA_ERR_INVALID_ARG;
    if (d % 8 || d > kMaxHeadDim || rope_dim % 16 || rope_dim > d || rope_dim > kMaxRopeDim) return MLA_ERR_UNSUPPORTED;
    if (num_tokens > 0x7fffffffLL || (long long)num_tokens * heads > (1LL << 35)) return MLA_ERR_UNSUPPORTED;
    if (num_tokens > 0 && (!x || !out || (rope_dim > 0 && (!positions || !turns)))) return MLA_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !real(eps) || (rope_dim > 0 && !real(rope_scale))) return MLA_ERR_INVALID_ARG;
    if (!rows_ok(x, x_token_stride, 0, false) || !rows_ok(x, x_head_stride, 0, false) || !aligned16(weight)) return MLA_ERR_INVALID_ARG;
    // written rows must not overlap: heads inside a token, or tokens inside a head
    const bool inside = out_head_stride >= d && out_token_stride >= (int64_t)(heads - 1) * out_head_stride + d;
    const bool across = out_token_stride >= d && out_head_stride >= (num_tokens - 1) * out_token_stride + d;
    if (!rows_ok(out, out_token_stride, 0, false) || !rows_ok(out, out_head_stride, 0, false) || (!inside && !across && num_tokens > 0))
        return MLA_ERR_INVALID_ARG;
    const bool in_place = x == out;
    if (in_place && (x_token_stride != out_token_stride || x_head_stride != out_head_stride)) return MLA_ERR_INVALID_ARG;
    if (num_tokens == 0) return MLA_OK;
    if (!weight && rope_dim == 0 && in_place) return MLA_OK;
    Range range("mla_norm_rope");
    NormRopeParams p{};
    p.x = static_cast<const uint16_t *>(x);
    p.x_token = x_token_stride;
    p.x_head = x_head_stride;
    p.out = static_cast<uint16_t *>(out);
    p.out_token = out_token_stride;
    p.out_head = out_head_stride;
    p.weight = static_cast<const uint16_t *>(weight);
    p.eps = eps;
    p.tokens = num_tokens;
    p.heads = heads;
    p.d = d;
    p.first = in_place && !weight ? d - rope_dim : 0;  // in place without a norm the rest stays as it is
    p.rope = {rope_dim > 0 ? positions : nullptr, turns, rope_dim, interleaved != 0, rope_scale};
    return result(launch_norm_rope(p, reinterpret_cast<cudaStream_t>(stream)));
}

int mla_norm_rope_cache_write(const void *latent, int64_t latent_stride, const void *k_rope, int64_t k_rope_stride,
                              int64_t num_rows, const void *weight, float eps, const int32_t *positions, const int64_t *turns,
                              int interleaved, float rope_scale, const int64_t *slots, void *kcache, int64_t num_blocks, int d,
                              void *latent_out, int64_t latent_out_stride, void *k_rope_out, int64_t k_rope_out_stride,
                              struct CUstream_st *stream) {
    return place_rows(latent, latent_stride, k_rope, k_rope_stride, num_rows, weight, eps, positions, turns, interleaved, rope_scale,
                      slots, kcache, num_blocks, d, latent_out, latent_out_stride, k_rope_out, k_rope_out_stride, false, stream);
}

int mla_norm_rope_cache_write_fp8(const void *latent, int64_t latent_stride, const void *k_rope, int64_t k_rope_stride,
                                  int64_t num_rows, const void *weight, float eps, const int32_t *positions,
                                  const int64_t *turns, int interleaved, float rope_scale, const int64_t *slots, void *kv_pages,
                                  int64_t num_blocks, int d, void *latent_out, int64_t latent_out_stride, void *k_rope_out,
                                  int64_t k_rope_out_stride, struct CUstream_st *stream) {
    return place_rows(latent, latent_stride, k_rope, k_rope_stride, num_rows, weight, eps, positions, turns, interleaved, rope_scale,
                      slots, kv_pages, num_blocks, d, latent_out, latent_out_stride, k_rope_out, k_rope_out_stride, true, stream);
}

}  // extern "C"
