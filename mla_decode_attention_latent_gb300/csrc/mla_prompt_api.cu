// C ABI of the prompt path: pages of requests, norms and rotations, rows placed
// into the cache.  See include/mla_decode.h for each contract.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cmath>

#include "mla_internal.h"
#include "mla_prefill.cuh"

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

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// shapes that a prompt attention takes
int prefill_shape(int batch, int64_t num_q, int h_q, int h_kv) {
    if (batch < 1 || num_q < 0 || h_q < 1 || h_kv < 1 || h_q % h_kv) return MLA_ERR_INVALID_ARG;
    if (h_q / h_kv > kPreTile || h_q > 16384 || num_q > 0x7fffffffLL / 2) return MLA_ERR_UNSUPPORTED;
    return MLA_OK;
}

// words of the partition, and the workspace: the partial results of cut items, then
// room for the partition when the caller brings none
struct PrefillLayout {
    int64_t max_blocks;
    size_t words, o_part, lse_part, metadata, total;
};

PrefillLayout prefill_layout(int batch, int64_t num_q, int group, int sms) {
    PrefillLayout l;
    l.max_blocks = pre_max_blocks(num_q, batch, group);
    l.words = pre_words(l.max_blocks, sms);
    const size_t rows = (size_t)pre_slots(sms) * kPreRows;
    l.o_part = 0;
    l.lse_part = align_up(rows * kPreHead * sizeof(float));
    l.metadata = l.lse_part + align_up(rows * sizeof(float));
    l.total = l.metadata + align_up(l.words * sizeof(int32_t));
    return l;
}

// key heads side by side: as many as keep their keys and values in half of L2
int prefill_head_chunk(int64_t num_k, int h_kv) {
    const int64_t side = (64LL << 20) / ((num_k > 0 ? num_k : 1) * 4 * kPreHead);
    return (int)(side < 1 ? 1 : side > h_kv ? h_kv : side);
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

int64_t mla_prefill_metadata_ints(int batch, int64_t num_q, int h_q, int h_kv) {
    int sms = 0;
    if (prefill_shape(batch, num_q, h_q, h_kv) != MLA_OK || device_sm_count(&sms) != cudaSuccess) return 0;
    return (int64_t)prefill_layout(batch, num_q, h_q / h_kv, sms).words;
}

size_t mla_prefill_workspace_bytes(int batch, int64_t num_q, int h_q, int h_kv) {
    int sms = 0;
    if (prefill_shape(batch, num_q, h_q, h_kv) != MLA_OK || device_sm_count(&sms) != cudaSuccess) return 0;
    return prefill_layout(batch, num_q, h_q / h_kv, sms).total;
}

int mla_get_metadata_prefill(const int32_t *cu_q, const int32_t *cu_k, int batch, int64_t num_q, int64_t num_k, int h_q, int h_kv,
                             int causal, int32_t *metadata, struct CUstream_st *stream) {
    const int st = prefill_shape(batch, num_q, h_q, h_kv);
    if (st != MLA_OK) return st;
    if (!cu_q || !cu_k || !metadata || num_k < 0) return MLA_ERR_INVALID_ARG;
    if (num_k > 0x7fffffffLL / 2) return MLA_ERR_UNSUPPORTED;
    Range range("mla_get_metadata_prefill");
    PrefillParams p{};
    if (device_sm_count(&p.sms) != cudaSuccess) return MLA_ERR_CUDA;
    p.cu_q = cu_q;
    p.cu_k = cu_k;
    p.batch = batch;
    p.num_q = num_q;
    p.num_k = num_k;
    p.h_q = h_q;
    p.h_kv = h_kv;
    p.group = h_q / h_kv;
    p.tile_tokens = pre_tile_tokens(p.group);
    p.causal = causal != 0;
    p.metadata = metadata;
    p.max_blocks = pre_max_blocks(num_q, batch, p.group);
    p.head_chunk = prefill_head_chunk(num_k, h_kv);
    if (status_address(&p.status) != MLA_OK) return MLA_ERR_CUDA;
    return result(launch_prefill_schedule(p, reinterpret_cast<cudaStream_t>(stream)));
}

int mla_prefill(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k, int64_t k_token_stride,
                int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride, const void *k_rope,
                int64_t k_rope_token_stride, const int32_t *cu_q, const int32_t *cu_k, int batch, int64_t num_q, int64_t num_k,
                int h_q, int h_kv, int d_qk, int d_v, float softmax_scale, int causal, const int32_t *metadata, void *out, float *lse,
                void *workspace, size_t workspace_bytes, struct CUstream_st *stream) {
    int st = prefill_shape(batch, num_q, h_q, h_kv);
    if (st != MLA_OK) return st;
    if (!cu_q || !cu_k || num_k < 0 || d_qk < 1 || d_v < 1) return MLA_ERR_INVALID_ARG;
    if (num_q > 0 && (!q || !out || !lse || !workspace)) return MLA_ERR_INVALID_ARG;
    if (num_q > 0 && num_k > 0 && (!k || !v)) return MLA_ERR_INVALID_ARG;
    if (num_k > 0x7fffffffLL / 2) return MLA_ERR_UNSUPPORTED;
    if (d_v != kPreHead || (d_qk != kPreHead && d_qk != kPreHead + kPreRope)) return MLA_ERR_UNSUPPORTED;
    const bool rope = d_qk > kPreHead;
    if (num_q > 0 && num_k > 0 && rope != (k_rope != nullptr)) return MLA_ERR_INVALID_ARG;  // empty tensors may be null
    // rows are ranked by raw scores, which is the order of the scaled ones for a positive scale only
    if (!(softmax_scale > 0.f) || !real(softmax_scale * 1.4426950408889634f)) return MLA_ERR_INVALID_ARG;
    auto heads = [](const void *ptr, int64_t token, int64_t head, int64_t n, int64_t h, int64_t d) {
        // 16-byte aligned heads that do not overlap, strides that a tensor map holds
        if (!aligned16(ptr) || token % 8 || head % 8 || token >= (1LL << 38) || head >= (1LL << 38)) return false;
        return (head >= d && token >= (h - 1) * head + d) || (token >= d && head >= (n - 1) * token + d);
    };
    if (num_q > 0 && !heads(q, q_token_stride, q_head_stride, num_q, h_q, d_qk)) return MLA_ERR_INVALID_ARG;
    if (num_q > 0 && num_k > 0) {
        if (!heads(k, k_token_stride, k_head_stride, num_k, h_kv, kPreHead)) return MLA_ERR_INVALID_ARG;
        if (!heads(v, v_token_stride, v_head_stride, num_k, h_kv, kPreHead)) return MLA_ERR_INVALID_ARG;
        if (rope && !heads(k_rope, k_rope_token_stride, kPreRope, num_k, 1, kPreRope)) return MLA_ERR_INVALID_ARG;
    }
    if ((reinterpret_cast<uintptr_t>(out) & 31) || (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1))) return MLA_ERR_INVALID_ARG;
    if (num_q == 0) return MLA_OK;
    PrefillParams p{};
    if (device_sm_count(&p.sms) != cudaSuccess) return MLA_ERR_CUDA;
    const PrefillLayout l = prefill_layout(batch, num_q, h_q / h_kv, p.sms);
    if (workspace_bytes < l.total) return MLA_ERR_WORKSPACE;
    Range range("mla_prefill");
    char *ws = static_cast<char *>(workspace);
    p.metadata = metadata ? const_cast<int32_t *>(metadata) : reinterpret_cast<int32_t *>(ws + l.metadata);
    if (!metadata) {
        st = mla_get_metadata_prefill(cu_q, cu_k, batch, num_q, num_k, h_q, h_kv, causal, p.metadata, stream);
        if (st != MLA_OK) return st;
    }
    p.q = static_cast<const uint16_t *>(q);
    p.q_token = q_token_stride;
    p.q_head = q_head_stride;
    p.k = static_cast<const uint16_t *>(k);
    p.k_token = k_token_stride;
    p.k_head = k_head_stride;
    p.v = static_cast<const uint16_t *>(v);
    p.v_token = v_token_stride;
    p.v_head = v_head_stride;
    p.k_rope = static_cast<const uint16_t *>(k_rope);
    p.k_rope_token = k_rope_token_stride;
    p.rope = rope;
    p.cu_q = cu_q;
    p.cu_k = cu_k;
    p.batch = batch;
    p.num_q = num_q;
    p.num_k = num_k;
    p.h_q = h_q;
    p.h_kv = h_kv;
    p.group = h_q / h_kv;
    p.tile_tokens = pre_tile_tokens(p.group);
    p.causal = causal != 0;
    p.scale = softmax_scale;
    p.scale_log2 = softmax_scale * 1.4426950408889634f;
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.max_blocks = l.max_blocks;
    p.o_part = reinterpret_cast<float *>(ws + l.o_part);
    p.lse_part = reinterpret_cast<float *>(ws + l.lse_part);
    p.head_chunk = prefill_head_chunk(num_k, h_kv);
    if (status_address(&p.status) != MLA_OK) return MLA_ERR_CUDA;
    return result(launch_prefill(p, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
