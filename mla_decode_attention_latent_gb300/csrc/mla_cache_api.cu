// C ABI of the cache calls: rows in and out of the pages, page keys, and the
// decode over selected pages.  See include/mla_decode.h for each contract.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "mla_internal.h"

namespace mla {
namespace {

struct Range {
    explicit Range(const char *name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
constexpr int kMaxDecodeBatch = 65535;  // sequences of one decode call
constexpr int kMaxDecodeHeads = 16384;  // 128 row tiles each: below the 2^24 tiles of one call

int result(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA; }

// the checks that every call over a paged cache shares
int check_cache(const void *cache, int64_t num_blocks, const int32_t *block_table, int max_blocks, int batch, int d,
                bool e4m3) {
    if (!cache || !block_table || num_blocks < 1 || max_blocks < 1 || batch < 1 || d < 1) return MLA_ERR_INVALID_ARG;
    if ((long long)max_blocks * kPage > 0x7fffffffLL || !aligned16(cache)) return MLA_ERR_INVALID_ARG;
    if (d != kDqk && (e4m3 || d != kDv)) return MLA_ERR_UNSUPPORTED;
    return MLA_OK;
}

int cache_rows(void *latent, int64_t latent_stride, void *k_rope, int64_t k_rope_stride, int64_t num_rows,
               const int32_t *cu_rows, const int32_t *starts, int batch, void *cache, int64_t num_blocks,
               const int32_t *block_table, int max_blocks, int d, bool e4m3, bool write, struct CUstream_st *stream) {
    int st = check_cache(cache, num_blocks, block_table, max_blocks, batch, d, e4m3);
    if (st != MLA_OK) return st;
    if (!starts || num_rows < 0) return MLA_ERR_INVALID_ARG;
    if (num_rows > 0 && (!latent || (d > kDv && !k_rope))) return MLA_ERR_INVALID_ARG;  // empty buffers may be null
    if (num_rows > 0x7fffffffLL) return MLA_ERR_UNSUPPORTED;
    if (!cu_rows && num_rows % batch) return MLA_ERR_INVALID_ARG;
    // 16-byte accesses; rows that overlap can be read but not written
    const int64_t least = write ? 0 : kDv, least_rope = write ? 0 : kDqk - kDv;
    if (!aligned16(latent) || latent_stride < least || latent_stride % 8) return MLA_ERR_INVALID_ARG;
    if (d > kDv && (!aligned16(k_rope) || k_rope_stride < least_rope || k_rope_stride % 8)) return MLA_ERR_INVALID_ARG;
    if (num_rows == 0) return MLA_OK;
    Range range(write ? "mla_cache_write" : "mla_cache_read");
    CacheRowsParams p{};
    p.latent = static_cast<uint16_t *>(latent);
    p.latent_stride = latent_stride;
    p.rope = static_cast<uint16_t *>(k_rope);
    p.rope_stride = k_rope_stride;
    p.num_rows = num_rows;
    p.cu_rows = cu_rows;
    p.rows_per_seq = num_rows / batch;
    p.starts = starts;
    p.batch = batch;
    p.cache = cache;
    p.num_blocks = num_blocks;
    p.block_table = block_table;
    p.max_blocks = max_blocks;
    if (status_address(&p.status) != MLA_OK) return MLA_ERR_CUDA;
    return result(launch_cache_rows(p, d, e4m3, write, reinterpret_cast<cudaStream_t>(stream)));
}

int update_page_keys(const void *cache, int64_t num_blocks, const int32_t *block_table, int max_blocks,
                     const int32_t *cache_seqlens, const int32_t *starts, int batch, int d, int8_t *page_keys,
                     float *page_scales, bool e4m3, struct CUstream_st *stream) {
    int st = check_cache(cache, num_blocks, block_table, max_blocks, batch, d, e4m3);
    if (st != MLA_OK) return st;
    if (!cache_seqlens || !page_keys || !page_scales || !aligned16(page_keys)) return MLA_ERR_INVALID_ARG;
    Range range("mla_update_page_keys");
    PageKeysParams p{};
    p.cache = cache;
    p.num_blocks = num_blocks;
    p.block_table = block_table;
    p.max_blocks = max_blocks;
    p.seqlens = cache_seqlens;
    p.starts = starts;
    p.batch = batch;
    p.keys = page_keys;
    p.scales = page_scales;
    if (status_address(&p.status) != MLA_OK) return MLA_ERR_CUDA;
    return result(launch_page_keys(p, d, e4m3, reinterpret_cast<cudaStream_t>(stream)));
}

// workspace of a page-selecting decode: the selection's arrays, then the decode's
struct BlocksLayout {
    size_t codes, units, scores, table, lens, metadata, splits, decode, total;
};

BlocksLayout blocks_layout(int tokens, int h_q, int max_blocks, int topk, int num_parts) {
    BlocksLayout l;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += align_up(bytes);
        return here;
    };
    l.codes = take((size_t)tokens * h_q * kDqk);
    l.units = take((size_t)tokens * h_q * sizeof(float));
    l.scores = take((size_t)tokens * max_blocks * sizeof(float));
    l.table = take((size_t)tokens * topk * sizeof(int32_t));
    l.lens = take((size_t)tokens * sizeof(int32_t));
    l.metadata = take((size_t)num_parts * kMdInts * sizeof(int32_t));
    const int entries = tokens * ((h_q + MLA_TILE_ROWS - 1) / MLA_TILE_ROWS);
    l.splits = take(((size_t)entries + 1) * sizeof(int32_t));
    l.decode = take(workspace_bytes(entries, MLA_TILE_ROWS, num_parts));
    l.total = at;
    return l;
}

int decode_blocks(const void *q, const void *cache, int64_t num_blocks, const int32_t *block_table, int max_blocks,
                  const int32_t *cache_seqlens, const int8_t *page_keys, const float *page_scales, int topk, int sink,
                  int local, int batch, int s_q, int h_q, int h_kv, int d, int dv, int num_parts, float softmax_scale,
                  int causal, void *o, float *lse, int32_t *pages, void *workspace, size_t ws_bytes, bool e4m3,
                  struct CUstream_st *stream) {
    int st = check_cache(cache, num_blocks, block_table, max_blocks, batch, d, e4m3);
    if (st != MLA_OK) return st;
    if (!q || !cache_seqlens || !page_keys || !page_scales || !o || !lse || !pages || !workspace) return MLA_ERR_INVALID_ARG;
    if (s_q < 1 || h_q < 1 || h_kv < 1 || dv < 1 || num_parts < 1) return MLA_ERR_INVALID_ARG;
    if (topk < 1 || sink < 0 || local < 1 || (long long)sink + local > topk) return MLA_ERR_INVALID_ARG;
    // the selection ranks q . k, which is the order of the scaled scores for a positive scale only
    if (!(softmax_scale > 0.f)) return MLA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(page_keys) || !aligned16(o) || (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)))
        return MLA_ERR_INVALID_ARG;
    if (dv != kDv || h_kv != 1) return MLA_ERR_UNSUPPORTED;
    if ((long long)batch * s_q > kMaxDecodeBatch || h_q > kMaxDecodeHeads || (long long)topk * kPage > 0x7fffffffLL)
        return MLA_ERR_UNSUPPORTED;
    const int tokens = batch * s_q;
    const BlocksLayout l = blocks_layout(tokens, h_q, max_blocks, topk, num_parts);
    if (ws_bytes < l.total) return MLA_ERR_WORKSPACE;
    Range range("mla_decode_kvcache_blocks");
    char *ws = static_cast<char *>(workspace);
    SelectParams p{};
    p.q = static_cast<const uint16_t *>(q);
    p.keys = page_keys;
    p.scales = page_scales;
    p.num_blocks = num_blocks;
    p.block_table = block_table;
    p.max_blocks = max_blocks;
    p.seqlens = cache_seqlens;
    p.batch = batch;
    p.s_q = s_q;
    p.h_q = h_q;
    p.d = d;
    p.topk = topk;
    p.sink = sink;
    p.local = local;
    p.causal = causal != 0;
    p.q_codes = reinterpret_cast<int8_t *>(ws + l.codes);
    p.q_units = reinterpret_cast<float *>(ws + l.units);
    p.scores = reinterpret_cast<float *>(ws + l.scores);
    p.sel_table = reinterpret_cast<int32_t *>(ws + l.table);
    p.sel_lens = reinterpret_cast<int32_t *>(ws + l.lens);
    p.pages = pages;
    p.num_parts = num_parts;
    p.metadata = reinterpret_cast<int32_t *>(ws + l.metadata);
    p.num_splits = reinterpret_cast<int32_t *>(ws + l.splits);
    if (status_address(&p.status) != MLA_OK) return MLA_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // without more pages than topk there is nothing to score
    if (max_blocks > topk && launch_page_scores(p, s) != cudaSuccess) return MLA_ERR_CUDA;
    if (launch_select_pages(p, s) != cudaSuccess) return MLA_ERR_CUDA;
    // one "sequence" per query token over its own block table
    return decode_tiled(q, cache, e4m3, num_blocks, p.sel_table, topk, p.sel_lens, tokens, h_q, d, p.metadata, p.num_splits,
                        num_parts, softmax_scale, o, lse, ws + l.decode, ws_bytes - l.decode, stream);
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

int mla_cache_write(const void *latent, int64_t latent_stride, const void *k_rope, int64_t k_rope_stride,
                    int64_t num_rows, const int32_t *cu_rows, const int32_t *starts, int batch, void *kcache,
                    int64_t num_blocks, const int32_t *block_table, int max_blocks_per_seq, int d,
                    struct CUstream_st *stream) {
    return cache_rows(const_cast<void *>(latent), latent_stride, const_cast<void *>(k_rope), k_rope_stride, num_rows,
                      cu_rows, starts, batch, kcache, num_blocks, block_table, max_blocks_per_seq, d, false, true, stream);
}

int mla_cache_write_fp8(const void *latent, int64_t latent_stride, const void *k_rope, int64_t k_rope_stride,
                        int64_t num_rows, const int32_t *cu_rows, const int32_t *starts, int batch, void *kv_pages,
                        int64_t num_blocks, const int32_t *block_table, int max_blocks_per_seq, int d,
                        struct CUstream_st *stream) {
    return cache_rows(const_cast<void *>(latent), latent_stride, const_cast<void *>(k_rope), k_rope_stride, num_rows,
                      cu_rows, starts, batch, kv_pages, num_blocks, block_table, max_blocks_per_seq, d, true, true, stream);
}

int mla_cache_read(const void *kcache, int64_t num_blocks, const int32_t *block_table, int max_blocks_per_seq,
                   const int32_t *starts, const int32_t *cu_rows, int batch, int64_t num_rows, void *latent,
                   int64_t latent_stride, void *k_rope, int64_t k_rope_stride, int d, struct CUstream_st *stream) {
    return cache_rows(latent, latent_stride, k_rope, k_rope_stride, num_rows, cu_rows, starts, batch,
                      const_cast<void *>(kcache), num_blocks, block_table, max_blocks_per_seq, d, false, false, stream);
}

int mla_cache_read_fp8(const void *kv_pages, int64_t num_blocks, const int32_t *block_table, int max_blocks_per_seq,
                       const int32_t *starts, const int32_t *cu_rows, int batch, int64_t num_rows, void *latent,
                       int64_t latent_stride, void *k_rope, int64_t k_rope_stride, int d, struct CUstream_st *stream) {
    return cache_rows(latent, latent_stride, k_rope, k_rope_stride, num_rows, cu_rows, starts, batch,
                      const_cast<void *>(kv_pages), num_blocks, block_table, max_blocks_per_seq, d, true, false, stream);
}

int mla_update_page_keys(const void *kcache, int64_t num_blocks, const int32_t *block_table, int max_blocks_per_seq,
                         const int32_t *cache_seqlens, const int32_t *starts, int batch, int d, int8_t *page_keys,
                         float *page_scales, struct CUstream_st *stream) {
    return update_page_keys(kcache, num_blocks, block_table, max_blocks_per_seq, cache_seqlens, starts, batch, d,
                            page_keys, page_scales, false, stream);
}

int mla_update_page_keys_fp8(const void *kv_pages, int64_t num_blocks, const int32_t *block_table, int max_blocks_per_seq,
                             const int32_t *cache_seqlens, const int32_t *starts, int batch, int d, int8_t *page_keys,
                             float *page_scales, struct CUstream_st *stream) {
    return update_page_keys(kv_pages, num_blocks, block_table, max_blocks_per_seq, cache_seqlens, starts, batch, d,
                            page_keys, page_scales, true, stream);
}

size_t mla_blocks_workspace_bytes(int batch, int s_q, int h_q, int h_kv, int dv, int max_blocks_per_seq, int topk_pages,
                                  int num_parts) {
    if (batch < 1 || s_q < 1 || h_q < 1 || h_kv != 1 || dv != kDv || max_blocks_per_seq < 1 || topk_pages < 1 || num_parts < 1)
        return 0;
    if ((long long)batch * s_q > kMaxDecodeBatch || h_q > kMaxDecodeHeads) return 0;
    return blocks_layout(batch * s_q, h_q, max_blocks_per_seq, topk_pages, num_parts).total;
}

int mla_decode_kvcache_blocks(const void *q, const void *kcache, int64_t num_blocks, const int32_t *block_table,
                              int max_blocks_per_seq, const int32_t *cache_seqlens, const int8_t *page_keys,
                              const float *page_scales, int topk_pages, int sink_pages, int local_pages, int batch,
                              int s_q, int h_q, int h_kv, int d, int dv, int num_parts, float softmax_scale, int causal,
                              void *o, float *lse, int32_t *pages, void *workspace, size_t ws_bytes,
                              struct CUstream_st *stream) {
    return decode_blocks(q, kcache, num_blocks, block_table, max_blocks_per_seq, cache_seqlens, page_keys, page_scales,
                         topk_pages, sink_pages, local_pages, batch, s_q, h_q, h_kv, d, dv, num_parts, softmax_scale,
                         causal, o, lse, pages, workspace, ws_bytes, false, stream);
}

int mla_decode_kvcache_blocks_fp8(const void *q, const void *kv_pages, int64_t num_blocks, const int32_t *block_table,
                                  int max_blocks_per_seq, const int32_t *cache_seqlens, const int8_t *page_keys,
                                  const float *page_scales, int topk_pages, int sink_pages, int local_pages, int batch,
                                  int s_q, int h_q, int h_kv, int d, int dv, int num_parts, float softmax_scale, int causal,
                                  void *o, float *lse, int32_t *pages, void *workspace, size_t ws_bytes,
                                  struct CUstream_st *stream) {
    return decode_blocks(q, kv_pages, num_blocks, block_table, max_blocks_per_seq, cache_seqlens, page_keys, page_scales,
                         topk_pages, sink_pages, local_pages, batch, s_q, h_q, h_kv, d, dv, num_parts, softmax_scale,
                         causal, o, lse, pages, workspace, ws_bytes, true, stream);
}

}  // extern "C"
