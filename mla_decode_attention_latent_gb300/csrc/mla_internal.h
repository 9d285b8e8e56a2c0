// Internal host-side interface between the C-ABI layer (mla_api.cu) and the
// kernel translation units.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "mla_decode.h"

namespace mla {

constexpr int kPage = MLA_PAGE_SIZE;       // tokens per cache page
constexpr int kDqk = MLA_HEAD_DIM;         // 512 latent + 64 RoPE dims
constexpr int kDv = MLA_V_DIM;             // value dims = first 512 dims of a row
constexpr int kMdInts = MLA_METADATA_INTS;
constexpr int kFixedCost = MLA_SCHED_FIXED_COST_PAGES;
constexpr int kCombineCost = MLA_SCHED_COMBINE_COST_PAGES;

// Everything a split-KV kernel needs for one decode call.
struct DecodeParams {
    const uint16_t *q;            // [batch][s_q][h_q][576] bf16
    const uint16_t *kcache;       // [num_blocks][64][1][576] bf16, or packed e4m3 pages (read as bytes)
    int64_t num_blocks;
    const int32_t *block_table;   // [batch][max_blocks]
    int max_blocks;
    const int32_t *seqlens;       // [batch]
    int batch, s_q, h_q;
    int rows;                     // s_q * h_q query rows per sequence
    const int32_t *metadata;      // [num_parts][8]
    const int32_t *num_splits;    // [batch + 1]
    int num_parts;
    int max_splits;               // batch + num_parts: capacity of the workspace
    float scale_log2;             // softmax_scale * log2(e)
    int causal;
    uint16_t *o;                  // [batch][s_q][h_q][512] bf16
    float *lse;                   // [batch][s_q][h_q]
    float *o_accum;               // [max_splits][rows][512] fp32 partial outputs
    float *lse_accum;             // [max_splits][rows] partial LSE (natural log)
    unsigned int *status;         // device status word (MLA_DEVERR_* bits)
    // sparse top-k decode only (seqlens then holds each sequence's list length)
    const int32_t *indices;       // [batch][s_q][topk] token positions per query token
    int topk;
    const int32_t *kv_lens;       // [batch] cache lengths: positions >= kv_lens[b] are ignored
    // draft-tree decode only
    const uint32_t *tree_mask;    // [batch][s_q][tree_words]: bit j of row i: node i sees node j
    int tree_words;               // ceil(s_q / 32)
    int tiles;                    // 128-row tiles of a sequence: the work line's entries
    const int32_t *tree_lens;     // [batch] nodes of each sequence, or null: s_q everywhere
};

// One call that writes or reads ragged rows of the paged cache.
struct CacheRowsParams {
    uint16_t *latent;             // [num_rows] rows of 512 bf16 (input of a write, output of a read)
    int64_t latent_stride;        // elements between rows
    uint16_t *rope;               // [num_rows] rows of 64 bf16 (d = 576)
    int64_t rope_stride;
    int64_t num_rows;
    const int32_t *cu_rows;       // [batch + 1] first row of each sequence, or null: rows_per_seq each
    int64_t rows_per_seq;
    const int32_t *starts;        // [batch] position of each sequence's first row
    int batch;
    void *cache;                  // bf16 [num_blocks][64][d] or packed e4m3 pages
    int64_t num_blocks;
    const int32_t *block_table;   // [batch][max_blocks]
    int max_blocks;
    unsigned int *status;
};

// One call that recomputes the keys of the pages that [starts[b], seqlens[b]) touches.
struct PageKeysParams {
    const void *cache;
    int64_t num_blocks;
    const int32_t *block_table;   // [batch][max_blocks]
    int max_blocks;
    const int32_t *seqlens;       // [batch]
    const int32_t *starts;        // [batch], or null: 0 everywhere
    int batch;
    int8_t *keys;                 // [num_blocks][d]
    float *scales;                // [num_blocks]
    unsigned int *status;
};

// One call that scores the pages of each query token, selects topk of them and
// partitions the decode over the selection.
struct SelectParams {
    const uint16_t *q;            // [batch][s_q][h_q][d] bf16
    const int8_t *keys;           // [num_blocks][d]
    const float *scales;          // [num_blocks]
    int64_t num_blocks;
    const int32_t *block_table;   // [batch][max_blocks]
    int max_blocks;
    const int32_t *seqlens;       // [batch]
    int batch, s_q, h_q, d;
    int topk, sink, local;
    int causal;
    int8_t *q_codes;              // workspace [batch * s_q][h_q][d]: the heads, quantised
    float *q_units;               // workspace [batch * s_q][h_q]: their scales
    float *scores;                // workspace [batch * s_q][max_blocks]
    int32_t *sel_table;           // workspace [batch * s_q][topk]: physical pages, the block table of the decode
    int32_t *sel_lens;            // workspace [batch * s_q]: lengths over the selected pages
    int32_t *pages;               // [batch][s_q][topk], out: logical pages, ascending, -1 behind them
    int num_parts;                // of the decode's work partition
    int32_t *metadata;            // workspace [num_parts][8]
    int32_t *num_splits;          // workspace [batch * s_q * row tiles + 1]
    unsigned int *status;
};

// Workspace carve-up shared by the API, the split kernel and the combine.
size_t workspace_bytes(int batch, int rows, int num_parts);
void carve_workspace(void *ws, int batch, int rows, int num_parts, float **o_accum, float **lse_accum);

cudaError_t launch_schedule(const int32_t *seqlens, int batch, int num_parts, int fixed_cost, int combine_cost,
                            int32_t *metadata, int32_t *num_splits, unsigned int *status, cudaStream_t stream);
// the tensor-core split-KV kernel for cached rows of width D (576 or 512), bf16
// rows or (E4M3, D = 576) packed e4m3 pages with per-token scales
template <int D, bool E4M3>
cudaError_t launch_split_kv_tc(const DecodeParams &p, cudaStream_t stream);
// the sparse top-k variant (576-wide bf16 rows gathered from index lists):
// the CTA pair splits each page's gathers with cluster multicast, or (local)
// each CTA gathers its own rows
cudaError_t launch_split_kv_tc_sparse(const DecodeParams &p, cudaStream_t stream);
cudaError_t launch_split_kv_tc_sparse_local(const DecodeParams &p, cudaStream_t stream);
int split_kv_tc_tile_rows();
// CTA pairs of the split-KV kernel that fit on the current device at once
template <int D, bool E4M3>
cudaError_t split_kv_tc_max_pairs(int *pairs);
cudaError_t launch_combine(const DecodeParams &p, cudaStream_t stream);
// draft trees: work entries are row tiles (entry e: tile e % tiles of sequence e / tiles)
cudaError_t launch_schedule_tree(const int32_t *seqlens, const int32_t *tree_lens, int batch, int tiles, int tile_rows,
                                 int h_q, int num_parts, int32_t *metadata, int32_t *num_splits, unsigned int *status,
                                 cudaStream_t stream);
cudaError_t launch_combine_tree(const DecodeParams &p, int tile_rows, cudaStream_t stream);
// the same kernel over row tiles, with a draft tree's mask over the last rows of
// each sequence (tree_mask null: no masks)
template <int D, bool E4M3>
cudaError_t launch_split_kv_tc_tree(const DecodeParams &p, cudaStream_t stream);

cudaError_t launch_cache_rows(const CacheRowsParams &p, int d, bool e4m3, bool write, cudaStream_t stream);
cudaError_t launch_page_keys(const PageKeysParams &p, int d, bool e4m3, cudaStream_t stream);
cudaError_t launch_page_scores(const SelectParams &p, cudaStream_t stream);
cudaError_t launch_select_pages(const SelectParams &p, cudaStream_t stream);
cudaError_t launch_tree_mask(const int32_t *parents, int batch, int s_q, uint32_t *mask, unsigned int *status,
                             cudaStream_t stream);

// decode of one query token per sequence on the tree kernels, without masks:
// work entries are row tiles (partition: launch_schedule_tree)
int decode_tiled(const void *q, const void *cache, bool e4m3, int64_t num_blocks, const int32_t *block_table, int max_blocks,
                 const int32_t *seqlens, int batch, int h_q, int d, const int32_t *metadata, const int32_t *num_splits,
                 int num_parts, float softmax_scale, void *o, float *lse, void *workspace, size_t ws_bytes,
                 struct CUstream_st *stream);

// address of the status word on the current device (MLA_OK or MLA_ERR_CUDA)
int status_address(unsigned int **out);
// multiprocessors of the current device
cudaError_t device_sm_count(int *sms);

// Launch a kernel that may be scheduled while the one before it on the stream
// finishes; the kernel waits (griddepcontrol.wait) before it touches memory.
template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                         const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace mla
