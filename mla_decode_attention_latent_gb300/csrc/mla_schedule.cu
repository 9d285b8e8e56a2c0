// Tile scheduler: cuts the (sequence, page) range of a decode batch into
// contiguous split-KV parts of near-equal cost.
//
// The usage page "FlashMLA란 무엇인가?" (section "FlashMLA 설치 및 사용", step 2
// "MLA 메타데이터 가져오기") computes tile_scheduler_metadata and num_splits
// from cache_seqlens once per decode step; every layer then reuses them.  The
// page names the outputs only; the partition below is this library's:
//   lay the sequences on one line of cost units, sequence b taking
//   c_b = F + n_b units (F = fixed cost of a segment, a call argument; n_b = ceil(T_b / 64)
//   pages) from S_b = c_0 + ... + c_{b-1}; Q = ceil(total / parts); part p
//   starts at unit p * Q.  A unit in a sequence's first F units maps to its
//   page 0, a later one to page (x - S_b - F); the last part ends at
//   (batch, 0).  A part that starts inside a sequence's pages pays F beyond
//   its Q units, so no part costs more than Q + F.
// Every part's bounds are independent of the others' (two binary searches
// over the prefix sums), so the whole partition is computed in parallel.
// Metadata row: {begin_seq, begin_page, end_seq, end_page, begin_split, 0, 0, 0}.
#include "mla_internal.h"
#include "mla_schedule.cuh"
#include "mla_sm103.cuh"

namespace mla {
namespace {

constexpr int kSchedThreads = 512;

// Lengths of the work line's entries.  A dense or sparse decode has one entry
// per sequence; a draft-tree decode one per row tile (entry e is tile
// e % tiles of sequence e / tiles), whose length is 0 when the tile holds only
// rows behind the sequence's tree.
struct Entries {
    const int32_t *seqlens;
    int tiles;                 // 1: entries are sequences
    int tile_rows, h_q;        // rows of a tile, rows of a query token
    const int32_t *tree_lens;  // or null: no row is behind a tree
    __device__ __forceinline__ int operator[](int e) const {
        if (tiles == 1 && !tree_lens) return seqlens[e];
        const int b = e / tiles, tile = e - b * tiles;
        const int t = seqlens[b];
        return tree_lens && t > 0 && tile * tile_rows / h_q >= tree_lens[b] ? 0 : t;
    }
};

__global__ void __launch_bounds__(kSchedThreads)
schedule_kernel(const Entries seqlens, int batch, int num_parts, int fixed_cost, int combine_cost,
                int32_t *__restrict__ metadata, int32_t *__restrict__ num_splits,
                unsigned int *status) {
    __shared__ ScheduleShared<kSchedThreads> shared;
    // the split-KV launch that follows may start its prologue now; it waits
    // for this grid to complete before it reads the partition
    if (threadIdx.x == 0) sm103::griddep_launch_dependents();
    sm103::griddep_wait();  // a draft tree's partition is a dependent launch itself
    schedule_body<false>(shared, seqlens, batch, num_parts, fixed_cost, combine_cost, metadata, num_splits, status);
}

}  // namespace

cudaError_t launch_schedule(const int32_t *seqlens, int batch, int num_parts, int fixed_cost, int combine_cost,
                            int32_t *metadata, int32_t *num_splits, unsigned int *status, cudaStream_t stream) {
    const Entries entries{seqlens, 1, 1, 1, nullptr};
    schedule_kernel<<<1, kSchedThreads, 0, stream>>>(entries, batch, num_parts, fixed_cost, combine_cost, metadata,
                                                     num_splits, status);
    return cudaGetLastError();
}

cudaError_t launch_schedule_tree(const int32_t *seqlens, const int32_t *tree_lens, int batch, int tiles, int tile_rows,
                                 int h_q, int num_parts, int32_t *metadata, int32_t *num_splits, unsigned int *status,
                                 cudaStream_t stream) {
    const Entries entries{seqlens, tiles, tile_rows, h_q, tree_lens};
    return launch_after(schedule_kernel, dim3(1), dim3(kSchedThreads), 0, stream, entries, batch * tiles, num_parts, kFixedCost,
                        kCombineCost, metadata, num_splits, status);
}

}  // namespace mla
