// Shared by the prompt attention's partition, kernel and combine.
#pragma once

#include <stdint.h>

#include "mla_internal.h"

namespace mla {

constexpr int kPreTile = 128;                 // rows of a query tile, keys of a step
constexpr int kPreTiles = 2;                  // query tiles of a block
constexpr int kPreRows = kPreTile * kPreTiles;
constexpr int kPreHead = MLA_PREFILL_HEAD_DIM;
constexpr int kPreRope = kDqk - kDv;

// A block of query tokens of one sequence, the same for every key head.
struct PreBlock {
    int q0, tokens;     // first query row, and tokens of the block
    int k0, keys;       // first key row, and keys of the sequence
    int seen;           // keys that the first token sees (the next one more, causal); or at least keys for all
    int steps;          // 128-key steps that its last token needs
    int pad[2];
};
// A place on the line of all items (block, key head), heads inside blocks.
struct PrePlace {
    int block, head, step, pad;
};
// An item whose steps several CTAs share: its parts' slots are slot0, 2 cta, 2 (cta + 1),
// .. (count in all).
struct PreCut {
    int block, head, slot0, cta, count, pad[3];
};
// Work of a call, as int32 words: a header, the blocks (most steps first), where each
// CTA begins on the line (line only), the cut items (line only).
struct PreHeader {
    int blocks, line, cuts, pad[5];
};

// tokens of a query tile: its 128 rows hold `group` heads per token
__host__ __device__ constexpr int pre_tile_tokens(int group) { return kPreTile / group; }
__host__ __device__ inline int64_t pre_max_blocks(int64_t num_q, int batch, int group) {
    const int64_t t = kPreTiles * pre_tile_tokens(group);
    return num_q / t + (num_q < batch ? num_q : batch);
}
// More rounds of whole items than this are even enough: the line is not considered.  By
// the most blocks that a call can have, which the host knows: it then leaves out the
// combine.
constexpr int kPreRounds = 8;
__host__ __device__ inline bool pre_line(int64_t max_blocks, int h_kv, int ctas) { return max_blocks * h_kv <= (int64_t)kPreRounds * ctas; }
// slots of partial results: a CTA's first and last item may be cut
__host__ __device__ constexpr int pre_slots(int ctas) { return 2 * ctas; }
// keys that token i of a block sees
__host__ __device__ inline int pre_seen(const PreBlock &b, int i) {
    const long long n = (long long)b.seen + i;
    return n < 0 ? 0 : n > b.keys ? b.keys : (int)n;
}
__host__ __device__ inline int pre_steps(int keys) { return keys / kPreTile + (keys % kPreTile != 0); }

struct PreWork {
    PreHeader *header;
    PreBlock *blocks;
    PrePlace *places;  // [ctas + 1]
    PreCut *cuts;      // [ctas]
    __host__ __device__ PreWork(int32_t *metadata, int64_t max_blocks, int ctas) {
        header = reinterpret_cast<PreHeader *>(metadata);
        blocks = reinterpret_cast<PreBlock *>(header + 1);
        places = reinterpret_cast<PrePlace *>(blocks + max_blocks);
        cuts = reinterpret_cast<PreCut *>(places + ctas + 1);
    }
};
__host__ __device__ inline size_t pre_words(int64_t max_blocks, int ctas) {
    return (sizeof(PreHeader) + max_blocks * sizeof(PreBlock) + (ctas + 1) * sizeof(PrePlace) + ctas * sizeof(PreCut)) / sizeof(int32_t);
}

// Rounds of whole items: heads go in chunks, a chunk's blocks longest first with its heads
// side by side, so that the CTAs of a moment share few heads' keys (in L2) and the
// last items are short.  Every other round runs backwards over the CTAs: over lengths
// that fall, each gets its share.
__host__ __device__ inline bool pre_round_item(int64_t round, int cta, int ctas, int blocks, int h_kv, int chunk, int &block, int &head) {
    const int64_t items = (int64_t)blocks * h_kv, first = round * ctas;
    if (first + cta >= items) return false;
    const int64_t last = items - 1 < first + ctas - 1 ? items - 1 : first + ctas - 1;
    const int64_t i = round & 1 ? last - cta : first + cta;
    const int64_t per = (int64_t)blocks * chunk;
    int c = 0;
    if (i >= per) c = items <= 0x7fffffff ? (int)((uint32_t)i / (uint32_t)per) : (int)(i / per);
    const int heads = chunk < h_kv - c * chunk ? chunk : h_kv - c * chunk;
    const int64_t in = i - c * per;
    block = in <= 0x7fffffff ? (int)((uint32_t)in / (uint32_t)heads) : (int)(in / heads);
    head = c * chunk + (int)(in - (int64_t)block * heads);
    return true;
}

}  // namespace mla
