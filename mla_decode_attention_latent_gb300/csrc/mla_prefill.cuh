// Shared by the prompt attention's partition, kernel and combine.
#pragma once

#include <stdint.h>

#include "mla_internal.h"

namespace mla {

constexpr int kPreTile = 128;                 // rows of a query tile, keys of a step
constexpr int kPreTiles = 2;                  // query tiles of a block
constexpr int kPreHead = MLA_PREFILL_HEAD_DIM;
constexpr int kPreRope = kDqk - kDv;

// One unit of work, for every key head: a block of query tokens over a range of
// key steps.
struct PreSegment {
    int q0, tokens;     // first query row, and tokens of the block
    int k0, keys;       // first key row, and keys of the sequence
    int seen;           // keys that the first token sees (the next one more, causal); or at least keys for all
    int step0, step1;   // 128-key steps
    int slot;           // of the partial results; -1: the only segment of its block
};
// A block whose steps were cut: its slots are slot0 .. slot0 + count - 1.
struct PreCut {
    int q0, tokens, slot0, count;
};
// Work of a call, as int32 words: a header, segments (most steps first), cut blocks.
struct PreHeader {
    int segments, cuts, pad[6];
};

// tokens of a query tile: its 128 rows hold `group` heads per token
__host__ __device__ constexpr int pre_tile_tokens(int group) { return kPreTile / group; }
// slots of the partial results: a cut block of s steps has ceil(s / c) of them, fewer
// than 2 s / c, and c is at least (all steps) * h_kv / sms
__host__ __device__ constexpr int pre_max_slots(int sms, int h_kv) { return 2 * sms / h_kv; }
__host__ __device__ inline int64_t pre_max_blocks(int64_t num_q, int batch, int group) {
    const int64_t t = kPreTiles * pre_tile_tokens(group);
    return num_q / t + (num_q < batch ? num_q : batch);
}
__host__ __device__ inline int64_t pre_max_segments(int64_t num_q, int batch, int group, int sms, int h_kv) {
    return pre_max_blocks(num_q, batch, group) + pre_max_slots(sms, h_kv);
}
// keys that token i of a block sees
__host__ __device__ inline int pre_seen(const PreSegment &s, int i) {
    const long long n = (long long)s.seen + i;
    return n < 0 ? 0 : n > s.keys ? s.keys : (int)n;
}
__host__ __device__ inline int pre_steps(int keys) { return keys / kPreTile + (keys % kPreTile != 0); }

}  // namespace mla
