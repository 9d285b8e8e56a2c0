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

// One unit of work, for every key head: a block of query tokens of one sequence, over a
// range of key steps.
struct PreSegment {
    int q0, tokens;     // first query row, and tokens of the block
    int k0, keys;       // first key row, and keys of the sequence
    int seen;           // keys that the first token sees (the next one more, causal); or at least keys for all
    int step0, step1;   // 128-key steps
    int part;           // h_kv slots of partial results from here on, one per head; -1: all steps of the block
};
// A block whose steps were cut: its parts are part .. part + count - 1.
struct PreCut {
    int q0, tokens, part, count;
};
// Work of a call, as int32 words: a header, the segments (most steps first), the cut blocks.
struct PreHeader {
    int segments, cuts;
    int causal, group, h_kv;  // of the call that it was made for
    int pad[3];
};

// tokens of a query tile: its 128 rows hold `group` heads per token
__host__ __device__ constexpr int pre_tile_tokens(int group) { return kPreTile / group; }
__host__ __device__ inline int64_t pre_max_blocks(int64_t num_q, int batch, int group) {
    const int64_t t = kPreTiles * pre_tile_tokens(group);
    return num_q / t + (num_q < batch ? num_q : batch);
}
// Blocks are cut only where at most this many items (segment, key head) come to a CTA: more
// are even enough.  By the most blocks and steps that a call can have, which the host
// knows: it then leaves out the combine.
constexpr int kPreRounds = 8;
// Steps of calls that are left whole.  By the costs in mla_prefill_schedule.cu a lone block of 9 would be cut: 64
// rows over 1152 keys at 16 heads 13.5 us for 17.9 with a partition in hand, but where nothing is cut the search and
// the idle combine cost 1 to 4 us a call (one row of 128 heads over 1100 keys 26.4 for 22.2).
constexpr int kPreWhole = 9;
__host__ __device__ inline bool pre_may_cut(int64_t max_blocks, int64_t num_k, int h_kv, int ctas) {
    return max_blocks * h_kv <= (int64_t)kPreRounds * ctas && num_k > kPreWhole * kPreTile;
}
__host__ __device__ inline int64_t pre_max_segments(int64_t max_blocks, int ctas) {
    return max_blocks > kPreRounds * ctas ? max_blocks : kPreRounds * ctas;
}
// slots of partial results, each of one part and key head
__host__ __device__ constexpr int pre_slots(int ctas) { return 2 * ctas; }
// Whether a partition is one for such a call: of its mask and heads, with no more segments than there is room for,
// and with cuts only where the host enqueues the combine (it goes by this call's rows and keys, which may be
// padded otherwise than those that the partition was made for).
__device__ inline bool pre_fits(const PreHeader &h, const PrefillParams &p) {
    return h.causal == (int)p.causal && h.group == p.group && h.h_kv == p.h_kv && h.segments <= pre_max_segments(p.max_blocks, p.sms) &&
           (h.cuts <= 0 || pre_may_cut(p.max_blocks, p.num_k, p.h_kv, p.sms));
}
// keys that token i of a block sees
__host__ __device__ inline int pre_seen(const PreSegment &b, int i) {
    const long long n = (long long)b.seen + i;
    return n < 0 ? 0 : n > b.keys ? b.keys : (int)n;
}
__host__ __device__ inline int pre_steps(int keys) { return keys / kPreTile + (keys % kPreTile != 0); }

struct PreWork {
    PreHeader *header;
    PreSegment *segments;
    PreCut *cuts;  // [slots]
    __host__ __device__ PreWork(int32_t *metadata, int64_t max_blocks, int ctas) {
        header = reinterpret_cast<PreHeader *>(metadata);
        segments = reinterpret_cast<PreSegment *>(header + 1);
        cuts = reinterpret_cast<PreCut *>(segments + pre_max_segments(max_blocks, ctas));
    }
};
__host__ __device__ inline size_t pre_words(int64_t max_blocks, int ctas) {
    return (sizeof(PreHeader) + pre_max_segments(max_blocks, ctas) * sizeof(PreSegment) + pre_slots(ctas) * sizeof(PreCut)) / sizeof(int32_t);
}

// Rounds over the CTAs: heads go in chunks, a chunk's segments longest first with its heads
// side by side, so that the CTAs of a moment share few heads' keys (in L2) and the
// last items are short.  Every other round runs backwards over the CTAs: over lengths
// that fall, each gets its share.
__host__ __device__ inline bool pre_round_item(int64_t round, int cta, int ctas, int segments, int h_kv, int chunk, int &segment, int &head) {
    const int64_t items = (int64_t)segments * h_kv, first = round * ctas;
    if (first + cta >= items) return false;
    const int64_t last = items - 1 < first + ctas - 1 ? items - 1 : first + ctas - 1;
    const int64_t i = round & 1 ? last - cta : first + cta;
    const int64_t per = (int64_t)segments * chunk;
    int c = 0;
    if (i >= per) c = items <= 0x7fffffff ? (int)((uint32_t)i / (uint32_t)per) : (int)(i / per);
    const int heads = chunk < h_kv - c * chunk ? chunk : h_kv - c * chunk;
    const int64_t in = i - c * per;
    segment = in <= 0x7fffffff ? (int)((uint32_t)in / (uint32_t)heads) : (int)(in / heads);
    head = c * chunk + (int)(in - (int64_t)segment * heads);
    return true;
}

}  // namespace mla
