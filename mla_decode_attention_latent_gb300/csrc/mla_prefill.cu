// Attention of packed prompts on the tensor cores.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j - m_i),  lse_i = m_i + ln(sum_j p_ij)
// over the keys j that query row i sees, d_qk = 128 or 128 + 64 (the 64 RoPE dims
// of a key shared by all heads, read from their own tensor), d_v = 128.
//
// A CTA takes one segment at a time, steps of a block of the partition
// (mla_prefill_schedule.cu) for one key head: two tiles A and B of 128 query rows (row r of a tile is
// head r % group of token r / group, so that grouped heads share the loads of their
// key head), walking steps of 128 keys together, so that every key and value
// that lands in shared memory serves 256 rows.  Tensor memory is full: S_A, S_B, O_A,
// O_B take 128 of the 512 columns each, and a tile's weights P overwrite its scores
// as bf16 operands.  The roles, of 12 warps:
//   0-3, 4-7  rows of A and of B, a thread per row: S from tensor memory, mask, weights and
//             their sum in fp32, P back in two halves; O read and written at the end
//   8         loads: Q of a segment, then keys and values of each step in turn, as chunks
//             of 16 KB through one ring (64 dims of 128 keys, 128 dims of 64 values)
//   9, 10     MMAs of A and of B, in turns of PV(j) QK(j+1): while the rows of one tile take
//             their maximum and exponents, the other tile's products run.  PV starts on
//             the first half of the weights
//   11        zeroes the value rows behind a sequence's last key, which belong to
//             another sequence (weight 0 times an infinity would be NaN)
// Products stop at multiples of 16 keys behind the last one that a tile sees.
//
// Bound by the tensor cores' operands: a step of both tiles is 2 x 128 x 128 x (d_qk + 128)
// products, 2560 cycles at d_qk = 192, and takes 3280, as QK's MMAs read 8 KB of shared
// memory each, as much as there is in their 64 cycles, and take 85.  4096 tokens of 128 heads
// (d_qk = 192, causal) 445 us in a burst, 1.54 PFLOP/s, and 480 call after call, under the
// power cap; d_qk = 128 without a mask 1.7.  A few rows
// behind long contexts take the same 2 us a step, on as many CTAs as equal parts give (4.1
// TB/s of keys and values).
//
// The code is kept small: a CTA's roles share an instruction cache, and what comes once per
// item (a first step, the output) is fetched anew each time.  The same work with its loops
// unrolled once more took prompts of 300 rows from 66 to 92 us.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "mla_prefill.cuh"
#include "mla_sm103.cuh"

namespace mla {
namespace {

using namespace sm103;

constexpr int kThreads = 384;
// registers of a thread: 168 at launch; the rows' threads, which keep what they know of the
// next item beside a half's scores and weights, get some of the others'
// (256 x 200 + 128 x 104 = 384 x 168)
constexpr int kRowRegs = 200, kOtherRegs = 104;
static_assert(256 * kRowRegs + 128 * kOtherRegs <= kThreads * 168, "a split of what the CTA was launched with");
constexpr int kLoadWarp = 8, kMmaWarp = 9, kZeroWarp = 11;  // MMAs: a warp per tile
constexpr uint32_t kSlotBytes = 16384;
constexpr uint32_t kTmemCols = 512;
constexpr float kMostWeight = 0x1p20f;  // that a row's 64 weights may add up to before their reference is raised

// shared memory: Q of both tiles, the ring, barriers
template <bool kRope>
struct Layout {
    static constexpr int kChunks = kRope ? 3 : 2;         // 64-dim chunks of a query or key
    static constexpr int kStepSlots = kChunks + 2;        // ring slots of a step: keys, then values
    static constexpr int kSlots = kRope ? 8 : 10;         // 1.6 or 2.5 steps
    static constexpr uint32_t kRing = kPreTiles * kChunks * kSlotBytes;
    static constexpr uint32_t kBars = kRing + kSlots * kSlotBytes;
    static constexpr uint32_t kItems = kBars + 512;       // descriptions of items
    static constexpr uint32_t kBytes = kItems + 256 + 1024;  // 1024: room to align the base
};
static_assert(Layout<true>::kBytes <= 232448 && Layout<false>::kBytes <= 232448, "shared memory of a CTA");

// Barriers.  The keys of a step are one load group, its values the next: group g has
// the barriers g % kGroups, whose next use, g + kGroups, is loaded into slots of g, so
// after g is used up.
constexpr int kGroups = 6;
enum { B_FULL = 0, B_EMPTY = B_FULL + kGroups, B_TAIL = B_EMPTY + kGroups, B_ZERO = B_TAIL + kGroups, B_QFULL = B_ZERO + kGroups,
       B_QEMPTY = B_QFULL + 2, B_S = B_QEMPTY + 2, B_P = B_S + 2, B_PV0 = B_P + 4, B_PV = B_PV0 + 2, B_OFREE = B_PV + 2, B_TURN = B_OFREE + 2, B_FINAL = B_TURN + 2, B_ITEM = B_FINAL + 2, B_READ = B_ITEM + 4,
       kNumBars = B_READ + 4 };
static_assert(kNumBars * 8 <= 512, "room for the barriers");
static_assert(Layout<true>::kSlots < kGroups / 2 * Layout<true>::kStepSlots && Layout<false>::kSlots < kGroups / 2 * Layout<false>::kStepSlots,
              "the ring holds fewer than kGroups groups");

struct Ctx {
    char *base;
    uint64_t *bars;
    unsigned int *status;
    __device__ uint64_t *bar(int i) const { return bars + i; }
    __device__ bool wait(int i, uint32_t parity) const { return mbar_wait(bars + i, parity, status); }
};

// The items (segment, key head) of a CTA, as the load warp goes through them.  The segment
// of the next one is fetched while the current one is loaded.
struct Walk {
    PreWork work;
    int segments, round = 0;
    bool more;
    PreSegment ahead;
    int ahead_head;
    __device__ Walk(const PrefillParams &p) : work(p.metadata, p.max_blocks, p.sms) {
        const bool fits = pre_fits(*work.header, p);
        if (!fits && blockIdx.x == 0 && (threadIdx.x & 31) == 0) atomicOr(p.status, MLA_DEVERR_SEQLEN);
        segments = !fits ? 0 : max(0, work.header->segments);
        fetch(p);
    }
    __device__ __forceinline__ void fetch(const PrefillParams &p) {
        int segment;
        more = pre_round_item(round, blockIdx.x, gridDim.x, segments, p.h_kv, p.head_chunk, segment, ahead_head);
        if (!more) return;
        const int4 *src = reinterpret_cast<const int4 *>(work.segments + segment);
        const int4 u = src[0], v = src[1];
        ahead = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
        ++round;
    }
};

// An item as all roles see it.
struct Item : PreSegment {
    int head;
    int seen_of[kPreTiles], steps_of[kPreTiles];  // of each tile: keys that its last token sees, steps of them in the segment
};
static_assert(sizeof(PreSegment) == 32, "an item is written as three 16-byte words");

__device__ Item make_item(const PrefillParams &p, PreSegment s, int head) {
    const int per = p.tile_tokens;
    // a partition of other lengths must not make the kernel leave its tensors
    if (s.q0 < 0 || s.tokens < 0 || s.tokens > kPreTiles * per || (int64_t)s.q0 + s.tokens > p.num_q || s.keys < 0 || s.k0 < 0 ||
        (int64_t)s.k0 + s.keys > p.num_k || s.step0 < 0 || s.step1 > pre_steps(s.keys) ||
        (s.part >= 0 && ((int64_t)s.part + 1) * p.h_kv > pre_slots(p.sms))) {
        if ((threadIdx.x & 31) == 0) atomicOr(p.status, MLA_DEVERR_SEQLEN);
        s.q0 = s.tokens = s.step0 = s.step1 = 0;
        s.part = -1;
    }
    Item x;
    static_cast<PreSegment &>(x) = s;
    x.head = head;
#pragma unroll
    for (int t = 0; t < kPreTiles; ++t) {
        const int last = min(s.tokens, (t + 1) * per) - 1;
        x.seen_of[t] = last < t * per ? 0 : p.causal ? pre_seen(s, last) : s.keys;
        x.steps_of[t] = max(0, min(pre_steps(x.seen_of[t]), s.step1) - s.step0);
    }
    return x;
}

// The items on their way from the load warp to the others, four at most, so that no role
// works an item out for itself between two others (which took 2 us of each): written
// an item ahead, read by a warp at once.  An item of q0 < 0 is the end.
constexpr int kItems = 4, kReaders = 11;

struct Items {
    uint32_t base, n = 0;
    __device__ Items(uint32_t at) : base(at) {}
    __device__ bool put(const Ctx &c, const Item &x) {
        const uint32_t i = n % kItems;
        if (!__all_sync(0xffffffffu, c.wait(B_READ + i, ((n / kItems) & 1) ^ 1))) return false;
        if (elect_one_lane()) {
            const uint32_t at = base + i * 64;
            sts128(at, x.q0, x.tokens, x.k0, x.keys);
            sts128(at + 16, x.seen, x.step0, x.step1, x.part);
            sts128(at + 32, x.seen_of[0], x.seen_of[1], x.steps_of[0], x.steps_of[1]);
            sts32(at + 48, x.head);
            mbar_arrive(c.bar(B_ITEM + i));
        }
        __syncwarp();
        ++n;
        return true;
    }
    // a warp's next item; false at the end (or when it does not come)
    __device__ __forceinline__ bool get(const Ctx &c, Item &x) {
        const uint32_t i = n % kItems, at = base + i * 64;
        if (!__all_sync(0xffffffffu, c.wait(B_ITEM + i, (n / kItems) & 1))) return false;
        const uint4 u = lds128(at), v = lds128(at + 16), w = lds128(at + 32);
        x.head = (int)lds32(at + 48);
        x.q0 = u.x, x.tokens = u.y, x.k0 = u.z, x.keys = u.w, x.seen = v.x, x.step0 = v.y, x.step1 = v.z, x.part = v.w;
        x.seen_of[0] = w.x, x.seen_of[1] = w.y, x.steps_of[0] = w.z, x.steps_of[1] = w.w;
        __syncwarp();
        if (elect_one_lane()) mbar_arrive(c.bar(B_READ + i));
        ++n;
        return x.q0 >= 0;
    }
};

// Whether step j of a segment has value rows behind the sequence's last key that a
// product reaches: zeroed, in the slots of the step's values.  The load role says when
// such a group has been issued (B_TAIL: only then is the group's B_FULL in the phase
// that the zeroing waits for), the zero role when it is done (B_ZERO).  The group's
// barriers are used again after both, so none is more than a phase ahead of who waits.
__device__ __forceinline__ bool tail_step(const PreSegment &s, int j) {
    return s.keys - (s.step0 + j) * kPreTile < kPreTile && s.keys % 16 != 0;
}

// One lane of a converged warp, the same one every time.  The load and MMA warps run
// their role as whole warps and only issue in the elected lane: where one lane runs the
// role alone, the compiler cannot tell that an operand is the same for the warp, and
// an MMA costs its issuer 200 cycles instead of the 64 that it takes.
__device__ __forceinline__ bool elected() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n}" : "=r"(yes));
    return yes != 0;
}

// ---------------------------------------------------------------- loads
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int head, int token) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(head), "r"(token)
        : "memory");
}

template <bool kRope>
__device__ void load_role(const PrefillParams &p, const Ctx &c, Items items, const CUtensorMap *mq, const CUtensorMap *mk, const CUtensorMap *mr,
                          const CUtensorMap *mv) {
    using L = Layout<kRope>;
    Walk walk(p);
    uint32_t slot = 0, group = 0, freed = 0, held = 0;  // groups issued and given back, slots that the others hold
    uint32_t qn[kPreTiles] = {0, 0};
    const uint32_t q_bytes = (uint32_t)(p.tile_tokens * p.group) * 128u;
    auto wait = [&](int bar, uint32_t parity) { return __all_sync(0xffffffffu, c.wait(bar, parity)) != 0; };
    // room for a group of n slots: groups come back in order, keys and values in turn
    auto room = [&](uint32_t n) {
        while (held + n > L::kSlots) {
            if (!wait(B_EMPTY + freed % kGroups, (freed / kGroups) & 1)) return false;
            held -= freed & 1 ? 2 : L::kChunks;
            ++freed;
        }
        held += n;
        return true;
    };
    auto next_slot = [&] {
        const uint32_t at = smem_u32(c.base + L::kRing) + slot * kSlotBytes;
        slot = slot + 1 == L::kSlots ? 0 : slot + 1;
        return at;
    };
    bool ok = true;
    Item next;
    // the next item, or the end, worked out and told to the others
    auto look_ahead = [&] {
        if (walk.more) {
            const PreSegment segment = walk.ahead;
            const int head = walk.ahead_head;
            walk.fetch(p);
            next = make_item(p, segment, head);
        } else {
            next.q0 = -1;
        }
        return items.put(c, next);
    };
    ok = look_ahead();
    while (ok && next.q0 >= 0) {
        const Item s = next;
        const int head = s.head, n = max(s.steps_of[0], s.steps_of[1]);
        if (!(ok = look_ahead())) break;
        // Q of the tiles that walk, ahead of the first keys, which so wait for its place too: it is
        // free only when the products of the segment before have read it
#pragma unroll
        for (int t = 0; t < kPreTiles; ++t) {
            if (!ok || s.steps_of[t] == 0) continue;
            ok = wait(B_QEMPTY + t, (qn[t] & 1) ^ 1);
            if (!ok) continue;
            ++qn[t];
            if (elected()) {
                mbar_arrive_expect_tx(c.bar(B_QFULL + t), L::kChunks * q_bytes);
                for (int ch = 0; ch < L::kChunks; ++ch)
                    tma_load(smem_u32(c.base + (t * L::kChunks + ch) * kSlotBytes), mq, c.bar(B_QFULL + t), 64 * ch, head * p.group,
                             s.q0 + t * p.tile_tokens);
            }
            __syncwarp();
        }
        for (int j = 0; ok && j < n; ++j) {
            const int k0 = s.k0 + (s.step0 + j) * kPreTile;
            if (!(ok = room(L::kChunks))) break;
            uint64_t *bar = c.bar(B_FULL + group % kGroups);
            ++group;
            if (elected()) mbar_arrive_expect_tx(bar, L::kChunks * kSlotBytes);
            __syncwarp();
#pragma unroll
            for (int ch = 0; ch < L::kChunks; ++ch) {
                const uint32_t dst = next_slot();
                if (elected()) {
                    if (ch < 2) tma_load(dst, mk, bar, 64 * ch, head, k0);
                    else tma_load(dst, mr, bar, 0, 0, k0);
                }
                __syncwarp();
            }
            if (!ok || !(ok = room(2))) break;
            bar = c.bar(B_FULL + group % kGroups);
            const uint32_t tail = group % kGroups;
#ifdef MLA_TEST_SKIP_ONE_LOAD
            // test builds only: CTA 0 never loads the values of its second step, so that
            // the issuers' bounded wait for them runs out and every role unwinds
            if (blockIdx.x == 0 && group == 3) {
                ++group;
                next_slot();
                next_slot();
                continue;
            }
#endif
            ++group;
            if (elected()) mbar_arrive_expect_tx(bar, 2 * kSlotBytes);
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t dst = next_slot();
                if (elected()) {
                    tma_load(dst, mv, bar, 0, head, k0 + 64 * h);
                    tma_load(dst + kSlotBytes / 2, mv, bar, 64, head, k0 + 64 * h);
                    if (h == 1 && tail_step(s, j)) mbar_arrive(c.bar(B_TAIL + tail));
                }
                __syncwarp();
            }
        }
    }
    // nothing may be in flight when the CTA ends (after a wait that gave up, too)
    for (uint32_t g = freed; g < group; ++g) c.wait(B_FULL + g % kGroups, (g / kGroups) & 1);
#pragma unroll
    for (int t = 0; t < kPreTiles; ++t)
        if (qn[t]) c.wait(B_QFULL + t, (qn[t] - 1) & 1);
}

// ---------------------------------------------------------------- MMAs
// instruction descriptors whose number of columns follows the keys in sight
__device__ __forceinline__ uint32_t idesc_keys(int keys) { return idesc_bf16(kPreTile, 0, false, false) | ((uint32_t)(keys >> 3) << 17); }
__device__ __forceinline__ int keys16(int keys) { return keys >= kPreTile ? kPreTile : (keys + 15) & ~15; }

// The MMAs of tile t.  An MMA holds its issuer for about its own duration, so a wait
// of one issuer would idle the pipe: the two tiles have a warp each, and one waits
// while the other issues.  Left alone they fall into step (both tiles' products at
// once, then both tiles' exponents), so they take turns: a turn is PV(j) QK(j+1), and is
// handed over a few MMAs before its end.
template <bool kRope>
__device__ void mma_role(const Ctx &c, Items items, uint32_t tmem, int t) {
    using L = Layout<kRope>;
    constexpr uint32_t kPvDesc = idesc_bf16(kPreTile, kPreHead, false, true);
    Item s;
    uint32_t slot = 0, group = 0, qn = 0, done = 0, turn = 0;
    uint32_t zeroed = 0;  // a bit per group barrier, the phase of its B_ZERO
    const uint32_t ring = smem_u32(c.base + L::kRing);
    const uint32_t s_col = tmem + t * 128, o_col = tmem + 256 + t * 128;
    const uint64_t q_desc = desc_sw128(smem_u32(c.base) + t * L::kChunks * kSlotBytes, 16, 1024), k_desc = desc_sw128(ring, 16, 1024),
                   v_desc = desc_sw128(ring, kSlotBytes / 2, 1024);
    auto wait = [&](int bar, uint32_t parity) { return __all_sync(0xffffffffu, c.wait(bar, parity)) != 0; };
    auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    auto after = [](uint32_t at, uint32_t n) { return at + n >= L::kSlots ? at + n - L::kSlots : at + n; };
    while (items.get(c, s)) {
        const int steps = uniform(t ? s.steps_of[1] : s.steps_of[0]), n = uniform(max(s.steps_of[0], s.steps_of[1])),
                  seen = uniform((t ? s.seen_of[1] : s.seen_of[0]) - s.step0 * kPreTile);
        // S = Q K(j)^T, the keys (group g) at slot `at`; `hand_over`: the turn ends here
        auto scores = [&](int j, uint32_t at, uint32_t g, bool hand_over) {
            const uint32_t idesc = idesc_keys(keys16(seen - j * kPreTile));
            uint64_t bd[L::kChunks];
#pragma unroll
            for (int ch = 0; ch < L::kChunks; ++ch) bd[ch] = k_desc + after(at, ch) * (kSlotBytes / 16);
            if (elected()) {
#pragma unroll
                for (int ch = 0; ch < L::kChunks; ++ch) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)  // 16 dims: 32 B
                        mma_ss(s_col, q_desc + ch * (kSlotBytes / 16) + 2 * i, bd[ch] + 2 * i, idesc, ch + i > 0);
                }
                if (hand_over) mbar_arrive(c.bar(B_TURN + 1 - t));
                mma_commit(c.bar(B_S + t));
                mma_commit(c.bar(B_EMPTY + g % kGroups));
                if (j == steps - 1) mma_commit(c.bar(B_QEMPTY + t));
            }
            __syncwarp();
        };
        // a group that the other tile alone uses (its keys lie behind this tile's rows)
        auto pass = [&](uint32_t g) {
            if (!wait(B_FULL + g % kGroups, (g / kGroups) & 1)) return false;
            if (elected()) mbar_arrive(c.bar(B_EMPTY + g % kGroups));
            __syncwarp();
            return true;
        };
        if (n == 0) continue;
        if (steps > 0) {
            if (!wait(B_QFULL + t, qn & 1) || !wait(B_FULL + group % kGroups, (group / kGroups) & 1)) return;
            ++qn;
            scores(0, slot, group, false);
        } else if (!pass(group)) {
            return;
        }
        ++group;
        slot = after(slot, L::kChunks);
        for (int j = 0; j < n; ++j, ++turn) {
            // the values of step j, then the keys of step j + 1
            const uint32_t vg = group % kGroups, kg = group + 1, k_at = after(slot, 2);
            const bool tail = tail_step(s, j), more = j + 1 < n, scores_too = j + 1 < steps;
            if (j < steps) {
                const uint64_t bd[2] = {v_desc + slot * (kSlotBytes / 16), v_desc + after(slot, 1) * (kSlotBytes / 16)};
                const int parts = keys16(seen - j * kPreTile) / 16;
                if (!wait(B_FULL + vg, (group / kGroups) & 1)) return;
                if (tail && !wait(B_ZERO + vg, (zeroed >> vg) & 1)) return;
                if (j == 0 && !wait(B_OFREE + t, qn & 1)) return;  // O of the segment before is read
                if (!wait(B_P + 2 * t, done & 1)) return;
                if (!wait(B_TURN + t, t == 0 ? (turn & 1) ^ 1 : turn & 1)) return;
                // O (+)= P V(j), the weights in two halves
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h && !wait(B_P + 2 * t + 1, done & 1)) return;
                    tc_fence_after();
                    if (elected()) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)  // 16 keys: 2048 B
                            if (4 * h + i < parts) mma_ts(o_col, s_col + 8 * (4 * h + i), bd[h] + 128 * i, kPvDesc, j + h + i > 0);
                        if (h == 0) {
                            mma_commit(c.bar(B_PV0 + t));
                        } else {
                            mma_commit(c.bar(B_PV + t));
                            mma_commit(c.bar(B_EMPTY + vg));
                            if (!scores_too) mbar_arrive(c.bar(B_TURN + 1 - t));
                        }
                    }
                    __syncwarp();
                }
                ++done;
                if (scores_too) {
                    if (!wait(B_FULL + kg % kGroups, (kg / kGroups) & 1)) return;
                    scores(j + 1, k_at, kg, true);
                }
            } else {
                if (!pass(group) || !wait(B_TURN + t, t == 0 ? (turn & 1) ^ 1 : turn & 1)) return;
                if (elected()) mbar_arrive(c.bar(B_TURN + 1 - t));
                __syncwarp();
            }
            if (tail) zeroed ^= 1u << vg;
            if (more && !scores_too && !pass(kg)) return;
            group += more ? 2 : 1;
            slot = more ? after(k_at, L::kChunks) : k_at;
        }
    }
}

// ---------------------------------------------------------------- value rows behind a sequence
template <bool kRope>
__device__ void zero_role(const Ctx &c, Items items) {
    using L = Layout<kRope>;
    Item s;
    uint32_t slot = 0, group = 0, tails = 0;  // tails: a bit per group barrier, the phase of its B_TAIL
    const int lane = threadIdx.x & 31;
    while (items.get(c, s)) {
        const int n = max(s.steps_of[0], s.steps_of[1]);
        if (n == 0) continue;
        if (tail_step(s, n - 1)) {
            const int valid = s.keys - (s.step0 + n - 1) * kPreTile;  // keys of the last step
            const uint32_t last = group + 2 * n - 1, g = last % kGroups;
            const uint32_t first = (uint32_t)((slot + (uint64_t)n * L::kStepSlots - 2) % L::kSlots);
            if (!__all_sync(0xffffffffu, c.wait(B_TAIL + g, (tails >> g) & 1))) return;
            tails ^= 1u << g;
            if (!__all_sync(0xffffffffu, c.wait(B_FULL + g, (last / kGroups) & 1))) return;
            // rows valid .. of the 16 that the products reach, all 256 bytes of each
            for (int i = lane; i < (16 - valid % 16) * 16; i += 32) {
                const int row = valid + i / 16, piece = i % 16;
                const uint32_t at = (first + row / 64) % L::kSlots;
                sts128(smem_u32(c.base + L::kRing + at * kSlotBytes) + (piece / 8) * (kSlotBytes / 2) + (row % 64) * 128 + (piece % 8) * 16, 0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(c.bar(B_ZERO + g));
        }
        group += 2 * n;
        slot = (uint32_t)((slot + (uint64_t)n * L::kStepSlots) % L::kSlots);
    }
}

// ---------------------------------------------------------------- rows
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 32 columns of tensor memory that are complete behind arrived()
__device__ __forceinline__ void arrived(uint32_t (&a)[32], uint32_t (&b)[32]) {
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(a[i]), "+r"(b[i]));  // no use moves before the wait
}

__device__ __forceinline__ void arrived(uint32_t (&a)[32]) {
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(a[i]));
}

// A row's weights are exp2(score * scale - reference).  The reference need not be the
// running maximum: bf16 and fp32 hold a weight as exactly at 2^20 as at 1.  So it is the
// largest of the row's first 64 scores, and is raised only when 64 weights add up to
// more than kMostWeight, which their sum tells without a maximum; then their
// maximum becomes the reference, O and the sum are scaled, and they are computed again.
__device__ __forceinline__ float largest(const uint32_t (&a)[32], const uint32_t (&b)[32]) {
    float mx[4] = {__uint_as_float(a[0]), __uint_as_float(a[1]), __uint_as_float(b[0]), __uint_as_float(b[1])};
#pragma unroll
    for (int i = 2; i < 30; i += 4) {
        mx[0] = max3f(mx[0], __uint_as_float(a[i]), __uint_as_float(a[i + 1]));
        mx[1] = max3f(mx[1], __uint_as_float(a[i + 2]), __uint_as_float(a[i + 3]));
        mx[2] = max3f(mx[2], __uint_as_float(b[i]), __uint_as_float(b[i + 1]));
        mx[3] = max3f(mx[3], __uint_as_float(b[i + 2]), __uint_as_float(b[i + 3]));
    }
    const float c = max3f(mx[0], mx[1], fmaxf(__uint_as_float(a[30]), __uint_as_float(a[31])));
    return max3f(c, max3f(mx[2], mx[3], __uint_as_float(b[30])), __uint_as_float(b[31]));
}

// Weights of 32 scores at a time as bf16 pairs, and the sum of all
struct Weigh {
    uint64_t scale2, shift2, sum[2];
    __device__ __forceinline__ Weigh(float m, float scale_log2) {
        const float shift = m == -INFINITY ? 0.f : -m * scale_log2;
        scale2 = f2_pack(scale_log2, scale_log2), shift2 = f2_pack(shift, shift);
        sum[0] = sum[1] = 0;
    }
    __device__ __forceinline__ void operator()(const uint32_t (&x)[32], uint32_t *w) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float lo, hi;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), scale2, shift2), lo, hi);
            lo = exp2_fast(lo);
            hi = exp2_fast(hi);
            sum[i & 1] = f2_add(sum[i & 1], f2_pack(lo, hi));
            w[i] = pack_bf16(lo, hi);
        }
    }
    __device__ __forceinline__ float total() const {
        float lo, hi;
        f2_unpack(f2_add(sum[0], sum[1]), lo, hi);
        return lo + hi;
    }
};

// 64 scores of a row, and what its weights refer to
struct Half {
    uint32_t s_col, o_col;  // tensor memory: the scores (the weights go to `p_col`), the tile's O
    uint32_t p_col;
    int left;               // scores in sight, from the first on
    float m, l;             // reference (a raw score), sum of the weights so far
    bool first;             // no reference yet
};
struct State {
    float m, l;
    int ok;
};

// The half that a warp meets now and then: some row's first scores, scores out of
// sight, or weights far above the reference.  Out of line, once, for the instruction cache.
__device__ __noinline__ State careful_half(const Half x, float scale_log2, uint64_t *products, uint32_t parity, unsigned int *status) {
    uint32_t a[32], b[32], w[32];
    if (!x.first && !__any_sync(0xffffffffu, x.left > 0)) {  // nothing in sight of the warp's rows
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = 0;
        tmem_st32(x.p_col, w);
        return {x.m, x.l, 1};
    }
    tmem_ld32(x.s_col, a);
    tmem_ld32(x.s_col + 32, b);
    arrived(a, b);
    if (__any_sync(0xffffffffu, x.left < 64)) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            a[i] = i < x.left ? a[i] : 0xff800000u;
            b[i] = i + 32 < x.left ? b[i] : 0xff800000u;
        }
    }
    float m = x.m, l = x.l, sum = 0.f;
    bool raise = x.first;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        if (__any_sync(0xffffffffu, raise)) {
            const float m_new = raise ? fmaxf(m, largest(a, b)) : m;
            const float f = !raise ? 1.f : m == -INFINITY ? 0.f : exp2_fast((m - m_new) * scale_log2);
            if (products) {
                // every product so far is in O
                if (!__all_sync(0xffffffffu, mbar_wait(products, parity, status))) return {m, l, 0};
                tc_fence_after();
#pragma unroll 1
                for (int i = 0; i < 8; ++i) {
                    uint32_t o[16];
                    tmem_ld16(x.o_col + 16 * i, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                    tmem_st16(x.o_col + 16 * i, o);
                }
                tmem_wait_st();
            }
            l *= f;
            m = m_new;
        }
        Weigh weigh(m, scale_log2);
        weigh(a, w);
        weigh(b, w + 16);
        sum = weigh.total();
        raise = !(sum <= kMostWeight) || (m == -INFINITY && x.left > 0);
        if (!__any_sync(0xffffffffu, raise)) break;
    }
    tmem_st32(x.p_col, w);
    return {m, l + sum, 1};
}

// A partial result's 4 dims 4 c .. of a row: rows side by side, as the rows' threads write them
__device__ __forceinline__ int64_t part_at(int64_t slot, int c, int row) { return (slot * (kPreHead / 4) + c) * kPreRows + row; }

// 32 bytes at once: a lane writes its own row, and a store instruction takes a cycle for each
// of the 32 lines that it touches
__device__ __forceinline__ void store32(void *dst, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]),
                 "r"(w[6]), "r"(w[7])
                 : "memory");
}

// kWholeSteps: the two halves of a step in sight in one go, half 1's first scores under way while half 0's last are
// weighed (all keys, d_qk = 128: 317 us against 336). At d_qk = 192 the MMAs set the pace, and half the code, for either
// half, is better: forty prompts of 300 62.7 against 64.6 (a prompt of 4096 at 128 heads 434 against 438, in bursts).
template <bool kWholeSteps>
__device__ void row_role(const PrefillParams &p, const Ctx &c, Items items, uint32_t tmem, int t) {
    const int warp = threadIdx.x >> 5, r = threadIdx.x & (kPreTile - 1);
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_col = tmem + lane_base + t * 128, o_col = tmem + lane_base + 256 + t * 128;
    const int per = p.tile_tokens, in_tile = r / p.group, hh = r - in_tile * p.group;
    Item s;
    uint32_t phase = 0;  // steps of this tile so far
    bool more = items.get(c, s);
    while (more) {
        const int head = s.head, steps = t ? s.steps_of[1] : s.steps_of[0];
        const int token = t * per + in_tile;
        const bool on = in_tile < per && token < s.tokens;
        // A row of no query beside rows of queries follows the tile's last, so that its warp need not
        // mask; a warp without queries has nothing in sight
        const int seen = __any_sync(0xffffffffu, on) ? !on ? (t ? s.seen_of[1] : s.seen_of[0]) : p.causal ? pre_seen(s, token) : s.keys : 0;
        float m = -INFINITY, l = 0.f;  // reference (a raw score), sum of the weights
        for (int j = 0; j < steps; ++j, ++phase) {
            if (!__all_sync(0xffffffffu, c.wait(B_S + t, phase & 1))) return;
            tc_fence_after();
            const int ahead = seen - (s.step0 + j) * kPreTile;
            auto handed = [&](int h) {
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(c.bar(B_P + 2 * t + h));
            };
            int h = 0;
            if (kWholeSteps && !__any_sync(0xffffffffu, j == 0 || ahead < kPreTile || m == -INFINITY)) {
                // 32 scores are on their way while 32 are weighed
                uint32_t x0[32], x1[32], w[32];
                Weigh first(m, p.scale_log2), second(m, p.scale_log2);
                tmem_ld32(s_col, x0);
                arrived(x0);
                tmem_ld32(s_col + 32, x1);
                first(x0, w);
                arrived(x1);
                tmem_ld32(s_col + 64, x0);
                first(x1, w + 16);
                const float sum0 = first.total();
                const bool good = __all_sync(0xffffffffu, sum0 <= kMostWeight);
                if (good) tmem_st32(s_col, w);
                arrived(x0);
                if (good) {
                    tmem_ld32(s_col + 96, x1);
                    second(x0, w);
                    handed(0);
                    arrived(x1);
                    second(x1, w + 16);
                    const float sum1 = second.total();
                    l += sum0;
                    h = 1;
                    if (__all_sync(0xffffffffu, sum1 <= kMostWeight)) {
                        tmem_st32(s_col + 32, w);
                        l += sum1;
                        handed(1);
                        h = 2;
                    }
                }
            }
#pragma unroll 1
            for (; h < 2; ++h) {
                bool weighed = false;
                if (!kWholeSteps && !__any_sync(0xffffffffu, j + h == 0 || ahead - 64 * h < 64 || m == -INFINITY)) {
                    uint32_t x0[32], x1[32], w[32];
                    Weigh weigh(m, p.scale_log2);
                    tmem_ld32(s_col + 64 * h, x0);
                    arrived(x0);
                    tmem_ld32(s_col + 64 * h + 32, x1);
                    weigh(x0, w);
                    arrived(x1);
                    weigh(x1, w + 16);
                    const float sum = weigh.total();
                    weighed = __all_sync(0xffffffffu, sum <= kMostWeight);
                    if (weighed) {
                        tmem_st32(s_col + 32 * h, w);
                        l += sum;
                    }
                }
                if (!weighed) {
                    // products so far: the step before's, or this step's first half
                    const Half x = {s_col + 64 * h, o_col, s_col + 32 * h, ahead - 64 * h, m, l, j + h == 0};
                    const State y = careful_half(x, p.scale_log2, j + h == 0 ? nullptr : c.bar((h ? B_PV0 : B_PV) + t), (h ? phase : phase - 1) & 1, c.status);
                    if (!y.ok) return;
                    m = y.m;
                    l = y.l;
                }
                handed(h);
            }
        }
        // epilogue: o = O / l, lse
        float lse = l == 0.f ? -INFINITY : m * p.scale + logf(l);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t row = (int64_t)(s.q0 + token) * p.h_q + head * p.group + hh;
        const int64_t slot = (int64_t)s.part * p.h_kv + head;
        const int part = s.part;
        more = items.get(c, s);
        if (on) {
            if (part < 0) p.lse[row] = lse;
            else p.lse_part[slot * kPreRows + t * kPreTile + r] = lse;
        }
        if (steps == 0) {
            if (on && part < 0)
                for (int i = 0; i < kPreHead / 8; ++i) reinterpret_cast<uint4 *>(p.out + row * kPreHead)[i] = make_uint4(0, 0, 0, 0);
            continue;
        }
        if (!__all_sync(0xffffffffu, c.wait(B_PV + t, (phase - 1) & 1))) return;
        tc_fence_after();
#pragma unroll 1
        for (int i2 = 0; i2 < 2; ++i2) {
            uint32_t both[2][32];
            __syncwarp();  // rows of no query come here ahead of the others, and the whole warp loads
            tmem_ld32(o_col + 64 * i2, both[0]);
            tmem_ld32(o_col + 64 * i2 + 32, both[1]);
            arrived(both[0], both[1]);
            if (i2 == 1) {
                tc_fence_before();
                mbar_arrive(c.bar(B_OFREE + t));
            }
            if (!on) continue;
#pragma unroll
            for (int i1 = 0; i1 < 2; ++i1) {
                const int i = 2 * i2 + i1;
                uint32_t (&o)[32] = both[i1];
                if (part < 0) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            w[e] = pack_bf16(__uint_as_float(o[16 * k + 2 * e]) * inv, __uint_as_float(o[16 * k + 2 * e + 1]) * inv);
                        store32(p.out + row * kPreHead + 32 * i + 16 * k, w);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        reinterpret_cast<float4 *>(p.o_part)[part_at(slot, 8 * i + k, t * kPreTile + r)] =
                            make_float4(__uint_as_float(o[4 * k]) * inv, __uint_as_float(o[4 * k + 1]) * inv, __uint_as_float(o[4 * k + 2]) * inv,
                                        __uint_as_float(o[4 * k + 3]) * inv);
                }
            }
        }
    }
}

template <bool kRope>
__global__ void __launch_bounds__(kThreads, 1)
prefill_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mr,
               const __grid_constant__ CUtensorMap mv, const __grid_constant__ PrefillParams p) {
    using L = Layout<kRope>;
    extern __shared__ char raw[];
    __shared__ uint32_t s_tmem;
    Ctx c;
    c.base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    c.bars = reinterpret_cast<uint64_t *>(c.base + L::kBars);
    c.status = p.status;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kGroups; ++i) {
            mbar_init(c.bar(B_FULL + i), 1);
            mbar_init(c.bar(B_EMPTY + i), kPreTiles);
            mbar_init(c.bar(B_TAIL + i), 1);
            mbar_init(c.bar(B_ZERO + i), 1);
        }
        for (int t = 0; t < kPreTiles; ++t) {
            mbar_init(c.bar(B_QFULL + t), 1);
            mbar_init(c.bar(B_QEMPTY + t), 1);
            mbar_init(c.bar(B_S + t), 1);
            mbar_init(c.bar(B_P + 2 * t), kPreTile);
            mbar_init(c.bar(B_P + 2 * t + 1), kPreTile);
            mbar_init(c.bar(B_PV0 + t), 1);
            mbar_init(c.bar(B_PV + t), 1);
            mbar_init(c.bar(B_OFREE + t), kPreTile);
            mbar_init(c.bar(B_TURN + t), 1);
            mbar_init(c.bar(B_FINAL + t), 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(c.bar(B_ITEM + i), 1);
            mbar_init(c.bar(B_READ + i), kReaders);
        }
        fence_mbar_init();
    }
    if (warp == kLoadWarp && elect_one_lane()) {
        tma_prefetch_desc(&mq);
        tma_prefetch_desc(&mk);
        if (kRope) tma_prefetch_desc(&mr);
        tma_prefetch_desc(&mv);
    }
    if (warp < 8 && (threadIdx.x & (kPreTile - 1)) >= p.tile_tokens * p.group) {
        // rows that no query ever comes to
        const int t = warp >> 2, r = threadIdx.x & (kPreTile - 1);
        for (int i = 0; i < L::kChunks * 8; ++i)
            sts128(smem_u32(c.base + (t * L::kChunks + i / 8) * kSlotBytes) + r * 128 + i % 8 * 16, 0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&s_tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
    const Items items(smem_u32(c.base + L::kItems));
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
        {
            // Before the kernel in front has ended: the code for a first half into the instruction
            // cache, run on what the tile's O happens to hold (the first PV overwrites it)
            const uint32_t at = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 256 + 128 * (warp >> 2);
            const Half none = {at, at + 64, at, 64, 0.f, 0.f, true};
            careful_half(none, 1.f, nullptr, 0, c.status);
            tmem_wait_st();
        }
        griddep_wait();
        row_role<!kRope>(p, c, items, tmem, warp >> 2);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        griddep_wait();
        if (warp == kLoadWarp) {
            load_role<kRope>(p, c, items, &mq, &mk, &mr, &mv);
        } else if (warp < kZeroWarp) {
            const int t = warp - kMmaWarp;
            mma_role<kRope>(c, items, tmem, t);
            if (elected()) mma_commit(c.bar(B_FINAL + t));  // every MMA of this thread is done before tensor memory is released
            __syncwarp();
            c.wait(B_FINAL + t, 0);
        } else {
            zero_role<kRope>(c, items);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------- combine of cut items
// A warp per 32 rows of an item and 16 of the dims, a lane per row (the partial results'
// order): o = sum_s w_s o_s, w_s = exp(lse_s - lse).  A part in which the row saw
// nothing (lse -inf) was not written and does not count.
constexpr int kCombineWarps = 4, kCombineDims = 16;

__global__ void __launch_bounds__(kCombineWarps * 32) prefill_combine_kernel(const __grid_constant__ PrefillParams p) {
    griddep_wait();
    const PreWork work(p.metadata, p.max_blocks, p.sms);
    const int lane = threadIdx.x & 31, per = pre_tile_tokens(p.group);
    constexpr int kUnits = kPreRows / 32 * (kPreHead / kCombineDims);  // of an item
    const int n = pre_fits(*work.header, p) ? max(0, min(work.header->cuts, pre_slots(p.sms))) : 0;
    const int64_t total = (int64_t)n * p.h_kv * kUnits, stride = gridDim.x * kCombineWarps;
    for (int64_t i = (int64_t)blockIdx.x * kCombineWarps + (threadIdx.x >> 5); i < total; i += stride) {
        const int unit = (int)(i % kUnits), head = (int)(i / kUnits % p.h_kv);
        const PreCut cut = work.cuts[i / kUnits / p.h_kv];
        if (cut.part < 0 || cut.count < 1 || ((int64_t)cut.part + cut.count) * p.h_kv > pre_slots(p.sms)) continue;
        const int r = unit % (kPreRows / 32) * 32 + lane, c0 = unit / (kPreRows / 32) * (kCombineDims / 4);
        const int t = r / kPreTile, in_tile = (r % kPreTile) / p.group, hh = (r % kPreTile) - in_tile * p.group, token = t * per + in_tile;
        if (in_tile >= per || token >= cut.tokens || cut.q0 < 0 || (int64_t)cut.q0 + token >= p.num_q) continue;
        const int64_t slot0 = (int64_t)cut.part * p.h_kv + head;
        float top = -INFINITY;
#pragma unroll 4
        for (int k = 0; k < cut.count; ++k) top = fmaxf(top, p.lse_part[(slot0 + (int64_t)k * p.h_kv) * kPreRows + r]);
        const float base = top == -INFINITY ? 0.f : top;
        float sum = 0.f, o[kCombineDims] = {};
#pragma unroll 4
        for (int k = 0; k < cut.count; ++k) {
            const int64_t slot = slot0 + (int64_t)k * p.h_kv;
            const float lse = p.lse_part[slot * kPreRows + r];
            const float w = exp2_fast((lse - base) * 1.4426950408889634f);
            const bool none = lse == -INFINITY;
            sum += w;
#pragma unroll
            for (int c = 0; c < kCombineDims / 4; ++c) {
                const float4 x = reinterpret_cast<const float4 *>(p.o_part)[part_at(slot, c0 + c, r)];
                o[4 * c] = none ? o[4 * c] : fmaf(w, x.x, o[4 * c]);
                o[4 * c + 1] = none ? o[4 * c + 1] : fmaf(w, x.y, o[4 * c + 1]);
                o[4 * c + 2] = none ? o[4 * c + 2] : fmaf(w, x.z, o[4 * c + 2]);
                o[4 * c + 3] = none ? o[4 * c + 3] : fmaf(w, x.w, o[4 * c + 3]);
            }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t row = (int64_t)(cut.q0 + token) * p.h_q + head * p.group + hh;
        uint32_t w[kCombineDims / 2];
#pragma unroll
        for (int k = 0; k < kCombineDims / 2; ++k) w[k] = pack_bf16(o[2 * k] * inv, o[2 * k + 1] * inv);
        uint4 *dst = reinterpret_cast<uint4 *>(p.out + row * kPreHead + 4 * c0);
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        if (c0 == 0) p.lse[row] = sum == 0.f ? -INFINITY : base + logf(sum);
    }
}

// ---------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess && q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// [tokens][heads][d] in boxes of 64 dims x `box_heads` x `box_tokens`, 128-byte swizzle
bool make_map(CUtensorMap *m, const void *ptr, int d, int64_t heads, int64_t tokens, int64_t head_stride, int64_t token_stride, int box_heads,
              int box_tokens) {
    auto enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)token_stride * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;

template <bool kRope>
cudaError_t launch(const PrefillParams &p, cudaStream_t stream) {
    static std::mutex mutex;
    static bool ready[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mutex);
        if (!ready[dev]) {
            e = cudaFuncSetAttribute(prefill_kernel<kRope>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<kRope>::kBytes);
            if (e != cudaSuccess) return e;
            ready[dev] = true;
        }
    }
    CUtensorMap mq, mk, mr, mv;
    const int d = kPreHead + (kRope ? kPreRope : 0);
    const bool none = p.num_k == 0;  // no step is walked: any map will do
    if (!make_map(&mq, p.q, d, p.h_q, p.num_q, p.q_head, p.q_token, p.group, pre_tile_tokens(p.group))) return cudaErrorInvalidValue;
    if (none) {
        mk = mv = mr = mq;
    } else {
        if (!make_map(&mk, p.k, kPreHead, p.h_kv, p.num_k, p.k_head, p.k_token, 1, kPreTile)) return cudaErrorInvalidValue;
        if (!make_map(&mv, p.v, kPreHead, p.h_kv, p.num_k, p.v_head, p.v_token, 1, 64)) return cudaErrorInvalidValue;
        mr = mk;
        if (kRope && !make_map(&mr, p.k_rope, kPreRope, 1, p.num_k, kPreRope, p.k_rope_token, 1, kPreTile)) return cudaErrorInvalidValue;
    }
    e = launch_after(prefill_kernel<kRope>, dim3(p.sms), dim3(kThreads), Layout<kRope>::kBytes, stream, mq, mk, mr, mv, p);
    if (e != cudaSuccess) return e;
    if (!pre_may_cut(p.max_blocks, p.num_k, p.h_kv, p.sms)) return cudaSuccess;
    return launch_after(prefill_combine_kernel, dim3(8 * p.sms), dim3(kCombineWarps * 32), 0, stream, p);
}

}  // namespace

cudaError_t launch_prefill(const PrefillParams &p, cudaStream_t stream) {
    return p.rope ? launch<true>(p, stream) : launch<false>(p, stream);
}

}  // namespace mla
