// Attention of packed prompts on the tensor cores.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j - m_i),  lse_i = m_i + ln(sum_j p_ij)
// over the keys j that query row i sees, d_qk = 128 or 128 + 64 (the 64 RoPE dims
// of a key shared by all heads, read from their own tensor), d_v = 128.
//
// A CTA takes one segment of the partition (mla_prefill_schedule.cu) for one
// key head at a time: two tiles A and B of 128 query rows (row r of a tile is
// head r % group of token r / group, so that grouped heads share the loads of their
// key head), walking steps of 128 keys together, so that every key and value
// that lands in shared memory serves 256 rows.  Tensor memory is full: S_A, S_B, O_A,
// O_B take 128 of the 512 columns each, and a tile's weights P overwrite its scores
// as bf16 operands.  The roles, of 12 warps (the last idles):
//   0-3, 4-7  rows of A and of B, a thread per row: S from tensor memory, mask, running
//             maximum and sum in fp32, P back; O read and written at the end.  O is only
//             rescaled when a maximum grows by more than 2^8 over the one in use
//   8         loads: Q of a segment, then chunks of 16 KB through one ring (a step's
//             keys are 64-dim chunks of 128 keys, its values 128-dim chunks of 64)
//   9         MMAs, in the order PV_A(j) QK_A(j+1) PV_B(j) QK_B(j+1): while the rows of one
//             tile take their maximum and exponents, the other tile's products run
//   10        zeroes the value rows behind a sequence's last key, which belong to
//             another sequence (weight 0 times an infinity would be NaN)
// Products stop at multiples of 16 keys behind the last one that a tile sees.
//
// Bound by the tensor cores: a step of both tiles is 2 x 128 x 128 x (d_qk + 128)
// products, 2560 cycles at d_qk = 192, against about 1000 issue slots per scheduler
// for the rows.
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
// registers of a thread: 168 at launch, then a thread of the rows keeps its 128 scores and
// gets some of the others' (256 x 200 + 128 x 104 = 384 x 168)
constexpr int kRowRegs = 200, kOtherRegs = 104;
static_assert(256 * kRowRegs + 128 * kOtherRegs <= kThreads * 168, "a split of what the CTA was launched with");
constexpr int kLoadWarp = 8, kMmaWarp = 9, kZeroWarp = 10;
constexpr int kRows = kPreTiles * kPreTile;
constexpr uint32_t kSlotBytes = 16384;
constexpr uint32_t kTmemCols = 512;
constexpr float kLazy = 8.f;  // log2: how far a maximum may pass the one in use

// shared memory: Q of both tiles, the ring, barriers
template <bool kRope>
struct Layout {
    static constexpr int kChunks = kRope ? 3 : 2;         // 64-dim chunks of a query or key
    static constexpr int kStepSlots = kChunks + 2;        // ring slots of a step: keys, then values
    static constexpr int kSlots = kRope ? 8 : 10;
    static constexpr uint32_t kRing = kPreTiles * kChunks * kSlotBytes;
    static constexpr uint32_t kBars = kRing + kSlots * kSlotBytes;
    static constexpr uint32_t kBytes = kBars + 512 + 1024;  // 1024: room to align the base
};
static_assert(Layout<true>::kBytes <= 232448 && Layout<false>::kBytes <= 232448, "shared memory of a CTA");

// barriers
constexpr int kMaxSlots = 10;
enum { B_FULL = 0, B_EMPTY = B_FULL + kMaxSlots, B_QFULL = B_EMPTY + kMaxSlots, B_QEMPTY = B_QFULL + 2, B_S = B_QEMPTY + 2, B_P = B_S + 2,
       B_PV = B_P + 2, B_OFREE = B_PV + 2, B_TAIL = B_OFREE + 2, B_ZERO = B_TAIL + kMaxSlots, B_FINAL = B_ZERO + kMaxSlots, kNumBars };
static_assert(kNumBars * 8 <= 512, "room for the barriers");

struct Ctx {
    char *base;
    uint64_t *bars;
    unsigned int *status;
    __device__ uint64_t *bar(int i) const { return bars + i; }
    __device__ bool wait(int i, uint32_t parity) const { return mbar_wait(bars + i, parity, status); }
};

// Items of a CTA: (segment, key head).  Heads go in chunks, a chunk's segments longest
// first with its heads side by side, so that the CTAs of a moment share few
// heads' keys (in L2) and the last items are short ones.
struct Walk {
    const PreHeader *header;
    const PreSegment *segments;
    int64_t at, items;
    int h_kv, chunk;
    __device__ Walk(const PrefillParams &p) {
        header = reinterpret_cast<const PreHeader *>(p.metadata);
        segments = reinterpret_cast<const PreSegment *>(header + 1);
        const int n = (int)min((long long)max(0, header->segments), (long long)p.max_segments);
        items = (int64_t)n * p.h_kv;
        h_kv = p.h_kv;
        chunk = p.head_chunk;
        at = blockIdx.x;
        count = n;
    }
    int count;
    __device__ bool next(const PrefillParams &p, PreSegment &s, int &head) {
        if (at >= items) return false;
        // every other round of the CTAs runs backwards: over lengths that fall, each CTA gets its share
        const int64_t round = at / gridDim.x, last = min((long long)items - 1, (long long)(round + 1) * gridDim.x - 1);
        const int64_t i = round & 1 ? last - (at - round * gridDim.x) : at;
        const int64_t per = (int64_t)count * chunk;
        const int c = (int)(i / per);
        const int heads = min(chunk, h_kv - c * chunk);
        const int64_t in = i - c * per;
        s = segments[in / heads];
        head = c * chunk + (int)(in % heads);
        at += gridDim.x;
        // a partition of other lengths must not make the kernel leave its tensors
        const int most = kPreTiles * pre_tile_tokens(p.group);
        if (s.q0 < 0 || s.tokens < 0 || s.tokens > most || (int64_t)s.q0 + s.tokens > p.num_q || s.slot >= p.max_slots ||
            s.keys < 0 || s.k0 < 0 || (int64_t)s.k0 + s.keys > p.num_k || s.step0 < 0 || s.step1 > pre_steps(s.keys)) {
            if ((threadIdx.x & 31) == 0) atomicOr(p.status, MLA_DEVERR_SEQLEN);
            s.tokens = s.step0 = s.step1 = 0;
        }
        return true;
    }
};

// Whether step j of a segment has value rows behind the sequence's last key that a
// product reaches: zeroed, in the slots of the step's values.  The load role says when
// such a step has been issued (B_TAIL of the values' first slot: only then are the
// slots' barriers in the phase that the zeroing waits for), the zero role when it is
// done (B_ZERO).  A slot's next use comes after both, so each barrier is at most one
// phase ahead of who waits for it.
__device__ __forceinline__ bool tail_step(const PreSegment &s, int j) {
    return s.keys - (s.step0 + j) * kPreTile < kPreTile && s.keys % 16 != 0;
}

// what a tile of a segment does: keys that its last token sees, and its steps
struct Tile {
    int seen, steps;
    __device__ Tile(const PrefillParams &p, const PreSegment &s, int t) {
        const int per = pre_tile_tokens(p.group), last = min(s.tokens, (t + 1) * per) - 1;
        seen = last < t * per ? 0 : p.causal ? pre_seen(s, last) : s.keys;
        steps = max(0, min(pre_steps(seen), s.step1) - s.step0);
    }
};

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
__device__ void load_role(const PrefillParams &p, const Ctx &c, const CUtensorMap *mq, const CUtensorMap *mk, const CUtensorMap *mr,
                          const CUtensorMap *mv) {
    using L = Layout<kRope>;
    Walk walk(p);
    PreSegment s;
    int head;
    uint32_t it = 0, qn[kPreTiles] = {0, 0};
    const uint32_t q_bytes = (uint32_t)(pre_tile_tokens(p.group) * p.group) * 128u;
    bool ok = true;
    while (ok && walk.next(p, s, head)) {
        const Tile a(p, s, 0), b(p, s, 1);
        const int n = max(a.steps, b.steps);
        for (int j = -1; ok && j < n; ++j) {
            if (j < 0) {
                // Q of the tiles that walk, each before the first keys are needed
#pragma unroll
                for (int t = 0; t < kPreTiles; ++t) {
                    if (!ok || (t ? b.steps : a.steps) == 0) continue;
                    ok = __all_sync(0xffffffffu, c.wait(B_QEMPTY + t, (qn[t] & 1) ^ 1));
                    if (!ok) continue;
                    ++qn[t];
                    if (elected()) {
                        mbar_arrive_expect_tx(c.bar(B_QFULL + t), L::kChunks * q_bytes);
                        for (int ch = 0; ch < L::kChunks; ++ch)
                            tma_load(smem_u32(c.base + (t * L::kChunks + ch) * kSlotBytes), mq, c.bar(B_QFULL + t), 64 * ch, head * p.group,
                                     s.q0 + t * pre_tile_tokens(p.group));
                    }
                    __syncwarp();
                }
                continue;
            }
            const int k0 = s.k0 + (s.step0 + j) * kPreTile;
            for (int ch = 0; ch < L::kStepSlots && ok; ++ch, ++it) {
                const int slot = it % L::kSlots;
                ok = __all_sync(0xffffffffu, c.wait(B_EMPTY + slot, ((it / L::kSlots) & 1) ^ 1));
                if (!ok) break;
                uint64_t *bar = c.bar(B_FULL + slot);
                const uint32_t dst = smem_u32(c.base + L::kRing + slot * kSlotBytes);
                if (elected()) {
                    mbar_arrive_expect_tx(bar, kSlotBytes);
                    if (ch < 2) {
                        tma_load(dst, mk, bar, 64 * ch, head, k0);
                    } else if (kRope && ch == 2) {
                        tma_load(dst, mr, bar, 0, 0, k0);
                    } else {
                        const int keys = k0 + 64 * (ch - L::kChunks);
                        tma_load(dst, mv, bar, 0, head, keys);
                        tma_load(dst + kSlotBytes / 2, mv, bar, 64, head, keys);
                        if (ch == L::kStepSlots - 1 && tail_step(s, j)) mbar_arrive(c.bar(B_TAIL + (it - 1) % L::kSlots));
                    }
                }
                __syncwarp();
            }
        }
    }
    // nothing may be in flight when the CTA ends (after a wait that gave up, too)
    for (uint32_t i = it > L::kSlots ? it - L::kSlots : 0; i < it; ++i) c.wait(B_FULL + i % L::kSlots, (i / L::kSlots) & 1);
#pragma unroll
    for (int t = 0; t < kPreTiles; ++t)
        if (qn[t]) c.wait(B_QFULL + t, (qn[t] - 1) & 1);
}

// ---------------------------------------------------------------- MMAs
// instruction descriptors whose number of columns follows the keys in sight
__device__ __forceinline__ uint32_t idesc_keys(int keys) { return idesc_bf16(kPreTile, 0, false, false) | ((uint32_t)(keys >> 3) << 17); }
__device__ __forceinline__ int keys16(int keys) { return keys >= kPreTile ? kPreTile : (keys + 15) & ~15; }

template <bool kRope>
__device__ void mma_role(const PrefillParams &p, const Ctx &c, uint32_t tmem) {
    using L = Layout<kRope>;
    constexpr uint32_t kPvDesc = idesc_bf16(kPreTile, kPreHead, false, true);
    Walk walk(p);
    PreSegment s;
    int head;
    uint32_t it = 0, qn[kPreTiles] = {0, 0}, steps[kPreTiles] = {0, 0}, zeroed = 0;  // zeroed: a bit per slot, the phase of its B_ZERO
    const uint32_t ring = smem_u32(c.base + L::kRing), qbase = smem_u32(c.base);
    auto wait = [&](int bar, uint32_t parity) { return __all_sync(0xffffffffu, c.wait(bar, parity)) != 0; };
    while (walk.next(p, s, head)) {
        const Tile tile[kPreTiles] = {Tile(p, s, 0), Tile(p, s, 1)};
        const int n = max(tile[0].steps, tile[1].steps);
        if (n == 0) continue;
        auto last_user = [&](int t, int j) { return t == 1 || tile[1].steps <= j; };  // of step j's keys or values
        auto first_user = [&](int t, int j) { return t == 0 || tile[0].steps <= j; };
        auto free_slots = [&](uint32_t first, int count) {
            for (int i = 0; i < count; ++i) mma_commit(c.bar(B_EMPTY + (first + i) % L::kSlots));
        };
        // S_t = Q_t K(j)^T
        auto scores = [&](int t, int j) {
            const uint32_t k = it + j * L::kStepSlots;
            const uint32_t idesc = idesc_keys(keys16(tile[t].seen - (s.step0 + j) * kPreTile));
#pragma unroll
            for (int ch = 0; ch < L::kChunks; ++ch) {
                const uint32_t slot = (k + ch) % L::kSlots;
                if (first_user(t, j) && !wait(B_FULL + slot, ((k + ch) / L::kSlots) & 1)) return false;
                const uint64_t ad = desc_sw128(qbase + (t * L::kChunks + ch) * kSlotBytes, 16, 1024), bd = desc_sw128(ring + slot * kSlotBytes, 16, 1024);
                if (elected()) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) mma_ss(tmem + t * 128, ad + 2 * i, bd + 2 * i, idesc, ch + i > 0);  // +32 B along the dims
                }
                __syncwarp();
            }
            if (elected()) {
                mma_commit(c.bar(B_S + t));
                if (j == tile[t].steps - 1) mma_commit(c.bar(B_QEMPTY + t));
                if (last_user(t, j)) free_slots(k, L::kChunks);
            }
            __syncwarp();
            return true;
        };
        // O_t (+)= P_t V(j)
        auto values = [&](int t, int j) {
            const uint32_t v = it + j * L::kStepSlots + L::kChunks;
            const int base = (s.step0 + j) * kPreTile, parts = keys16(tile[t].seen - base) / 16;
            if (first_user(t, j)) {
                for (int i = 0; i < 2; ++i)
                    if (!wait(B_FULL + (v + i) % L::kSlots, ((v + i) / L::kSlots) & 1)) return false;
                if (tail_step(s, j)) {
                    const uint32_t slot = v % L::kSlots;
                    if (!wait(B_ZERO + slot, (zeroed >> slot) & 1)) return false;
                    zeroed ^= 1u << slot;
                }
            }
            if (elected()) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint64_t bd = desc_sw128(ring + (v + h) % L::kSlots * kSlotBytes, kSlotBytes / 2, 1024);
#pragma unroll
                    for (int i = 0; i < 4; ++i)  // 16 keys: 2048 B
                        if (4 * h + i < parts) mma_ts(tmem + 256 + t * 128, tmem + t * 128 + 8 * (4 * h + i), bd + 128 * i, kPvDesc, j + h + i > 0);
                }
                mma_commit(c.bar(B_PV + t));
                if (last_user(t, j)) free_slots(v, 2);
            }
            __syncwarp();
            return true;
        };
#pragma unroll
        for (int t = 0; t < kPreTiles; ++t) {
            if (tile[t].steps == 0) continue;
            if (!wait(B_QFULL + t, qn[t] & 1)) return;
            if (!scores(t, 0)) return;
        }
        for (int j = 0; j < n; ++j)
#pragma unroll
            for (int t = 0; t < kPreTiles; ++t) {
                if (j >= tile[t].steps) continue;
                if (j == 0 && !wait(B_OFREE + t, (qn[t] & 1) ^ 1)) return;  // O of the segment before is read
                if (!wait(B_P + t, (steps[t] + j) & 1)) return;
                tc_fence_after();
                if (!values(t, j)) return;
                if (j + 1 < tile[t].steps && !scores(t, j + 1)) return;
            }
        it += n * L::kStepSlots;
#pragma unroll
        for (int t = 0; t < kPreTiles; ++t) {
            if (tile[t].steps) ++qn[t];
            steps[t] += tile[t].steps;
        }
    }
}

// ---------------------------------------------------------------- value rows behind a sequence
template <bool kRope>
__device__ void zero_role(const PrefillParams &p, const Ctx &c) {
    using L = Layout<kRope>;
    Walk walk(p);
    PreSegment s;
    int head;
    uint32_t it = 0, tails = 0;  // tails: a bit per slot, the phase of its B_TAIL
    const int lane = threadIdx.x & 31;
    while (walk.next(p, s, head)) {
        const Tile a(p, s, 0), b(p, s, 1);
        const int n = max(a.steps, b.steps);
        if (n > 0 && tail_step(s, n - 1)) {
            const int valid = s.keys - (s.step0 + n - 1) * kPreTile;  // keys of the last step
            const uint32_t v = it + (n - 1) * L::kStepSlots + L::kChunks, first = v % L::kSlots;
            if (!__all_sync(0xffffffffu, c.wait(B_TAIL + first, (tails >> first) & 1))) return;
            tails ^= 1u << first;
            for (int i = 0; i < 2; ++i)
                if (!__all_sync(0xffffffffu, c.wait(B_FULL + (v + i) % L::kSlots, ((v + i) / L::kSlots) & 1))) return;
            // rows valid .. of the 16 that the products reach, all 256 bytes of each
            for (int i = lane; i < (16 - valid % 16) * 16; i += 32) {
                const int row = valid + i / 16, piece = i % 16;
                const uint32_t slot = (v + row / 64) % L::kSlots;
                sts128(smem_u32(c.base + L::kRing + slot * kSlotBytes) + (piece / 8) * (kSlotBytes / 2) + (row % 64) * 128 + (piece % 8) * 16, 0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(c.bar(B_ZERO + first));
        }
        it += n * L::kStepSlots;
    }
}

// ---------------------------------------------------------------- rows
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ void row_role(const PrefillParams &p, const Ctx &c, uint32_t tmem, int t) {
    const int warp = threadIdx.x >> 5, r = threadIdx.x & (kPreTile - 1);
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_col = tmem + lane_base + t * 128, o_col = tmem + lane_base + 256 + t * 128;
    const int per = pre_tile_tokens(p.group), in_tile = r / p.group, hh = r - in_tile * p.group;
    const float lazy = kLazy / p.scale_log2;  // in units of the raw scores
    Walk walk(p);
    PreSegment s;
    int head;
    uint32_t phase = 0;  // steps of this tile so far
    while (walk.next(p, s, head)) {
        const Tile tile(p, s, t);
        const int token = t * per + in_tile;
        const bool on = in_tile < per && token < s.tokens;
        const int seen = !on ? 0 : p.causal ? pre_seen(s, token) : s.keys;
        float m = -INFINITY, l = 0.f;  // maximum in use (raw scores), sum of the weights
        for (int j = 0; j < tile.steps; ++j, ++phase) {
            if (!__all_sync(0xffffffffu, c.wait(B_S + t, phase & 1))) return;
            tc_fence_after();
            float x[128];
            {
                uint32_t u[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_ld32(s_col + 32 * i, u[i]);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 128; ++i) x[i] = __uint_as_float(u[i / 32][i % 32]);
            }
            const int left = seen - (s.step0 + j) * kPreTile;
            if (left < kPreTile) {
#pragma unroll
                for (int i = 0; i < 128; ++i) x[i] = i < left ? x[i] : -INFINITY;
            }
            float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int i = 4; i < 124; i += 8) {
#pragma unroll
                for (int k = 0; k < 4; ++k) mx[k] = max3f(mx[k], x[i + 2 * k], x[i + 2 * k + 1]);
            }
            float top = max3f(max3f(mx[0], mx[1], mx[2]), max3f(mx[3], x[124], x[125]), fmaxf(x[126], x[127]));
            const bool grow = top > m + lazy;  // (m = -inf: the first score of the row)
            const float m_new = grow ? top : m;
            if (j > 0 && __any_sync(0xffffffffu, grow)) {
                // O is in units of the old maximum, or of none
                if (!__all_sync(0xffffffffu, c.wait(B_PV + t, (phase - 1) & 1))) return;
                tc_fence_after();
                const float f = grow ? (m == -INFINITY ? 0.f : exp2_fast((m - m_new) * p.scale_log2)) : 1.f;
                l *= f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t o[32];
                    tmem_ld32(o_col + 32 * i, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                    tmem_st32(o_col + 32 * i, o);
                }
                tmem_wait_st();
            }
            m = m_new;
            const float shift = m == -INFINITY ? 0.f : -m * p.scale_log2;
            const uint64_t scale2 = f2_pack(p.scale_log2, p.scale_log2), shift2 = f2_pack(shift, shift);
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float a, b;
                    f2_unpack(f2_fma(f2_pack(x[64 * h + 2 * i], x[64 * h + 2 * i + 1]), scale2, shift2), a, b);
                    a = exp2_fast(a);
                    b = exp2_fast(b);
                    sum[i & 1] = f2_add(sum[i & 1], f2_pack(a, b));
                    w[i] = pack_bf16(a, b);
                }
                tmem_st32(s_col + 32 * h, w);
            }
            {
                float a, b;
                f2_unpack(f2_add(sum[0], sum[1]), a, b);
                l += a + b;
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(c.bar(B_P + t));
        }
        // epilogue: o = O / l, lse
        float lse = l == 0.f ? -INFINITY : m * p.scale + logf(l);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t row = (int64_t)(s.q0 + token) * p.h_q + head * p.group + hh;
        const int64_t part = ((int64_t)s.slot * p.h_kv + head) * kRows + t * kPreTile + r;
        if (on) {
            if (s.slot < 0) p.lse[row] = lse;
            else p.lse_part[part] = lse;
        }
        if (tile.steps == 0) {
            if (on && s.slot < 0)
                for (int i = 0; i < kPreHead / 8; ++i) reinterpret_cast<uint4 *>(p.out + row * kPreHead)[i] = make_uint4(0, 0, 0, 0);
            continue;
        }
        if (!__all_sync(0xffffffffu, c.wait(B_PV + t, (phase - 1) & 1))) return;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t o[32];
            tmem_ld32(o_col + 32 * i, o);
            tmem_wait_ld();
            if (i == 3) {
                tc_fence_before();
                mbar_arrive(c.bar(B_OFREE + t));
            }
            if (!on) continue;
            if (s.slot < 0) {
                uint4 *dst = reinterpret_cast<uint4 *>(p.out + row * kPreHead + 32 * i);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = pack_bf16(__uint_as_float(o[8 * k + 2 * e]) * inv, __uint_as_float(o[8 * k + 2 * e + 1]) * inv);
                    dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            } else {
                float4 *dst = reinterpret_cast<float4 *>(p.o_part + part * kPreHead + 32 * i);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    dst[k] = make_float4(__uint_as_float(o[4 * k]) * inv, __uint_as_float(o[4 * k + 1]) * inv, __uint_as_float(o[4 * k + 2]) * inv,
                                         __uint_as_float(o[4 * k + 3]) * inv);
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
        for (int i = 0; i < L::kSlots; ++i) {
            mbar_init(c.bar(B_FULL + i), 1);
            mbar_init(c.bar(B_EMPTY + i), 1);
            mbar_init(c.bar(B_TAIL + i), 1);
            mbar_init(c.bar(B_ZERO + i), 1);
        }
        for (int t = 0; t < kPreTiles; ++t) {
            mbar_init(c.bar(B_QFULL + t), 1);
            mbar_init(c.bar(B_QEMPTY + t), 1);
            mbar_init(c.bar(B_S + t), 1);
            mbar_init(c.bar(B_P + t), kPreTile);
            mbar_init(c.bar(B_PV + t), 1);
            mbar_init(c.bar(B_OFREE + t), kPreTile);
        }
        mbar_init(c.bar(B_FINAL), 1);
        fence_mbar_init();
    }
    if (warp == kLoadWarp && elect_one_lane()) {
        tma_prefetch_desc(&mq);
        tma_prefetch_desc(&mk);
        if (kRope) tma_prefetch_desc(&mr);
        tma_prefetch_desc(&mv);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&s_tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    griddep_wait();
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
        row_role(p, c, tmem, warp >> 2);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kLoadWarp) {
            load_role<kRope>(p, c, &mq, &mk, &mr, &mv);
        } else if (warp == kMmaWarp) {
            mma_role<kRope>(p, c, tmem);
            if (elected()) mma_commit(c.bar(B_FINAL));  // every MMA of this thread is done before tensor memory is released
            __syncwarp();
            c.wait(B_FINAL, 0);
        } else if (warp == kZeroWarp) {
            zero_role<kRope>(p, c);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------- combine of cut blocks
// A warp per (block, head, row): o = sum_s w_s o_s, w_s = exp(lse_s - lse); a part in
// which the row saw nothing (lse -inf) was not written and is not read.
constexpr int kCombineWarps = 8;

__global__ void __launch_bounds__(kCombineWarps * 32) prefill_combine_kernel(const __grid_constant__ PrefillParams p) {
    griddep_wait();
    const PreHeader *header = reinterpret_cast<const PreHeader *>(p.metadata);
    const PreCut *cuts = reinterpret_cast<const PreCut *>(reinterpret_cast<const PreSegment *>(header + 1) + p.max_segments);
    const int lane = threadIdx.x & 31, per = pre_tile_tokens(p.group);
    const int n = min(header->cuts, p.max_slots);
    const int64_t total = (int64_t)n * p.h_kv * kRows, stride = (int64_t)gridDim.x * kCombineWarps;
    for (int64_t i = (int64_t)blockIdx.x * kCombineWarps + (threadIdx.x >> 5); i < total; i += stride) {
        const int r = (int)(i % kRows), head = (int)(i / kRows % p.h_kv);
        const PreCut cut = cuts[i / kRows / p.h_kv];
        const int t = r / kPreTile, in_tile = (r % kPreTile) / p.group, hh = (r % kPreTile) - in_tile * p.group, token = t * per + in_tile;
        if (in_tile >= per || token >= cut.tokens || cut.slot0 < 0 || cut.slot0 + cut.count > p.max_slots || (int64_t)cut.q0 + token >= p.num_q) continue;
        const int64_t step = (int64_t)p.h_kv * kRows, first = ((int64_t)cut.slot0 * p.h_kv + head) * kRows + r;
        float top = -INFINITY;
        for (int k = 0; k < cut.count; ++k) top = fmaxf(top, p.lse_part[first + k * step]);
        const float base = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < cut.count; ++k) {
            const float lse = p.lse_part[first + k * step];
            if (lse == -INFINITY) continue;
            const float w = exp2_fast((lse - base) * 1.4426950408889634f);
            const float4 x = reinterpret_cast<const float4 *>(p.o_part + (first + k * step) * kPreHead)[lane];
            sum += w;
            o.x = fmaf(w, x.x, o.x);
            o.y = fmaf(w, x.y, o.y);
            o.z = fmaf(w, x.z, o.z);
            o.w = fmaf(w, x.w, o.w);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t row = (int64_t)(cut.q0 + token) * p.h_q + head * p.group + hh;
        reinterpret_cast<uint2 *>(p.out + row * kPreHead)[lane] = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        if (lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : base + logf(sum);
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
    const int64_t items = p.max_segments * p.h_kv;
    const unsigned grid = (unsigned)(items < p.sms ? items : p.sms);
    e = launch_after(prefill_kernel<kRope>, dim3(grid), dim3(kThreads), Layout<kRope>::kBytes, stream, mq, mk, mr, mv, p);
    if (e != cudaSuccess || p.max_slots == 0) return e;
    return launch_after(prefill_combine_kernel, dim3(2 * p.sms), dim3(kCombineWarps * 32), 0, stream, p);
}

}  // namespace

cudaError_t launch_prefill(const PrefillParams &p, cudaStream_t stream) {
    return p.rope ? launch<true>(p, stream) : launch<false>(p, stream);
}

}  // namespace mla
