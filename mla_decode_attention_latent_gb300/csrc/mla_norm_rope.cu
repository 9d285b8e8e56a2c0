// Norm and rotation of rows in one pass: query or key heads, and latent rows on
// their way into the paged cache.
//
//   y = x / sqrt(mean(x^2) + eps) * w        (heads, or the 512 latent dims of a row; optional)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t), each times `scale`, for the
//   pairs of the last rope_dim values, t = position * frequency
// in fp32 from bf16 values, rounded once when a value is stored.
//
// Angles.  A frequency is a whole number of 2^-64 turns per position, so the
// phase of a position is one 64-bit product that drops whole turns by itself: exact,
// at any position, where an angle in radians loses a bit for every doubling, but for the frequency's own
// roundings, half a unit and those of the doubles that mla_rope_turns computes it in (2^-50 of it: at position
// 2^31 2^-21 turns at most, 2^-24 measured).  Its distance to the nearest whole turn goes to
// sincospif as a float, so a small angle keeps its 24 bits.
//
// Heads: a group of 8 lanes per head (32 above 256 values), lane l taking the 16-byte pieces l, l + 8, ...
// (128 contiguous bytes per load and group; a head of 192 keeps every lane busy,
// where a warp per head would idle a quarter of them).  A CTA takes a run of
// consecutive heads of consecutive tokens and computes the tokens' sines once, in
// shared memory, for all of their heads.  Everything is loaded once and stays in
// registers, the next head on its way while one is computed; the partner of a value in
// the half layout is in the same lane (rotations of 128 values), comes from the lane that
// has it, or is loaded again where heads are cut oddly, in all cases before anything of its
// head is stored, so that a call may be in place.
// Bound by HBM on prompts (4096 tokens of 128 heads of 192 values: 68.6 us, 5.9 TB/s), by
// the launch on single tokens (64 tokens: 2.1 us), and between them, where the rows come out
// of L2, by latency (1777 tokens of 40 heads of 128: 8.6 us, one wave of CTAs at half of the issue
// slots; two heads under way per group instead of one gained nothing).  The half layout of heads of 192
// values with a norm spills 12 bytes at its 64 registers.
//
// Rows: a warp per cached row, the 512 latent dims as 64 pieces over its lanes and
// the RoPE key as 8 more; each lane computes one of the row's 32 angles.  A step of 64 rows
// takes 1.9 us, 5000 bf16 rows 3.6, 32,768 rows into e4m3 pages 15.1 (3.8 TB/s, two thirds of
// the issue slots: a warp's row is one chain from its loads to its stores).
#include <cuda_runtime.h>

#include "mla_internal.h"
#include "mla_sm103.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kNarrow = 8, kWide = 32;          // lanes of a head of up to 256 values, and of a wider one
constexpr int kMaxAngles = 4096;                // of a CTA: 32 KB

// cosine and sine of position * turns, times scale
__device__ __forceinline__ float2 angle(int position, int64_t turns, float scale) {
    const int64_t phase = (int64_t)((uint64_t)turns * (uint64_t)(int64_t)position);  // turns to the nearest whole one, units of 2^-64
    float s, c;
    sincospif((float)phase * 0x1p-63f, &s, &c);
    return make_float2(c * scale, s * scale);
}

__device__ __forceinline__ void widen8(uint4 x, float (&f)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 round8(const float (&f)[8]) {
    return make_uint4(sm103::pack_bf16(f[0], f[1]), sm103::pack_bf16(f[2], f[3]), sm103::pack_bf16(f[4], f[5]),
                      sm103::pack_bf16(f[6], f[7]));
}

// sum of the squares of 8 values, each times k
__device__ __forceinline__ float squares(uint4 x, float k = 1.f) {
    float f[8], s = 0.f;
    widen8(x, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(f[i] * k, f[i] * k, s);
    return s;
}

// 8 values times 2^90: exact for values below 2^-45, which stay bf16 values
__device__ __forceinline__ uint4 raised8(uint4 x) {
    auto raised = [](uint32_t pair) {
        uint32_t y;
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(pair), "r"(0x6c806c80u));
        return y;
    };
    return make_uint4(raised(x.x), raised(x.y), raised(x.z), raised(x.w));
}

// What is added to the mean of the squares: with nothing, the reciprocal of a root can leave fp32
// (rows of bf16's subnormal values), with the smallest eps it is at most 2^75.
enum Eps { kSome, kNone };

// 1 / sqrt(mean of x^2 + eps) for a row whose sum of squares of k x is sum(k), the
// same in all of its lanes.  Values near the ends of the type, whose squares leave
// fp32, are scaled by a power of two first; the whole warp takes that way together.
// The power is in the result, but for small values (each below 2^-45) without an eps: they are to
// be multiplied by 2^90 by raise(), and the result is theirs.
template <Eps kEps, typename Sum, typename Raise>
__device__ __forceinline__ float inverse_rms(Sum sum, Raise raise, int d, float eps) {
    float s = sum(1.f);
    const float share = 1.f / (float)d;
    float inv = rsqrtf(s * share + eps);
    const bool large = !(s < 0x1p120f), small = s < 0x1p-90f && eps < 0x1p-60f;
    if (__any_sync(0xffffffffu, large || small)) {
        const float k = large ? 0x1p-70f : kEps == kNone ? 0x1p90f : 0x1p70f;
        s = sum(k);
        if constexpr (kEps == kNone) {
            if (large) inv = k * rsqrtf(s * share);
            if (small) {
                inv = rsqrtf(s * share);
                raise();
            }
        } else if (large || small) {
            inv = k * rsqrtf(s * share + eps * k * k);
        }
    }
    return inv;
}

__device__ __forceinline__ void scale8(float (&f)[8], uint4 w, float r) {
    float g[8];
    widen8(w, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] * r * g[i];  // (x r first: at most sqrt(d))
}

// A pair turned: rounded the same way wherever a partner comes from, so that a call in place has
// the bits of one that is not.
__device__ __forceinline__ float turned_low(float a, float b, float2 t) { return __fmaf_rn(a, t.x, -__fmul_rn(b, t.y)); }
__device__ __forceinline__ float turned_high(float a, float b, float2 t) { return __fmaf_rn(b, t.x, __fmul_rn(a, t.y)); }
__device__ __forceinline__ void turn(float &a, float &b, float2 t) {
    const float x = a;
    a = turned_low(x, b, t);
    b = turned_high(x, b, t);
}

// 8 values of the rotated part turned by the angles of their pairs.  Interleaved:
// four pairs.  Halves: the values of the first (low) or second half, `other` their partners.
template <bool kInterleaved>
__device__ __forceinline__ void rotate8(float (&f)[8], const float (&other)[8], const float2 (&cs)[8], bool low) {
    if constexpr (kInterleaved) {
#pragma unroll
        for (int k = 0; k < 4; ++k) turn(f[2 * k], f[2 * k + 1], cs[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = low ? turned_low(f[k], other[k], cs[k]) : turned_high(other[k], f[k], cs[k]);
    }
}

// Where the partner of a rotated value is.
enum Pairs {
    kNeighbours,  // interleaved: in the same piece
    kOwn,         // halves of as many pieces as lanes, from the first lane on: the lane's piece before or behind
    kOther,       // halves of a power of two of pieces, both inside the lanes: the lane `half` away
    kReload,      // any other place: loaded again
};

// kGroup: lanes of a head, kPieces: 16-byte pieces of a lane, kEps: of a norm
template <int kGroup, int kPieces, bool kNorm, Pairs kPairs, Eps kEps>
__global__ void __launch_bounds__(kThreads, kPairs == kReload ? 2 : kPieces <= 3 ? 4 : 3) norm_rope_kernel(const NormRopeParams p, int rows_per_cta) {
    constexpr int kGroups = kThreads / kGroup;
    extern __shared__ float2 s_angle[];  // [tokens of the CTA][rope_dim / 2]
    __shared__ uint4 s_weight[kGroup * kPieces];
    sm103::griddep_wait();
    const int group = threadIdx.x / kGroup, lane = threadIdx.x % kGroup;
    const int64_t rows = p.tokens * p.heads, row0 = (int64_t)blockIdx.x * rows_per_cta;
    const int64_t row1 = min((long long)row0 + rows_per_cta, (long long)rows);
    const int64_t token0 = row0 / p.heads;
    const int head0 = (int)(row0 - token0 * p.heads), count = (int)(row1 - row0);
    const int pairs = p.rope.positions ? p.rope.rope_dim / 2 : 0;
    const int piece0 = p.first / 8 + lane, pieces = p.d / 8, rope0 = pieces - pairs / 4, half = pairs / 8;
    constexpr int kAgain = kPairs == kReload ? kPieces : 1;
    // one row's pieces (and, loaded again, the partners of its rotated ones)
    struct Pieces {
        uint4 x[kPieces], again[kAgain];
    };
    auto place = [&](int i, int &token, int &head) {
        const unsigned at = (unsigned)(head0 + i);
        token = (int)(at / (unsigned)p.heads);
        head = (int)(at - (unsigned)token * (unsigned)p.heads);
    };
    auto load = [&](int i, Pieces &v) {
        int token, head;
        place(min(i, count - 1), token, head);
        const uint4 *src = reinterpret_cast<const uint4 *>(p.x + (token0 + token) * p.x_token + head * p.x_head);
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const int at = piece0 + kGroup * j;
            v.x[j] = at < pieces ? src[at] : make_uint4(0, 0, 0, 0);
            if constexpr (kPairs == kReload) v.again[j] = at >= rope0 && at < pieces ? src[at - rope0 < half ? at + half : at - half] : make_uint4(0, 0, 0, 0);
        }
    };
    Pieces next;
    load(group, next);  // under way while the angles are computed
    if (pairs) {
        const int tokens = (head0 + count - 1) / p.heads + 1;
        for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
            const int t = i / pairs, k = i - t * pairs;
            s_angle[i] = angle(p.rope.positions[token0 + t], p.rope.turns[k], p.rope.scale);
        }
    }
    // the weights, in shared memory: in registers they would cost a CTA per SM
    if constexpr (kNorm) {
        if (threadIdx.x < pieces - p.first / 8) s_weight[threadIdx.x] = reinterpret_cast<const uint4 *>(p.weight)[threadIdx.x];
    }
    if (pairs || kNorm) __syncthreads();
    // every group makes the same number of turns, for the shuffles
    for (int r = group; r - group < count; r += kGroups) {
        Pieces v = next;
        if (r - group + kGroups < count) load(r + kGroups, next);
        if constexpr (kPairs == kReload) __syncwarp();  // in place: no lane stores a head before all have loaded it
        int token, head;
        place(min(r, count - 1), token, head);
        uint4 *dst = reinterpret_cast<uint4 *>(p.out + (token0 + token) * p.out_token + head * p.out_head);
        float inv = 1.f;
        if constexpr (kNorm) {
            inv = inverse_rms<kEps>([&](float k) {
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < kPieces; ++j) s += squares(v.x[j], k);
#pragma unroll
                for (int off = 1; off < kGroup; off <<= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
                return s;
            }, [&] {
#pragma unroll
                for (int j = 0; j < kPieces; ++j) {
                    v.x[j] = raised8(v.x[j]);
                    if constexpr (kPairs == kReload) v.again[j] = raised8(v.again[j]);
                }
            }, p.d, p.eps);
        }
        const float2 *cs = s_angle + token * pairs;
        if constexpr (kPairs == kOwn) {
            // the halves are whole pieces of this lane: both are turned by the same angles
            const int low = (rope0 - p.first / 8) / kGroup;
            if (r >= count) continue;
            float f[kPieces][8];
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                widen8(v.x[j], f[j]);
                if constexpr (kNorm) scale8(f[j], s_weight[piece0 + kGroup * j], inv);
            }
#pragma unroll
            for (int j = 0; j + 1 < kPieces; ++j) {
                if (j != low) continue;
                const float4 *from = reinterpret_cast<const float4 *>(cs + 8 * lane);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 two = from[k];
                    turn(f[j][2 * k], f[j + 1][2 * k], make_float2(two.x, two.y));
                    turn(f[j][2 * k + 1], f[j + 1][2 * k + 1], make_float2(two.z, two.w));
                }
            }
#pragma unroll
            for (int j = 0; j < kPieces; ++j)
                if (kNorm || j == low || j == low + 1) dst[piece0 + kGroup * j] = round8(f[j]);
                else dst[piece0 + kGroup * j] = v.x[j];
        } else {
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                const int at = piece0 + kGroup * j, part = at - rope0;
                const bool turned = part >= 0 && at < pieces, low = part < half;
                uint4 other = make_uint4(0, 0, 0, 0);
                if constexpr (kPairs == kOther) {
                    if (__any_sync(0xffffffffu, turned)) {
                        other.x = __shfl_xor_sync(0xffffffffu, v.x[j].x, half);
                        other.y = __shfl_xor_sync(0xffffffffu, v.x[j].y, half);
                        other.z = __shfl_xor_sync(0xffffffffu, v.x[j].z, half);
                        other.w = __shfl_xor_sync(0xffffffffu, v.x[j].w, half);
                    }
                } else if constexpr (kPairs == kReload) {
                    other = v.again[j];
                }
                if (r >= count || at >= pieces) continue;
                uint4 y = v.x[j];
                if (kNorm || turned) {
                    float f[8], g[8];
                    widen8(v.x[j], f);
                    if constexpr (kNorm) scale8(f, s_weight[at], inv);
                    if (turned) {
                        float2 t[8];
                        // two angles a load
                        const float4 *from = reinterpret_cast<const float4 *>(cs + (kPairs == kNeighbours ? 4 * part : 8 * (low ? part : part - half)));
#pragma unroll
                        for (int k = 0; k < (kPairs == kNeighbours ? 2 : 4); ++k) {
                            const float4 two = from[k];
                            t[2 * k] = make_float2(two.x, two.y);
                            t[2 * k + 1] = make_float2(two.z, two.w);
                        }
                        if constexpr (kPairs != kNeighbours) {
                            widen8(other, g);
                            if constexpr (kNorm) scale8(g, s_weight[low ? at + half : at - half], inv);
                        }
                        rotate8<kPairs == kNeighbours>(f, g, t, low);
                    }
                    y = round8(f);
                }
                dst[at] = y;
            }
        }
    }
}

template <int kGroup, int kPieces, bool kNorm, Eps kEps>
void (*heads_kernel(Pairs pairs))(NormRopeParams, int) {
    switch (pairs) {
        case kNeighbours: return norm_rope_kernel<kGroup, kPieces, kNorm, kNeighbours, kEps>;
        case kOwn: return norm_rope_kernel<kGroup, kPieces, kNorm, (kGroup == kNarrow && kPieces > 1) ? kOwn : kReload, kEps>;  // (halves of 64 values)
        case kOther: return norm_rope_kernel<kGroup, kPieces, kNorm, kOther, kEps>;
        default: return norm_rope_kernel<kGroup, kPieces, kNorm, kReload, kEps>;
    }
}

template <int kGroup, int kPieces>
cudaError_t launch_heads(const NormRopeParams &p, cudaStream_t stream) {
    constexpr int kGroups = kThreads / kGroup;
    const int pairs = p.rope.positions ? p.rope.rope_dim / 2 : 0;
    const int64_t rows = p.tokens * p.heads;
    int sms = 0;
    cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    // as many turns of the groups as leave about kCtas CTAs per SM, at most kTurns: they share
    // the tokens' angles (at most 1 / 4 / 8 / 16 turns: 1777 tokens of 40 heads of 128 10.5 / 9.0 /
    // 8.6 / 8.6 us, 4096 tokens of 128 heads of 192 81.8 / 68.8 / 68.7 / 69.0)
    constexpr int64_t kCtas = 3, kTurns = 8;
    const int64_t turns = (rows + kGroups * kCtas * sms - 1) / (kGroups * kCtas * sms);
    int per_cta = kGroups * (int)(turns < kTurns ? turns : kTurns);
    if (pairs) {
        // the tokens that a run of heads touches have their angles in shared memory
        const int tokens = kMaxAngles / pairs;
        while (per_cta > 1 && (per_cta - 1) / p.heads + 2 > tokens) per_cta /= 2;
    }
    const size_t smem = pairs ? ((size_t)(per_cta - 1) / p.heads + 2) * pairs * sizeof(float2) : 0;
    const int64_t ctas = (rows + per_cta - 1) / per_cta;
    if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
    const int half = pairs / 8, rel = (p.d - p.first) / 8 - pairs / 4;  // pieces of a half, and before the first
    const Pairs where = p.rope.interleaved || !pairs ? kNeighbours : half == kGroup && rel % kGroup == 0 ? kOwn
                        : 2 * half <= kGroup && (half & (half - 1)) == 0 && rel % (2 * half) == 0 ? kOther : kReload;
    // (the raised rows of calls without an eps in a kernel of their own: in the others, which never meet them, they cost
    // 4096 tokens of 32 heads of 192, neighbours turned, 16.9 us for 15.9)
    auto kernel = !p.weight ? heads_kernel<kGroup, kPieces, false, kSome>(where)
                  : p.eps > 0.f ? heads_kernel<kGroup, kPieces, true, kSome>(where) : heads_kernel<kGroup, kPieces, true, kNone>(where);
    return launch_after(kernel, dim3((unsigned)ctas), dim3(kThreads), smem, stream, p, per_cta);
}

// ---------------------------------------------------------------- rows into the cache
constexpr int kRowWarps = 4;  // (8: 32,768 e4m3 rows 15.3 us for 15.1, 5000 bf16 rows 3.64 for 3.55)
constexpr int kRopeDims = kDqk - kDv;

// e4m3(y / c) of 8 values, the quotient by a reciprocal and a fused remainder (Markstein's
// method).  With inv the rounded reciprocal of c, q = y inv, the remainder
// y - q c is exact in one fused operation, and q + (y - q c) inv is the quotient to
// within its last bit.  Two values per instruction.  A zero's code is +0.
__device__ __forceinline__ uint2 quantise8(const float (&y)[8], float c, float inv) {
    uint32_t code[4];
    const uint64_t inv2 = sm103::f2_pack(inv, inv), minus_c2 = sm103::f2_pack(-c, -c), zero2 = sm103::f2_pack(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint64_t v = sm103::f2_pack(y[2 * k], y[2 * k + 1]);
        const uint64_t q = sm103::f2_fma(v, inv2, zero2), r = sm103::f2_fma(q, minus_c2, v);
        float a, b;
        sm103::f2_unpack(sm103::f2_fma(r, inv2, q), a, b);
        code[k] = sm103::pack_e4m3x2(a, b);
    }
    return make_uint2(code[0] | (code[1] << 16), code[2] | (code[3] << 16));
}

// the same for rows so small that the remainder and the reciprocal leave the normal range
__device__ __forceinline__ uint2 quantise8_small(const float (&y)[8], float c) {
    uint32_t code[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) code[k] = sm103::pack_e4m3x2(y[2 * k] / c + 0.f, y[2 * k + 1] / c + 0.f);
    return make_uint2(code[0] | (code[1] << 16), code[2] | (code[3] << 16));
}

// max |y| / 448, rounded to nearest: with 1/448 rounded, one fused remainder makes it so
__device__ __forceinline__ float row_scale(float top) {
    constexpr float kInv = 1.f / 448.f;
    const float q = top * kInv;
    return fmaf(fmaf(q, -448.f, top), kInv, q);
}

template <int D, bool kE4m3, Eps kEps>
__global__ void __launch_bounds__(kRowWarps * 32) place_rows_kernel(const PlaceRowsParams p) {
    constexpr bool kRope = D > kDv;
    sm103::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    if (r >= p.num_rows) return;
    const uint4 *src = reinterpret_cast<const uint4 *>(p.latent + r * p.latent_stride);
    const uint4 raw[2] = {src[lane], src[lane + 32]};
    uint4 key = make_uint4(0, 0, 0, 0), other = make_uint4(0, 0, 0, 0);
    const int half = kRopeDims / 16;
    if constexpr (kRope) {
        const uint4 *at = reinterpret_cast<const uint4 *>(p.k_rope + r * p.k_rope_stride);
        key = at[lane & 7];
        if (!p.rope.interleaved) other = at[(lane & 7) ^ half];
    }
    const int64_t slot = p.slots[r];
    float f[3][8];
    widen8(raw[0], f[0]);
    widen8(raw[1], f[1]);
    if (p.weight) {
        const float inv = inverse_rms<kEps>([&](float k) {
            float s = squares(raw[0], k) + squares(raw[1], k);
#pragma unroll
            for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            return s;
        }, [&] {
#pragma unroll
            for (int k = 0; k < 8; ++k) f[0][k] *= 0x1p90f, f[1][k] *= 0x1p90f;
        }, kDv, p.eps);
        const uint4 *w = reinterpret_cast<const uint4 *>(p.weight);
        scale8(f[0], w[lane], inv);
        scale8(f[1], w[lane + 32], inv);
    }
    if constexpr (kRope) {
        // lane i turns pair i; eight lanes (four groups of them, alike) need 8 or 4 pairs each
        const float2 mine = angle(p.rope.positions[r], p.rope.turns[lane], p.rope.scale);
        const int i = lane & 7;
        float2 cs[8];
        float g[8];
        widen8(key, f[2]);
        if (p.rope.interleaved) {
#pragma unroll
            for (int k = 0; k < 4; ++k) cs[k] = make_float2(__shfl_sync(0xffffffffu, mine.x, 4 * i + k), __shfl_sync(0xffffffffu, mine.y, 4 * i + k));
            rotate8<true>(f[2], g, cs, true);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                cs[k] = make_float2(__shfl_sync(0xffffffffu, mine.x, 8 * (i & 3) + k), __shfl_sync(0xffffffffu, mine.y, 8 * (i & 3) + k));
            widen8(other, g);
            rotate8<false>(f[2], g, cs, i < half);
        }
    }
    if (p.latent_out) {
        uint4 *out = reinterpret_cast<uint4 *>(p.latent_out + r * p.latent_out_stride);
        out[lane] = round8(f[0]);
        out[lane + 32] = round8(f[1]);
    }
    if (kRope && p.k_rope_out && lane < 8) reinterpret_cast<uint4 *>(p.k_rope_out + r * p.k_rope_out_stride)[lane] = round8(f[2]);
    if (slot < 0) return;
    if (slot >= p.num_blocks * kPage) {
        if (lane == 0) atomicOr(p.status, MLA_DEVERR_BLOCK_ID);
        return;
    }
    if constexpr (!kE4m3) {
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.cache) + slot * D);
        dst[lane] = round8(f[0]);
        dst[lane + 32] = round8(f[1]);
        if (kRope && lane < 8) dst[64 + lane] = round8(f[2]);
    } else {
        // the row's largest magnitude, by its bits: infinities and NaN on top
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 3; ++j)
#pragma unroll
            for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(f[j][k]) & 0x7fffffffu);
        top = __reduce_max_sync(0xffffffffu, top);
        // (rows of values that fp32 holds to fewer bits take divisions)
        const bool small = top < 0x12800000u;  // 2^-90: a scale below 2^-98
        const float m = __uint_as_float(top);
        const float c = top >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : !top ? 1.f : small ? fmaxf(m / 448.f, 0x1p-149f) : row_scale(m);
        uint8_t *page = static_cast<uint8_t *>(p.cache) + (slot / kPage) * (int64_t)MLA_FP8_PAGE_BYTES(kDqk);
        const int off = (int)(slot % kPage);
        if (lane == 0) {
            if (!(c < (float)MLA_FP8_SCALE_LIMIT)) atomicOr(p.status, MLA_DEVERR_SCALE);
            reinterpret_cast<float *>(page + kPage * kDqk)[off] = c;
        }
        uint2 *dst = reinterpret_cast<uint2 *>(page + off * kDqk);
        if (small && top) {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (j < 2 || lane < 8) dst[lane + 32 * j] = quantise8_small(f[j], c);
        } else {
            const float inv = 1.f / c;
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (j < 2 || lane < 8) dst[lane + 32 * j] = quantise8(f[j], c, inv);
        }
    }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams &p, cudaStream_t stream) {
    const int pieces = (p.d - p.first) / 8;
    if (pieces > 4 * kNarrow) return launch_heads<kWide, 3>(p, stream);
    switch ((pieces + kNarrow - 1) / kNarrow) {
        case 1: return launch_heads<kNarrow, 1>(p, stream);
        case 2: return launch_heads<kNarrow, 2>(p, stream);
        case 3: return launch_heads<kNarrow, 3>(p, stream);
        default: return launch_heads<kNarrow, 4>(p, stream);
    }
}

template <Eps kEps>
static void (*rows_kernel(int d, bool e4m3))(PlaceRowsParams) {
    return e4m3 ? place_rows_kernel<kDqk, true, kEps> : d == kDqk ? place_rows_kernel<kDqk, false, kEps> : place_rows_kernel<kDv, false, kEps>;
}

cudaError_t launch_place_rows(const PlaceRowsParams &p, int d, bool e4m3, cudaStream_t stream) {
    const unsigned grid = (unsigned)((p.num_rows + kRowWarps - 1) / kRowWarps);
    auto kernel = p.eps > 0.f ? rows_kernel<kSome>(d, e4m3) : rows_kernel<kNone>(d, e4m3);
    return launch_after(kernel, dim3(grid), dim3(kRowWarps * 32), 0, stream, p);
}

}  // namespace mla
