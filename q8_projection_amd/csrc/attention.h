// attention.h -- what the attention's kernels share: the cache's values as operands of
// the f16 matrix cores, queries and weights in two binary16 words, the end of a row.
//
// Every value of the cache is a binary16 number times a power of two exactly, so one side of
// each product needs no rounding, and the f32 side is split in two words, x = hi + lo with
// hi = rne16(x), lo = rne16(x - hi): 22 bits of it, as long as lo does not end on binary16's grid of
// 2^-24 (queries are lifted for that, and weights' scale follows the scores).  Both words go through the
// matrix cores into the same f32 sums.
//
// A product's depth may be taken in any order, if both operands take the same, and rows in any: scores are
// made with keys as rows and queries as columns, sums with the values' dimensions as rows and weights as
// columns, and the tokens are put on the scores' rows such that a lane's scores are the weights that it
// gives to the sums.  So scores turn into weights without leaving their lane.
#pragma once

#include "cache.h"
#include "device.h"

namespace q8 {

using half2 = _Float16 __attribute__((ext_vector_type(2)));
using half8 = _Float16 __attribute__((ext_vector_type(8)));
using f32x4 = float __attribute__((ext_vector_type(4)));
using f32x16 = float __attribute__((ext_vector_type(16)));
using u32x2 = uint32_t __attribute__((ext_vector_type(2)));
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kNoMax = -3.0e38f;   // the scale of no scores: weights of masked tokens are then 0, too
// Weights are exp2(z - m + 11). m, a whole number (so that rescaling is exact), follows the scores of the tiles that a wave
// takes one after the other: sums are rescaled only where a row's largest score of a tile is over m + 4.75 or under m - 12, and
// m becomes that score, rounded down. So a weight never passes 2^15.75 (binary16 ends at 2^16), the largest of a row and
// tile is 2^-1 or more, and that of the row's largest score 2^11: a weight's words, which end on binary16's grid of 2^-24,
// are off by 2^-22 of it or by 2^-24 of the largest beside it in its tile. Where one token has nearly all of the weight,
// m comes down again for the tiles after it; the tokens of its own tile keep 2^-36 of it. (The last rows of a prompt of
// 4096 tokens whose first has a value of zero and scores 14 nats above the others, 128 dimensions: off by 8e-7 in the
// 2-norm, by 3e-6 where m only goes up; 16 nats above, 5e-6 and 2e-5.)
constexpr float kWeightShift = 11.0f, kMaxSlack = 4.75f, kMinSlack = 12.0f;
// What a lane's sum of weights may reach when m comes down, 2^90 (so m is at most some 2^79 below a row's largest): with
// four lanes, values of 2^16, 12 waves and 2^12 parts sums stay below 2^125.
constexpr float kMaxSum = 90.0f;

__device__ __forceinline__ half2 as_half2(uint32_t v) { return __builtin_bit_cast(half2, v); }
__device__ __forceinline__ half2 splat(_Float16 v) { return half2{v, v}; }

// (x & mask) | bits as one instruction: the masks stay in a vector and a scalar register, where the
// compiler would spend an instruction on each.
__device__ __forceinline__ half2 and_or(uint32_t x, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(x), "v"(mask), "s"(bits));
    return as_half2(r);
}

// How an operand's values follow from codes and a word: v = code' * d + c, exactly, where code' is
// the code under the exponent of 16 (4 bits: 16 + n) or 1024 (8 bits: 1024 + n + 128).  d is the
// scale times kDown: with the scale itself c would pass binary16's range (31 * 4352, 1152 * 512),
// and the scales' lowest bits (2^-19, 2^-17) leave room below.  c = -(16 + z) d has 5 + 6 bits,
// c = -1152 d 4 + 4, so that both are exact and the sum's exact value, a multiple of d, is, too.
template <int BITS>
struct Scales {
    half2 d, c;

    static constexpr float kDown = BITS == 4 ? 0.25f : 0.0625f;
    static constexpr float kUp = 1.0f / kDown;

    // of two words
    __device__ __forceinline__ void set(uint32_t words) {
        if (BITS == 4) {
            d = as_half2(words & 0x7fe07fe0u) * splat(static_cast<_Float16>(kDown));
            c = and_or(words << 6, 0x03c003c0u, 0x4c004c00u) * -d;
        } else {
            d = as_half2(words) * splat(static_cast<_Float16>(kDown));
            c = d * splat(static_cast<_Float16>(-1152.0f));
        }
    }
};

__device__ __forceinline__ half8 join(half2 a, half2 b, half2 c, half2 d) {
    return half8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// Eight codes: a dword of 4 bits, in pairs (0, 4), (1, 5), (2, 6), (3, 7); s[p] the scales of pair p.
__device__ __forceinline__ half8 values_of(uint32_t x, const Scales<4> &s0, const Scales<4> &s1, const Scales<4> &s2,
                                           const Scales<4> &s3) {
    constexpr uint32_t m = 0x03c003c0u, e = 0x4c004c00u;
    const half2 h0 = and_or(x << 6, m, e), h1 = and_or(x << 2, m, e), h2 = and_or(x >> 2, m, e), h3 = and_or(x >> 6, m, e);
    return join(__builtin_elementwise_fma(h0, s0.d, s0.c), __builtin_elementwise_fma(h1, s1.d, s1.c),
                __builtin_elementwise_fma(h2, s2.d, s2.c), __builtin_elementwise_fma(h3, s3.d, s3.c));
}

// Eight codes: two dwords of 8 bits, in the bytes' order.
__device__ __forceinline__ half8 values_of(uint32_t x, uint32_t y, const Scales<8> &s0, const Scales<8> &s1,
                                           const Scales<8> &s2, const Scales<8> &s3) {
    constexpr uint32_t e = 0x64646464u;
    const half2 h0 = as_half2(__builtin_amdgcn_perm(e, x, 0x04010400u)), h1 = as_half2(__builtin_amdgcn_perm(e, x, 0x04030402u)),
                h2 = as_half2(__builtin_amdgcn_perm(e, y, 0x04010400u)), h3 = as_half2(__builtin_amdgcn_perm(e, y, 0x04030402u));
    return join(__builtin_elementwise_fma(h0, s0.d, s0.c), __builtin_elementwise_fma(h1, s1.d, s1.c),
                __builtin_elementwise_fma(h2, s2.d, s2.c), __builtin_elementwise_fma(h3, s3.d, s3.c));
}

__device__ __forceinline__ f32x4 mfma(half8 a, half8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma(half8 a, half8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// Two f32 as two binary16 words each.  (The empty asms make the pair one value, which else is converted half by
// half once more for the difference, and hide the factor: a mixed multiply-add takes the words as they are.)
__device__ __forceinline__ void two_words(float x, float y, half2 &hi, half2 &lo) {
    float minus = -1.0f;
    asm("" : "+s"(minus));
    hi = half2{static_cast<_Float16>(x), static_cast<_Float16>(y)};
    asm("" : "+v"(hi));
    lo = half2{static_cast<_Float16>(__builtin_fmaf(static_cast<float>(hi.x), minus, x)),
               static_cast<_Float16>(__builtin_fmaf(static_cast<float>(hi.y), minus, y))};
}
__device__ __forceinline__ void two_words(const float (&x)[8], half8 &hi, half8 &lo) {
    half2 h[4], l[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) two_words(x[2 * p], x[2 * p + 1], h[p], l[p]);
    hi = join(h[0], h[1], h[2], h[3]);
    lo = join(l[0], l[1], l[2], l[3]);
}

// A lane's value and its partner's, 32 or 16 lanes away (a swap of a register with its copy leaves the one in the
// first and the other in the second).
__device__ __forceinline__ float2 lane_pair32(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    const uint32_t x = r[0], y = r[1];
    return make_float2(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y));
}
__device__ __forceinline__ float2 lane_pair16(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    const uint32_t x = r[0], y = r[1];
    return make_float2(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y));
}
__device__ __forceinline__ float exp2_of(float v) { return __builtin_amdgcn_exp2f(v); }

// A power of two that brings values of up to `most` into [2^14, 2^15) (small ones below), as its f32
// exponent field.  (Elements under 2^-17 of that have fewer than 22 bits: their second words are off by 2^-39 of it.)
__device__ __forceinline__ uint32_t lift_of(float most) {
    const int e = static_cast<int>(__builtin_bit_cast(uint32_t, most) >> 23);  // biased
    return static_cast<uint32_t>(min(141 + 127 - e, 253)) << 23;
}

// A query row as B operands of the scores' products, eight dimensions from dims(step) on for a lane and step.
template <int STEPS>
struct QueryRow {
    float x[STEPS][8];

    // (null: zeros)
    template <typename Dims>
    __device__ __forceinline__ void load(const float *row, Dims dims) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
            if (row) {
                const float4 *p = reinterpret_cast<const float4 *>(row + dims(s));
                a = p[0], b = p[1];
            }
            x[s][0] = a.x, x[s][1] = a.y, x[s][2] = a.z, x[s][3] = a.w, x[s][4] = b.x, x[s][5] = b.y, x[s][6] = b.z, x[s][7] = b.w;
        }
    }
};

// The row times scale * log2(e), lifted, as operands: out(step, hi, lo).  column_max is the largest over a
// column's lanes.  Returns what a score is multiplied by: a power of two.
template <int BITS, int STEPS, typename Max, typename Fn>
__device__ __forceinline__ float query_words(const QueryRow<STEPS> &row, float scale, Max column_max, Fn out) {
    float x[STEPS][8];
    float most = 0.0f;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // the order of values_of: pairs (0, 4), (1, 5), .. of 4 bits
            x[s][e] = row.x[s][BITS == 4 ? (e >> 1) + 4 * (e & 1) : e] * (scale * kLog2e);
            most = fmaxf(most, fabsf(x[s][e]));
        }
    }
    const uint32_t lift = lift_of(column_max(most));
    const float f = __builtin_bit_cast(float, lift);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[s][e] *= f;
        half8 hi, lo;
        two_words(x[s], hi, lo);
        out(s, hi, lo);
    }
    return __builtin_bit_cast(float, (254u << 23) - lift) * Scales<BITS>::kUp;
}

// Tiles that sequence s's rows see, [first, first + n).  A sequence without any keeps one, which
// has no token, so that its rows are written; one without rows has none.
struct Span {
    int first, n;
};

__device__ __forceinline__ Span span_of(const AttentionArgs &a, const Rows &r) {
    if (r.n == 0) return {0, 0};
    const int begin = a.window ? max(r.at - a.window + 1, 0) : 0;
    const int end = min(r.at + r.n, r.end);
    const int first = begin / kTileTokens;
    return {first, max((end + kTileTokens - 1) / kTileTokens - first, 1)};
}

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t add_dpp(uint32_t v) {
    return v + static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ int64_t lane_of(int64_t v, int l) {
    return static_cast<int64_t>(static_cast<uint64_t>(__builtin_amdgcn_readlane(static_cast<int>(v >> 32), l)) << 32 |
                                static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), l)));
}
// Inclusive sum over the lanes.
template <int CTRL, int ROWS>
__device__ __forceinline__ int64_t add_dpp(int64_t v) {
    const int lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xf, false);
    const int hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(v >> 32), CTRL, ROWS, 0xf, false);
    return v + static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32 | static_cast<uint32_t>(lo));
}
template <typename T>
__device__ __forceinline__ T wave_scan(T v) {
    v = add_dpp<0x111, 0xf>(v);  // row_shr 1, 2, 4, 8
    v = add_dpp<0x112, 0xf>(v);
    v = add_dpp<0x114, 0xf>(v);
    v = add_dpp<0x118, 0xf>(v);
    v = add_dpp<0x142, 0xa>(v);  // row_bcast 15 into rows 1 and 3
    return add_dpp<0x143, 0xc>(v);  // row_bcast 31 into rows 2 and 3
}
__device__ __forceinline__ uint32_t lane_of(uint32_t v, int l) {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), l));
}

// Keeps the weights' scale near `most`, the lane's largest score of a tile, and the sums in step with it:
// rescale(factor) multiplies the others.  (A lane has a part of its row's scores: whether there is anything to do, which
// is seldom, its column's decide. That is a branch of its own because the sums' registers are moved about in the second.)
template <typename Max, typename Fn>
__device__ __forceinline__ void follow_max(float most, float &top, float &sum, Max column_max, Fn rescale) {
    constexpr float kMid = 0.5f * (kMaxSlack - kMinSlack), kHalf = 0.5f * (kMaxSlack + kMinSlack);
    float now = top;
    bool changes = false;
    if (__any(fabsf(most - top - kMid) > kHalf)) {
        const float tile = column_max(most);
        // (-inf: none of the tile's tokens is seen)
        const bool under = tile < top - kMinSlack && tile > kNoMax;
        if (__any(tile > top + kMaxSlack || under)) {
            now = fmaxf(floorf(tile), top);
            if (__any(under)) {
                const float room = floorf(kMaxSum - __builtin_amdgcn_logf(column_max(sum)));
                now = under ? fmaxf(floorf(tile), top - fminf(fmaxf(room, 0.0f), kMaxSum)) : now;
            }
            changes = true;
        }
    }
    if (changes) {
        const float keep = exp2_of(top - now);
        top = now;
        sum *= keep;
        rescale(keep);
    }
}

// Two scores to weights in two words, and to their sum.
__device__ __forceinline__ void weigh_pair(float s, float t, float to_score, float top, float &sum, half2 &hi, half2 &lo) {
    const float below = kWeightShift - top;
    const float x = exp2_of(__builtin_fmaf(s, to_score, below)), y = exp2_of(__builtin_fmaf(t, to_score, below));
    sum += x;
    sum += y;
    two_words(x, y, hi, lo);
}

// Row x of a sequence and kv head: which of the call's.
struct Where {
    int64_t row;
    int head;
};
__device__ __forceinline__ Where where(const AttentionArgs &a, const Rows &r, int kv_head, int x) {
    const int i = x / a.group;
    return {int64_t(r.first) + i, kv_head * a.group + x - i * a.group};
}

template <int D>
__device__ __forceinline__ void write_row(const AttentionArgs &a, const Where &at, int dim, f32x4 o, float total, float top) {
    const float f = total > 0 ? 1.0f / total : 0.0f;
    *reinterpret_cast<f32x4 *>(a.out + (at.row * a.heads + at.head) * D + dim) = o * f;
    if (dim == 0 && a.lse) {
        // (the total's exponent joins the scale's, which may be far from it, before they are rounded)
        const float e = static_cast<float>(__builtin_amdgcn_frexp_expf(total));
        const float lse = (top + (e - kWeightShift)) * kLn2 + logf(__builtin_amdgcn_frexp_mantf(total));
        a.lse[at.row * a.heads + at.head] = total > 0 ? lse : -INFINITY;
    }
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, static_cast<int>(bytes), 0x00020000);
}
// Loads of a tile: its base is uniform and a lane's place in it 32 bits, where pointers would take 64-bit
// additions in the lanes, and registers for them.
__device__ __forceinline__ uint32_t load1(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t more) {
    return __builtin_amdgcn_raw_buffer_load_b32(r, at, more, 0);
}
__device__ __forceinline__ u32x2 load2(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t more) {
    return __builtin_amdgcn_raw_buffer_load_b64(r, at, more, 0);
}
__device__ __forceinline__ u32x4 load4(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t more) {
    return __builtin_amdgcn_raw_buffer_load_b128(r, at, more, 0);
}

// Parts go to the workspace and come back past the XCDs' own caches (agent scope: sc1), 16 bytes at a
// time, which the language's atomics do not offer.
constexpr int kAgent = 16;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t parts_of(float *p, uint32_t floats) { return buffer_of(p, floats * 4); }
__device__ __forceinline__ void store_part(__amdgpu_buffer_rsrc_t r, uint32_t at, f32x4 v) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, at * 4, 0, kAgent);
}
__device__ __forceinline__ f32x4 load_part(__amdgpu_buffer_rsrc_t r, uint32_t at) {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at * 4, 0, kAgent));
}

// A softmax's sums so far, and more of them.
struct Sums {
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    float top = kNoMax, sum = 0.0f;

    __device__ __forceinline__ void add(f32x4 o2, float top2, float sum2) {
        const float now = fmaxf(top, top2);
        const float keep = exp2_of(top - now), more = exp2_of(top2 - now);
        top = now;
        sum = sum * keep + sum2 * more;
        o = o * keep + o2 * more;
    }
};

}  // namespace q8
