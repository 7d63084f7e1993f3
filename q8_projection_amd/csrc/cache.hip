// cache.hip -- keys and values quantized as they are written into a paged cache,
// and read back (q8_cache.h has the formulas and the layout).
//
// One wave serves a 32-token tile of one sequence and 64 dimensions of one kv head.
// Both kernels move each f32 value and each code once and are bound by that and, for
// a few tokens, by one wave's chain of load, reduction and store.  Three prompts of up to 2048 tokens (31 MB
// of f32, 4.4 MB of codes) are appended in 11.9 us, of which some 6 are the quantization's instructions; eight whole sequences
// of up to 4099 tokens are read back, 165 MB in all, in 29 us while the last-level cache takes the output, and
// 51 from and to memory (3.2 TB/s; stores that pass the caches by: 45, but 61 instead of 44 for a call by
// itself, whose output is then not there for its reader).  One token is read in 3.2 us.  Another
// sequence of the call may have the same page and the tokens beside a sequence's own (chunks of one prompt that
// meet there), so a wave writes nothing but its tokens' codes: whole dwords or bytes, and, where a byte of two
// 4-bit codes may be shared, an exclusive or of what changes (one token 4.1 us and one each of 64 sequences 4.4; with dwords
// loaded, changed and stored, which loses the other's codes, 3.9 and 4.2; bytes of 8 bits 4.2, so 5.0).
//   keys  : lane = 8 tokens x 8 dimensions: a block's 32 values lie in 4 lanes, whose
//           smallest and largest meet in two DPP steps.
//   values: lane (g, b) = tokens 8 g .. 8 g + 7 of dimensions 4 b .. 4 b + 3: the lane holds
//           all eight tokens of its dwords, and a block's values lie in 8 lanes.
#include <algorithm>
#include <type_traits>
#include <utility>

#include "cache.h"
#include "device.h"

namespace q8 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// The format's constants: the scale keeps 23 - kDrop mantissa bits.
template <int BITS>
struct Format {
    static constexpr int kDrop = BITS == 4 ? 18 : 20;
    static constexpr float kSteps = BITS == 4 ? 15.0f : 127.0f;
    static constexpr float kTop = BITS == 4 ? 4352.0f : 512.0f;
    static constexpr float kLowest = BITS == 4 ? 0x1p-19f : 0x1p-17f;  // the smallest scale
};

// high - low, rounded up where it rounds: a span just over kSteps d must not pass for kSteps d.
__device__ __forceinline__ float span_of(float low, float high) {
    const float s = high - low, t = s - high;
    const float rest = (high - (s - t)) - (low + t);  // the exact difference's other part
    return rest > 0.0f ? __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, s) + 1u) : s;
}

// The smallest scale d of the format with kSteps d >= span.  span / kSteps is off by less
// than half a step of f32, and no quotient of an f32 by 15 or 127 rounds to a scale of at most
// 6 bits without being that scale (it would lie nearer to it than the products' common grid
// allows), so rounding the quotient up on the scales' grid is exact.
template <int BITS>
__device__ __forceinline__ float scale_of(float span) {
    using F = Format<BITS>;
    // (a quotient that rounds to 0 is one of a span over 0)
    const float t = fminf(fmaxf(span / F::kSteps, fminf(span, 0x1p-149f)), F::kTop);
    constexpr uint32_t step = (1u << F::kDrop) - 1;
    const float up = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, t) + step) & ~step);
    const float low = ceilf(t * (1.0f / F::kLowest)) * F::kLowest;  // binary16's subnormal grid
    return t < 0x1p-14f ? low : up;
}

// x / d, with r = 1 / d correctly rounded.  The first correction of x * r, which is up to
// one and a half steps off, leaves one of the two neighbours of x / d, the second the correctly
// rounded quotient (Markstein's theorem), and that is a half-integer only if the exact one is (x
// has 24 bits, d six).  One correction alone rounds some quotients next to a half-integer wrongly.
__device__ __forceinline__ float quotient(float x, float d, float r) {
    float q = x * r;
    q = __builtin_fmaf(__builtin_fmaf(-q, d, x), r, q);
    return __builtin_fmaf(__builtin_fmaf(-q, d, x), r, q);
}

// Smallest and largest over each 8 lanes.
__device__ __forceinline__ float eight_min(float v) {
    v = fminf(v, dpp_f32<0xb1>(v));          // quad_perm [1,0,3,2]
    v = fminf(v, dpp_f32<0x4e>(v));          // quad_perm [2,3,0,1]
    return fminf(v, dpp_f32<0x141>(v));      // row_half_mirror
}
__device__ __forceinline__ float eight_max(float v) {
    v = fmaxf(v, dpp_f32<0xb1>(v));
    v = fmaxf(v, dpp_f32<0x4e>(v));
    return fmaxf(v, dpp_f32<0x141>(v));
}

// Where in a tile the codes are of the group g's tokens and dimensions 64 part + 4 b (.. + 3, each 16 bytes on).
template <int BITS, int D>
__device__ __forceinline__ uint32_t value_place(int part, int g, int b) {
    const int w = b / 4, c = b % 4 * 4;  // dimension 16 w + c of the part
    if (BITS == 4) return Tile<BITS, D>::kValues + ((part * 4 + g) * 16 + c) * 16 + w * 4;
    return Tile<BITS, D>::kValues + (((part * 2 + w / 2) * 4 + g) * 16 + c) * 16 + w % 2 * 8;
}

__device__ __forceinline__ uint32_t half_bits(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
}

template <int CTRL>
__device__ __forceinline__ int dpp_i32(int v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, false);
}
// The value of each eight lanes' lane N (row_newbcast of it to the row's first eight, of lane N + 8 to the others).
template <int N>
__device__ __forceinline__ int eight_lane(int v) {
    const int low = __builtin_amdgcn_update_dpp(0, v, 0x150 + N, 0xf, 0x3, false);
    return __builtin_amdgcn_update_dpp(low, v, 0x158 + N, 0xf, 0xc, false);
}
template <int N>
__device__ __forceinline__ float eight_lane(float v) {
    return __builtin_bit_cast(float, eight_lane<N>(__builtin_bit_cast(int, v)));
}

// Whole numbers near rint(x / d) come as the bits of kMagic + x / d, rounded to the nearest there (ties to the
// even, as kMagic is): kMagicBits + n, in order for all x, so that they are clamped as integers.
constexpr float kMagic = 0x1.8p23f;
constexpr int kMagicBits = 0x4b400000;

// A block's scale, its reciprocal, and where codes begin: code 0 (4 bits) or 1 (8 bits) as x / d's bits.
template <int BITS>
struct Block {
    float d, r;
    int least;

    // low, high: the block's smallest value or 0, its largest or 0
    __device__ __forceinline__ void set(float low, float high) {
        d = scale_of<BITS>(BITS == 4 ? span_of(low, high) : fmaxf(high, -low));
        r = d > 0 ? 1.0f / d : 0.0f;
        least = BITS == 4 ? max(__builtin_bit_cast(int, kMagic - quotient(-low, d, r)), kMagicBits - 15) : kMagicBits - 127;
    }
    __device__ __forceinline__ uint32_t word() const {
        return half_bits(d) | (BITS == 4 ? static_cast<uint32_t>(kMagicBits - least) : 0u);
    }
    __device__ __forceinline__ uint32_t code(float x) const {
        const int n = __builtin_bit_cast(int, quotient(x, d, r) + kMagic);
        return static_cast<uint32_t>(min(max(n, least), least + (BITS == 4 ? 15 : 254)) - least + (BITS == 4 ? 0 : 1));
    }
    // another lane's
    template <int CTRL>
    __device__ __forceinline__ Block of() const {
        Block b;
        b.d = dpp_f32<CTRL>(d), b.r = dpp_f32<CTRL>(r);
        b.least = BITS == 4 ? dpp_i32<CTRL>(least) : least;
        return b;
    }
    template <int N>
    __device__ __forceinline__ Block of_eight() const {
        Block b;
        b.d = eight_lane<N>(d), b.r = eight_lane<N>(r);
        b.least = BITS == 4 ? eight_lane<N>(least) : least;
        return b;
    }
};

template <typename Fn, int... I>
__device__ __forceinline__ void each_of(Fn fn, std::integer_sequence<int, I...>) {
    (fn(std::integral_constant<int, I>{}), ...);
}
// fn(0), .. fn(N - 1) with constants.
template <int N, typename Fn>
__device__ __forceinline__ void each(Fn fn) {
    each_of(fn, std::make_integer_sequence<int, N>{});
}

// What a wave serves: a tile of a sequence, 64 dimensions of a kv head.
struct Work {
    int s, tile, head, part;
};

template <int D>
__device__ __forceinline__ Work work_of(const CacheArgs &c, uint32_t tiles, uint32_t wave) {
    constexpr int kParts = D / 64;
    const uint32_t per = c.kv_heads * kParts, rest = wave / per, u = wave - rest * per, s = rest / tiles;
    return {static_cast<int>(s), static_cast<int>(rest - s * tiles), static_cast<int>(u / kParts), static_cast<int>(u % kParts)};
}

// Tiles that the rows of one sequence can lie in: `rows` tokens anywhere.
inline int64_t tiles_of(int rows) { return (int64_t(rows) + kTileTokens - 2) / kTileTokens + 1; }

template <int BITS, int D>
__device__ __forceinline__ void append(const AppendArgs &a, const Work &w) {
    using T = Tile<BITS, D>;
    const Rows rows = sequence_rows(a.c, w.s);
    const int t = max(rows.at, 0) / kTileTokens + w.tile;  // tile of the sequence
    const int t0 = t * kTileTokens;
    // tokens [lo, hi) of the tile are written
    const int lo = max(rows.at - t0, 0), hi = min(min(rows.at + rows.n, rows.end) - t0, kTileTokens);
    if (lo >= hi) return;
    const int lane = threadIdx.x & 63;
    const int row0 = rows.first + (t0 - rows.at);  // row of the tile's token 0
    const int dim0 = w.part * 64;
    const int64_t column = int64_t(w.head) * D + dim0;

    // Loads first.  A token that is not written loads the nearest one that is.
    const int sub = lane >> 3, j = lane & 7;
    float kx[4][8];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int tok = min(max(p * 8 + sub, lo), hi - 1);
        const float *src = a.k + (row0 + tok) * a.k_ld + column + j * 8;
        const float4 x = *reinterpret_cast<const float4 *>(src), y = *reinterpret_cast<const float4 *>(src + 4);
        kx[p][0] = x.x, kx[p][1] = x.y, kx[p][2] = x.z, kx[p][3] = x.w;
        kx[p][4] = y.x, kx[p][5] = y.y, kx[p][6] = y.z, kx[p][7] = y.w;
    }
    const int g = lane >> 4, dims = lane & 15;
    float vx[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
        const int tok = min(max(g * 8 + n, lo), hi - 1);
        const float4 x = *reinterpret_cast<const float4 *>(a.v + (row0 + tok) * a.v_ld + column + 4 * dims);
        vx[n][0] = x.x, vx[n][1] = x.y, vx[n][2] = x.z, vx[n][3] = x.w;
    }
    uint8_t *tile = tile_at<BITS, D>(a.c, w.s, t, w.head);
    if (!tile) return;
    // 4 bits: the groups of eight tokens that the call has a part of alone (the first and the last can be such), and
    // what their dwords are, one a lane.  (The bits of this wave's tokens nobody else changes: what they were they are.)
    const int group[2] = {lo / 8, (hi - 1) / 8};
    const bool edge[2] = {lo % 8 != 0 || hi < group[0] * 8 + 8, group[1] != group[0] && hi % 8 != 0};
    const auto edge_at = [&](int i) {
        return reinterpret_cast<uint32_t *>(tile + T::kValues + (w.part * 4 + group[i]) * 256) + lane;
    };
    uint32_t was[2] = {0, 0};
    if constexpr (BITS == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (edge[i]) was[i] = *edge_at(i);
    }

    // Keys: a pass is 8 tokens.  A block's scale is made by one of its four lanes: lane p of them has pass p's.
    const auto pass_is = [&](int p) { return p * 8 < hi && p * 8 + 8 > lo; };
    {
        float low = 0.0f, high = 0.0f;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            float l = 0.0f, h = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) l = fminf(l, kx[p][e]), h = fmaxf(h, kx[p][e]);
            l = fminf(l, dpp_f32<0xb1>(l)), h = fmaxf(h, dpp_f32<0xb1>(h));
            l = fminf(l, dpp_f32<0x4e>(l)), h = fmaxf(h, dpp_f32<0x4e>(h));
            low = j % 4 == p ? l : low, high = j % 4 == p ? h : high;
        }
        Block<BITS> mine;
        mine.set(low, high);
        const int my_tok = j % 4 * 8 + sub;
        if (my_tok >= lo && my_tok < hi)
            reinterpret_cast<uint16_t *>(tile + T::kKeyWords)[key_word(my_tok, dim0 / 32 + j / 4, T::kBlocks)] =
                static_cast<uint16_t>(mine.word());
        each<4>([&](auto P) {
            constexpr int p = P;
            if (!pass_is(p)) return;
            const Block<BITS> b = mine.template of<0x55 * p>();  // quad_perm [p,p,p,p]
            uint32_t code[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 8; ++e) code[BITS == 4 ? 0 : e / 4] |= b.code(kx[p][e]) << (BITS == 4 ? 4 * e : 8 * (e % 4));
            const int tok = p * 8 + sub;
            if (tok < lo || tok >= hi) return;
            uint32_t *dst = reinterpret_cast<uint32_t *>(tile + tok * T::kRow + (dim0 + j * 8) * BITS / 8);
            dst[0] = code[0];
            if (BITS == 8) dst[1] = code[1];
        });
    }

    // Values.  A block's scale is made by one of its eight lanes: lane n of them has that of the group's token n.
    const auto token_is = [&](int n) { return hi - lo >= 8 || ((n - lo) & 7) < hi - lo; };  // a group's n, of any group
    constexpr int kWords = BITS / 4;  // dwords of a dimension's tokens
    uint32_t code[4][kWords] = {};
    float low = 0.0f, high = 0.0f;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
        if (!token_is(n)) continue;
        float l = 0.0f, h = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) l = fminf(l, vx[n][e]), h = fmaxf(h, vx[n][e]);
        l = eight_min(l), h = eight_max(h);
        low = dims % 8 == n ? l : low, high = dims % 8 == n ? h : high;
    }
    Block<BITS> mine;
    mine.set(low, high);
    const int my_tok = g * 8 + dims % 8;
    if (my_tok >= lo && my_tok < hi)
        reinterpret_cast<uint16_t *>(tile + T::kValueWords)[value_word(my_tok, dim0 / 32 + dims / 8)] = static_cast<uint16_t>(mine.word());
    each<8>([&](auto N) {
        constexpr int n = N;
        if (!token_is(n)) return;
        const Block<BITS> b = mine.template of_eight<n>();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t q = b.code(vx[n][e]);
            // 8 bits: byte 2 (n % 4) + n / 4
            if (BITS == 4) code[e][0] |= q << (4 * n);
            else code[e][(n & 3) >> 1] |= q << (16 * (n & 1) + 8 * (n >> 2));
        }
    });
    // the lane's tokens that are written
    const int first = max(lo - g * 8, 0), last = min(hi - g * 8, 8);
    uint8_t *dst = tile + value_place<BITS, D>(w.part, g, dims);
    if constexpr (BITS == 4) {
        if (first == 0 && last == 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) *reinterpret_cast<uint32_t *>(dst + 16 * e) = code[e][0];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (!edge[i]) continue;
            // dword 4 c + w of the group is the lane's: from lane 4 w + c / 4 of the group's, its number c % 4
            const int from = 4 * (16 * group[i] + 4 * (lane & 3) + (lane >> 4));
            uint32_t mine = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t c = static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(from, static_cast<int>(code[e][0])));
                mine = (lane >> 2 & 3) == e ? c : mine;
            }
            const int begin = max(lo - group[i] * 8, 0), end = min(hi - group[i] * 8, 8);
            const uint32_t owned = 0xffffffffu >> (32 - 4 * (end - begin)) << (4 * begin);
            __hip_atomic_fetch_xor(edge_at(i), (was[i] ^ mine) & owned, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            // tokens 2 i, 2 i + 1, 2 i + 4, 2 i + 5 in the dword's bytes
            if (first <= 2 * i && last >= 2 * i + 6) {
#pragma unroll
                for (int e = 0; e < 4; ++e) reinterpret_cast<uint32_t *>(dst + 16 * e)[i] = code[e][i];
                continue;
            }
            each<4>([&](auto B) {
                constexpr int byte = B;
                const int n = 2 * i + byte / 2 + 4 * (byte % 2);
                if (!token_is(n)) return;
                if (n >= first && n < last)
#pragma unroll
                    for (int e = 0; e < 4; ++e) dst[16 * e + 4 * i + byte] = static_cast<uint8_t>(code[e][i] >> (8 * byte));
            });
        }
    }
}

template <int BITS, int D>
__device__ __forceinline__ void read(const ReadArgs &a, const Work &w) {
    using T = Tile<BITS, D>;
    const Rows rows = sequence_rows(a.c, w.s);
    // the first row's token may lie before the sequence: its tile is then a negative one
    const int t = (rows.at >> 5) + w.tile, t0 = t * kTileTokens;
    const int lo = max(rows.at - t0, 0), hi = min(rows.at + rows.n - t0, kTileTokens);  // rows of the call
    if (lo >= hi) return;
    const int have = rows.end - t0;  // tokens from here on are none
    const uint8_t *tile = t < 0 || have <= 0 ? nullptr : tile_at<BITS, D>(a.c, w.s, t, w.head);
    const int lane = threadIdx.x & 63, dim0 = w.part * 64;
    const int64_t ld = int64_t(a.c.kv_heads) * D;
    const int64_t origin = (rows.first + (t0 - rows.at)) * ld + int64_t(w.head) * D + dim0;  // token 0's

    const int sub = lane >> 3, j = lane & 7;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int tok = p * 8 + sub;
        if (tok < lo || tok >= hi) continue;
        float x[8] = {};
        if (tile && tok < have) {
            const uint32_t *src = reinterpret_cast<const uint32_t *>(tile + tok * T::kRow + (dim0 + j * 8) * BITS / 8);
            const uint32_t code[2] = {src[0], BITS == 8 ? src[1] : 0};
            const uint32_t word = reinterpret_cast<const uint16_t *>(tile + T::kKeyWords)[key_word(tok, dim0 / 32 + j / 4, T::kBlocks)];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = value_of<BITS>(word, BITS == 4 ? code[0] >> (4 * e) & 15u : code[e / 4] >> (8 * (e % 4)) & 255u);
        }
        float *dst = a.k + origin + tok * ld + j * 8;
        *reinterpret_cast<float4 *>(dst) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(dst + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }

    const int g = lane >> 4, dims = lane & 15;
    constexpr int kWords = BITS / 4;
    uint32_t code[4][kWords] = {};
    uint4 words = make_uint4(0, 0, 0, 0);
    if (tile) {
        const uint8_t *src = tile + value_place<BITS, D>(w.part, g, dims);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < kWords; ++i) code[e][i] = reinterpret_cast<const uint32_t *>(src + 16 * e)[i];
        words = *reinterpret_cast<const uint4 *>(tile + T::kValueWords + ((dim0 / 32 + dims / 8) * 4 + g) * 16);
    }
    const uint32_t word[4] = {words.x, words.y, words.z, words.w};
#pragma unroll
    for (int n = 0; n < 8; ++n) {
        const int tok = g * 8 + n;
        if (tok < lo || tok >= hi) continue;
        // words lie in pairs of tokens n, n + 4
        const uint32_t m = word[n & 3] >> (16 * (n >> 2)) & 0xffffu;
        const bool there = tile && tok < have;
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t q = BITS == 4 ? code[e][0] >> (4 * n) & 15u : code[e][(n & 3) >> 1] >> (16 * (n & 1) + 8 * (n >> 2)) & 255u;
            x[e] = there ? value_of<BITS>(m, q) : 0.0f;
        }
        *reinterpret_cast<float4 *>(a.v + origin + tok * ld + 4 * dims) = make_float4(x[0], x[1], x[2], x[3]);
    }
}

// The waves' work in turn: more waves than that only where most find nothing to do.
constexpr int64_t kMaxBlocks = 1 << 20;

template <int BITS, int D>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a, uint32_t tiles, uint32_t waves) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (uint32_t i = blockIdx.x * kWaves + wave; i < waves; i += gridDim.x * kWaves) append<BITS, D>(a, work_of<D>(a.c, tiles, i));
}

template <int BITS, int D>
__global__ __launch_bounds__(kThreads) void read_kernel(ReadArgs a, uint32_t tiles, uint32_t waves) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (uint32_t i = blockIdx.x * kWaves + wave; i < waves; i += gridDim.x * kWaves) read<BITS, D>(a, work_of<D>(a.c, tiles, i));
}

template <typename Args, typename Kernel>
hipError_t launch(Kernel kernel, const Args &a, int parts, hipStream_t stream) {
    const int64_t tiles = tiles_of(a.c.max_rows);
    const int64_t waves = a.c.sequences * tiles * a.c.kv_heads * parts;  // below 2^31 by the limits of a call
    const int64_t blocks = std::min((waves + kWaves - 1) / kWaves, kMaxBlocks);
    kernel<<<dim3(static_cast<uint32_t>(blocks)), dim3(kThreads), 0, stream>>>(a, static_cast<uint32_t>(tiles), static_cast<uint32_t>(waves));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_append(int bits, int dim, const AppendArgs &a, hipStream_t stream) {
    if (bits == 4)
        return dim == 64    ? launch(append_kernel<4, 64>, a, 1, stream)
               : dim == 128 ? launch(append_kernel<4, 128>, a, 2, stream)
                            : launch(append_kernel<4, 256>, a, 4, stream);
    return dim == 64    ? launch(append_kernel<8, 64>, a, 1, stream)
           : dim == 128 ? launch(append_kernel<8, 128>, a, 2, stream)
                        : launch(append_kernel<8, 256>, a, 4, stream);
}

hipError_t launch_cache_read(int bits, int dim, const ReadArgs &a, hipStream_t stream) {
    if (bits == 4)
        return dim == 64    ? launch(read_kernel<4, 64>, a, 1, stream)
               : dim == 128 ? launch(read_kernel<4, 128>, a, 2, stream)
                            : launch(read_kernel<4, 256>, a, 4, stream);
    return dim == 64    ? launch(read_kernel<8, 64>, a, 1, stream)
           : dim == 128 ? launch(read_kernel<8, 128>, a, 2, stream)
                        : launch(read_kernel<8, 256>, a, 4, stream);
}

}  // namespace q8
