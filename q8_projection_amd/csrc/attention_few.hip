// attention_few.hip -- attention of few rows a sequence and kv head (decode steps, drafted tokens): at
// most 32 query rows share the keys and values of a kv head, which are read once.
//
// A kv head's tiles are divided into pieces of about equal size over the whole batch, as many pieces
// as keep the chip busy; a workgroup takes a piece (short sequences are one piece).  Its waves take the piece's
// tiles in turn, each with a running maximum and sum of its own, and meet in LDS at the end; a kv
// head of several pieces is joined by the last workgroup to finish one, in the pieces' order.
// Codes go from memory to registers, in the order of the matrix cores' operands, and become binary16
// values there.
#include <algorithm>

#include "attention.h"
#include "launch.h"

namespace q8 {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kPiecesPerCu = 3;
constexpr int kMinTiles = 16;  // tiles of a piece, at least (but for shorter sequences)

struct FewArgs {
    AttentionArgs a;
    int pieces;         // wanted
    uint32_t *arrived;  // [2 pieces], zero between calls
    float *parts;       // [2 pieces][slot]
    int slot;           // floats of a part: rows * (D + 2)
};

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
// Inclusive sum over the lanes.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
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

// Codes and words of a lane's keys, and of its values.
template <int BITS, int D>
struct Keys {
    static constexpr int kUnits = BITS == 4 ? (D + 127) / 128 : D / 64;  // loads of a token
    static constexpr int kIn = BITS == 4 ? (D == 64 ? 2 : 4) : 2;        // steps of a load
    u32x4 x[2][kUnits];                                                  // (4 bits, D 64: half of it)
    uint32_t w[kUnits];

    __device__ __forceinline__ void load(const uint8_t *tile, int g, int c) {
        using T = Tile<BITS, D>;
        const int t = (c >> 2) * 8 + (c & 3);  // token of half 0
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint8_t *p = tile + (t + 4 * i) * T::kRow;
                if (BITS == 4 && D == 64) {
                    const u32x2 v = *reinterpret_cast<const u32x2 *>(p + g * 8);
                    x[i][u] = u32x4{v.x, v.y, 0, 0};
                } else {
                    x[i][u] = *reinterpret_cast<const u32x4 *>(p + u * 64 + g * 16);
                }
            }
            const int block = BITS == 4 ? (D == 64 ? g >> 1 : 4 * u + g) : 2 * u + (g >> 1);
            w[u] = *reinterpret_cast<const uint32_t *>(tile + T::kKeyWords + (c * T::kBlocks + block) * 4);
        }
    }
};

template <int BITS, int D>
struct Values {
    using O = Out<BITS, D>;
    u32x4 x[O::kChunks], w[O::kBlocks];

    __device__ __forceinline__ void load(const uint8_t *tile, int g, int c) {
        using T = Tile<BITS, D>;
        const int u = O::unit(c);
#pragma unroll
        for (int m = 0; m < O::kChunks; ++m)
            x[m] = *reinterpret_cast<const u32x4 *>(tile + T::kValues + ((u * 4 + g) * 16 + O::chunk(c, m)) * 16);
#pragma unroll
        for (int b = 0; b < O::kBlocks; ++b)
            w[b] = *reinterpret_cast<const u32x4 *>(tile + T::kValueWords + ((u * O::kBlocks + b) * 4 + g) * 16);
    }
};

// Which tokens of a tile count: [lo, hi) are there (others' codes may be anything), and row n of the
// lane sees [begin, end).
struct Seen {
    bool masked;  // some token of the tile is not seen by some row, or is none
    int t0, lo, hi;
};

template <int BITS, int D, int NR>
struct Wave {
    using O = Out<BITS, D>;
    static constexpr int kSteps = D / 32;
    float to_score[NR];
    int begin[NR], end[NR];
    float top[NR], sum[NR];
    f32x4 acc[NR][O::kChunks][O::kIn];
    half8 p_hi[NR], p_lo[NR];

    __device__ __forceinline__ void scores(const Keys<BITS, D> &k, const half8 *q, int lane, f32x4 (&s)[NR][2]) {
        using K = Keys<BITS, D>;
#pragma unroll
        for (int n = 0; n < NR; ++n) s[n][0] = s[n][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < K::kUnits; ++u) {
            Scales<BITS> sc[2];
            sc[0].set(__builtin_amdgcn_perm(k.w[u], k.w[u], 0x01000100u));
            sc[1].set(__builtin_amdgcn_perm(k.w[u], k.w[u], 0x03020302u));
#pragma unroll
            for (int e = 0; e < K::kIn; ++e) {
                half8 v[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if constexpr (BITS == 4) v[i] = values_of(k.x[i][u][e], sc[i], sc[i], sc[i], sc[i]);
                    else v[i] = values_of(k.x[i][u][2 * e], k.x[i][u][2 * e + 1], sc[i], sc[i], sc[i], sc[i]);
                }
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    const half8 *at = q + (n * kSteps + u * K::kIn + e) * 128 + lane;
                    const half8 hi = at[0], lo = at[64];
#pragma unroll
                    for (int i = 0; i < 2; ++i) s[n][i] = mfma(v[i], hi, s[n][i]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) s[n][i] = mfma(v[i], lo, s[n][i]);
                }
            }
        }
    }

    // Scores to weights, with the running maximum and sum.
    __device__ __forceinline__ void weights(f32x4 (&s)[NR][2], const Seen &seen, int g) {
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            float z[8];  // pairs (token p, token p + 4) of the lane's eight
#pragma unroll
            for (int p = 0; p < 4; ++p) z[2 * p] = s[n][0][p], z[2 * p + 1] = s[n][1][p];
            if (seen.masked) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int t = seen.t0 + 8 * g + (e >> 1) + 4 * (e & 1);
                    z[e] = t >= max(begin[n], seen.lo) && t < min(end[n], seen.hi) ? z[e] : -INFINITY;
                }
            }
            float most = z[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) most = fmaxf(most, z[e]);
            most = column_max(most) * to_score[n];
            if (__any(most > top[n])) {
                const float now = fmaxf(most, top[n]);
                const float keep = exp2_of(top[n] - now);
                top[n] = now;
                sum[n] *= keep;
#pragma unroll
                for (int m = 0; m < O::kChunks; ++m)
#pragma unroll
                    for (int w = 0; w < O::kIn; ++w) acc[n][m][w] *= keep;
            }
            const float below = kWeightShift - top[n];
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                w[e] = exp2_of(__builtin_fmaf(z[e], to_score[n], below));
                sum[n] += w[e];
            }
            two_words(w, p_hi[n], p_lo[n]);
        }
    }

    __device__ __forceinline__ void add_values(const Values<BITS, D> &v, const Seen &seen, int g) {
        Scales<BITS> sc[O::kBlocks][4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            uint32_t there = 0xffffffffu;
            if (seen.masked) {
                const int t = seen.t0 + 8 * g + p;
                there = (t >= seen.lo && t < seen.hi ? 0xffffu : 0u) | (t + 4 >= seen.lo && t + 4 < seen.hi ? 0xffff0000u : 0u);
            }
#pragma unroll
            for (int b = 0; b < O::kBlocks; ++b) sc[b][p].set(v.w[b][p] & there);
        }
#pragma unroll
        for (int m = 0; m < O::kChunks; ++m) {
#pragma unroll
            for (int w = 0; w < O::kIn; ++w) {
                half8 x;
                if constexpr (BITS == 4) x = values_of(v.x[m][w], sc[w / 2][0], sc[w / 2][1], sc[w / 2][2], sc[w / 2][3]);
                else x = values_of(v.x[m][2 * w], v.x[m][2 * w + 1], sc[0][0], sc[0][1], sc[0][2], sc[0][3]);
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    acc[n][m][w] = mfma(x, p_hi[n], acc[n][m][w]);
                    acc[n][m][w] = mfma(x, p_lo[n], acc[n][m][w]);
                }
            }
        }
    }
};

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
    if (dim == 0 && a.lse)
        a.lse[at.row * a.heads + at.head] = total > 0 ? (top - kWeightShift) * kLn2 + logf(total) : -INFINITY;
}

__device__ __forceinline__ void store_agent(float *p, float x, float y) {
    const uint64_t v = (uint64_t(__builtin_bit_cast(uint32_t, y)) << 32) | __builtin_bit_cast(uint32_t, x);
    __hip_atomic_store(reinterpret_cast<uint64_t *>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 load_agent(const float *p) {
    const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t *>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return make_float2(__builtin_bit_cast(float, static_cast<uint32_t>(v)), __builtin_bit_cast(float, static_cast<uint32_t>(v >> 32)));
}

// A piece: tiles [from, to) of the span of a sequence, for one kv head; piece `index` of `n` of it, whose
// parts are first, first + 1, ..
struct Piece {
    int s, head, index, n;
    int64_t first;
};

// Finds piece after piece, in ascending order.
struct Pieces {
    int target;               // tiles of a piece at most
    int s0 = 0;               // sequences s0 .. s0 + 63 are the lanes'
    int64_t pieces = 0, parts = 0;  // before them
    uint32_t count, scan, scan_parts;

    __device__ __forceinline__ void look(const AttentionArgs &a, int lane) {
        const int s = s0 + lane;
        const int n = s < a.c.sequences ? span_of(a, sequence_rows(a.c, s)).n : 0;
        set(n);
    }
    __device__ __forceinline__ void set(int n) {
        count = static_cast<uint32_t>((n + target - 1) / target);
        scan = wave_scan(count);
        scan_parts = wave_scan(count > 1 ? count : 0u);
    }
    // Piece p, or false if there are fewer.
    __device__ __forceinline__ bool find(const AttentionArgs &a, int64_t p, int lane, Piece &out) {
        for (;;) {
            const uint64_t above = __ballot(pieces + int64_t(scan) * a.c.kv_heads > p);
            if (above) {
                const int l = __builtin_ctzll(above);
                const int64_t before = pieces + (l ? int64_t(lane_of(scan, l - 1)) * a.c.kv_heads : 0);
                out.s = s0 + l;
                out.n = static_cast<int>(lane_of(count, l));
                const int rest = static_cast<int>(p - before);
                out.head = rest / out.n;
                out.index = rest - out.head * out.n;
                out.first = parts + (l ? int64_t(lane_of(scan_parts, l - 1)) * a.c.kv_heads : 0) + out.head * out.n;
                return true;
            }
            if (s0 + 64 >= a.c.sequences) return false;
            pieces += int64_t(lane_of(scan, 63)) * a.c.kv_heads;
            parts += int64_t(lane_of(scan_parts, 63)) * a.c.kv_heads;
            s0 += 64;
            look(a, lane);
        }
    }
};

template <int BITS, int D, int NR>
__global__ __launch_bounds__(kThreads, NR == 1 && D <= 128 ? 3 : 2) void few_kernel(FewArgs f) {
    using O = Out<BITS, D>;
    constexpr int kRows = 16 * NR;
    constexpr int kPad = D + 4;
    constexpr int kQuery = NR * (D / 32) * 2 * 64 * 16;       // bytes of the queries' words
    constexpr int kMeet = kWaves / 2 * kRows * kPad * 4;      // of the waves' sums
    __shared__ __align__(16) uint8_t shared[kQuery > kMeet ? kQuery : kMeet];
    __shared__ float tops[kWaves][kRows], sums[kWaves][kRows], to_scores[kRows];
    __shared__ uint32_t last;
    half8 *query = reinterpret_cast<half8 *>(shared);
    float *meet = reinterpret_cast<float *>(shared);
    const AttentionArgs &a = f.a;
    const CacheArgs &c = a.c;
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    // How many tiles there are, and so how many make a piece.
    int64_t total = 0;
    int tiles = 0;
    for (int s0 = 0; s0 < c.sequences; s0 += 64) {
        const int s = s0 + lane;
        tiles = s < c.sequences ? span_of(a, sequence_rows(c, s)).n : 0;
        total += lane_of(wave_scan(tiles), 63);
    }
    Pieces pieces;
    // (no sequence has more than 2^25 tiles)
    pieces.target = static_cast<int>(min(max((total * c.kv_heads + f.pieces - 1) / f.pieces, int64_t(kMinTiles)), int64_t(1) << 26));
    if (c.sequences <= 64) pieces.set(tiles);
    else pieces.look(a, lane);

    Piece piece;
    for (int64_t p = blockIdx.x; pieces.find(a, p, lane, piece); p += gridDim.x) {
        const Rows r = sequence_rows(c, piece.s);
        const Span span = span_of(a, r);
        const int from = static_cast<int>(int64_t(span.n) * piece.index / piece.n);
        const int to = static_cast<int>(int64_t(span.n) * (piece.index + 1) / piece.n);
        const int rows = r.n * a.group, head = piece.head;
        // tokens that any row sees, and those that every one does
        const int lo = a.window ? max(r.at - a.window + 1, 0) : 0, hi = min(r.at + r.n, r.end);
        const int all_lo = a.window ? max(r.at + r.n - a.window, 0) : 0, all_hi = min(r.at + 1, r.end);

        // This wave's tiles, 64 at a time: lane l looks up the page of the l-th.
        const int shift = c.page_shift - 5;
        int base = from + wid, mine = 0, page = -1;
        const auto look_up = [&] {
            mine = base < to ? min((to - base + kWaves - 1) / kWaves, 64) : 0;
            const int t = span.first + base + lane * kWaves;
            page = -1;
            if (lane < mine && t * kTileTokens < hi) page = c.table[piece.s * c.table_ld + (t >> shift)];
            if (page < 0 || page >= c.pages) page = -1;
        };
        const auto tile_of = [&](int l) -> const uint8_t * {
            const int t = span.first + base + l * kWaves;
            const int64_t pg = max(__builtin_amdgcn_readlane(page, l), 0);  // (none: the pool's first, not looked at)
            return c.data + (((pg * c.kv_heads + head) << shift) + (t & ((1 << shift) - 1))) * Tile<BITS, D>::kBytes;
        };
        Keys<BITS, D> keys;
        Values<BITS, D> values;
        look_up();
        if (mine) {
            const uint8_t *tile = tile_of(0);
            keys.load(tile, g, col);
            values.load(tile, g, col);
        }

        Wave<BITS, D, NR> w;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const int x = n * 16 + col;
            w.begin[n] = w.end[n] = 0;
            if (x < rows) {
                const int at = r.at + x / a.group;
                w.begin[n] = a.window ? max(at - a.window + 1, 0) : 0;
                w.end[n] = min(at + 1, r.end);
            }
            if (wid == n) {
                const float *row = nullptr;
                if (x < rows) {
                    const Where q = where(a, r, head, x);
                    row = a.q + q.row * a.q_ld + int64_t(q.head) * D;
                }
                const float t = load_query<BITS, D>(row, a.scale, lane, query + n * (D / 32) * 128);
                if (g == 0) to_scores[x] = t;
            }
            w.top[n] = kNoMax;
            w.sum[n] = 0.0f;
#pragma unroll
            for (int m = 0; m < O::kChunks; ++m)
#pragma unroll
                for (int j = 0; j < O::kIn; ++j) w.acc[n][m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NR; ++n) w.to_score[n] = to_scores[n * 16 + col];

        while (mine) {
            for (int l = 0; l < mine; ++l) {
                const int t0 = (span.first + base + l * kWaves) * kTileTokens;
                const Seen seen = {t0 < all_lo || t0 + kTileTokens > all_hi, t0, lo, hi};
                const bool there = __builtin_amdgcn_readlane(page, l) >= 0;
                const uint8_t *next = tile_of(min(l + 1, mine - 1));
                f32x4 s[NR][2];
                if (there) w.scores(keys, query, lane, s);
                keys.load(next, g, col);
                if (there) {
                    w.weights(s, seen, g);
                    w.add_values(values, seen, g);
                }
                values.load(next, g, col);
            }
            base += 64 * kWaves;
            look_up();
            if (mine) {
                const uint8_t *tile = tile_of(0);
                keys.load(tile, g, col);
                values.load(tile, g, col);
            }
        }

        // The waves' sums meet: half of the waves give theirs to the other half, until one has all.
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const float all = column_sum(w.sum[n]);
            if (g == 0) tops[wid][n * 16 + col] = w.top[n], sums[wid][n * 16 + col] = all;
        }
        __syncthreads();  // and the queries' words are free
        float top[NR], sum[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const int x = n * 16 + col;
            top[n] = tops[0][x];
#pragma unroll
            for (int v = 1; v < kWaves; ++v) top[n] = fmaxf(top[n], tops[v][x]);
            sum[n] = 0.0f;
#pragma unroll
            for (int v = 0; v < kWaves; ++v) sum[n] += sums[v][x] * exp2_of(tops[v][x] - top[n]);
            const float f = exp2_of(w.top[n] - top[n]) * Scales<BITS>::kUp;
#pragma unroll
            for (int m = 0; m < O::kChunks; ++m)
#pragma unroll
                for (int j = 0; j < O::kIn; ++j) w.acc[n][m][j] *= f;
        }
#pragma unroll
        for (int half = kWaves / 2; half >= 1; half /= 2) {
            if (wid >= half && wid < 2 * half) {
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    if (n * 16 + col < rows)
#pragma unroll
                        for (int m = 0; m < O::kChunks; ++m)
#pragma unroll
                            for (int j = 0; j < O::kIn; ++j)
                                *reinterpret_cast<f32x4 *>(meet + ((wid - half) * kRows + n * 16 + col) * kPad + ((m * O::kIn + j) * 4 + g) * 4) = w.acc[n][m][j];
            }
            __syncthreads();
            if (wid < half) {
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    if (n * 16 + col < rows)
#pragma unroll
                        for (int m = 0; m < O::kChunks; ++m)
#pragma unroll
                            for (int j = 0; j < O::kIn; ++j)
                                w.acc[n][m][j] += *reinterpret_cast<const f32x4 *>(meet + (wid * kRows + n * 16 + col) * kPad + ((m * O::kIn + j) * 4 + g) * 4);
            }
            __syncthreads();
        }
        // wave 0 has the piece's sums; they go out by whole rows
        if (wid == 0) {
#pragma unroll
            for (int n = 0; n < NR; ++n)
                if (n * 16 + col < rows)
#pragma unroll
                    for (int m = 0; m < O::kChunks; ++m)
#pragma unroll
                        for (int j = 0; j < O::kIn; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                meet[(n * 16 + col) * kPad + O::out_dim(4 * g + e, m, j)] = w.acc[n][m][j][e];
#pragma unroll
            for (int n = 0; n < NR; ++n)
                if (g == 0) tops[0][n * 16 + col] = top[n], sums[0][n * 16 + col] = sum[n];
        }
        __syncthreads();
        float *part = f.parts + (piece.first + piece.index) * f.slot;
        for (int e = threadIdx.x; e < rows * (D / 4); e += kThreads) {
            const int x = e / (D / 4), dim = e % (D / 4) * 4;
            const f32x4 o = *reinterpret_cast<const f32x4 *>(meet + x * kPad + dim);
            if (piece.n == 1) {
                write_row<D>(a, where(a, r, head, x), dim, o, sums[0][x], tops[0][x]);
            } else {
                float *dst = part + x * D + dim;
                store_agent(dst, o.x, o.y);
                store_agent(dst + 2, o.z, o.w);
                if (dim == 0) store_agent(part + rows * D + 2 * x, tops[0][x], sums[0][x]);
            }
        }
        if (piece.n > 1) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
            if (threadIdx.x == 0) {
                uint32_t *counter = f.arrived + piece.first;
                const uint32_t done = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                last = done == static_cast<uint32_t>(piece.n) - 1;
                if (last) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
            __syncthreads();
            if (last) {
                const float *first = f.parts + piece.first * f.slot;
                for (int e = threadIdx.x; e < rows * (D / 4); e += kThreads) {
                    const int x = e / (D / 4), dim = e % (D / 4) * 4;
                    float top_x = kNoMax, sum_x = 0.0f;
                    f32x4 o = {0.f, 0.f, 0.f, 0.f};
                    constexpr int kAhead = 8;
                    for (int i0 = 0; i0 < piece.n; i0 += kAhead) {
                        float2 st[kAhead], v0[kAhead], v1[kAhead];
#pragma unroll
                        for (int i = 0; i < kAhead; ++i) {
                            const float *q = first + int64_t(min(i0 + i, piece.n - 1)) * f.slot;
                            st[i] = load_agent(q + rows * D + 2 * x);
                            v0[i] = load_agent(q + x * D + dim);
                            v1[i] = load_agent(q + x * D + dim + 2);
                        }
#pragma unroll
                        for (int i = 0; i < kAhead; ++i) {
                            if (i0 + i >= piece.n) break;
                            const float now = fmaxf(top_x, st[i].x);
                            const float keep = exp2_of(top_x - now), add = exp2_of(st[i].x - now);
                            top_x = now;
                            sum_x = sum_x * keep + st[i].y * add;
                            o = o * keep + f32x4{v0[i].x, v0[i].y, v1[i].x, v1[i].y} * add;
                        }
                    }
                    write_row<D>(a, where(a, r, head, x), dim, o, sum_x, top_x);
                }
            }
        }
        __syncthreads();  // LDS is free again
    }
}

int few_pieces() { return device_info().cus * kPiecesPerCu; }

template <int BITS, int D>
hipError_t run(const FewArgs &f, hipStream_t stream) {
    // every piece a workgroup, unless there are very many
    const int64_t most = f.pieces + int64_t(f.a.c.sequences) * f.a.c.kv_heads;
    const dim3 grid(static_cast<uint32_t>(std::min<int64_t>(most, 32 * int64_t(f.pieces))));
    if (f.a.c.max_rows * f.a.group <= 16) few_kernel<BITS, D, 1><<<grid, kThreads, 0, stream>>>(f);
    else few_kernel<BITS, D, 2><<<grid, kThreads, 0, stream>>>(f);
    return hipGetLastError();
}

int64_t counter_bytes(int64_t pieces) { return (2 * pieces * 4 + 255) / 256 * 256; }

}  // namespace

int64_t few_workspace(int dim, const AttentionArgs &a) {
    const int64_t pieces = few_pieces(), rows = int64_t(a.c.max_rows) * a.group;
    return counter_bytes(pieces) + 2 * pieces * rows * (dim + 2) * 4;
}

hipError_t launch_few(int bits, int dim, const AttentionArgs &a, void *workspace, hipStream_t stream) {
    FewArgs f = {};
    f.a = a;
    f.pieces = few_pieces();
    f.arrived = static_cast<uint32_t *>(workspace);
    f.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + counter_bytes(f.pieces));
    f.slot = a.c.max_rows * a.group * (dim + 2);
    if (bits == 4) return dim == 64 ? run<4, 64>(f, stream) : dim == 128 ? run<4, 128>(f, stream) : run<4, 256>(f, stream);
    return dim == 64 ? run<8, 64>(f, stream) : dim == 128 ? run<8, 128>(f, stream) : run<8, 256>(f, stream);
}

}  // namespace q8
