// attention_few.hip -- attention of few rows a sequence and kv head (decode steps, drafted tokens): at
// most 32 query rows share the keys and values of a kv head, which are read once.
//
// A kv head's tiles are divided into pieces of about equal size over the whole batch, as many pieces
// as keep the chip busy; a workgroup takes a piece (short sequences are one piece).  Its waves take the piece's
// tiles in turn, each with a running maximum and sum of its own, and meet in LDS at the end; a kv
// head of several pieces is joined by the last workgroup to finish one, in the pieces' order.
// Codes go from memory to registers, in the order of the matrix cores' operands, and become binary16
// values there.
//
// Measured, 4 bits, 32 heads of 8 kv heads and 128 dimensions: one sequence of 131071 tokens 39 us, 151 MB at 3.8 TB/s; a
// batch of 64 of up to 8192 tokens 76 us, 294 MB at 3.9 TB/s.  A tile takes a wave some 370 vector instructions (codes
// to values most of all, then weights) and 32 products: it is their issue that bounds long calls, and short ones the chain
// of some 8 us from the lengths to the table, the codes, the waves' meeting and the join.
//
// v_mfma_f32_16x16x32_f16, as its lanes hold it (lane = 16 g + c):
//   A: row c, depth 8 g + e (e = 0 .. 7);  B: column c, depth 8 g + e;  C: column c, rows 4 g + r
// Scores: row c of half i is token 8 (c / 4) + 4 i + c % 4 of a tile, so that lane (g, c) gets row c's
// scores of tokens 8 g + 4 i + r, i = 0, 1, and gives their weights to the sums.
#include <algorithm>

#include "attention.h"
#include "launch.h"

namespace q8 {
namespace {

constexpr int kAhead = 8;      // parts whose loads are in flight at once
// Tiles of a piece, at least (but for shorter sequences).  One sequence of 500 tokens takes 10.6 us, at 12 11.7; of 4000
// tokens 14.5, at 24 15.6, at 48 18.4.
constexpr int kMinTiles = 16;
constexpr int kPiecesPerSlot = 2;  // pieces for each workgroup that the chip holds (twice as many counters: kCountersPerCu)
static_assert(2 * 3 * kPiecesPerSlot <= kCountersPerCu);
// A workgroup takes a whole CU up to a kv head of some sequence for kBigItems CUs: fewer parts to join.  16 kv heads at 32000 tokens
// 24.9 us, with workgroups of four waves 33.7, 64 of them 66 and 77; at 2 for kBigItems, 128 of up to 4096 tokens 28.4 and 21.9.
constexpr int kBigItems = 4;

struct FewArgs {
    AttentionArgs a;
    int pieces;         // wanted
    uint32_t *arrived;  // [2 pieces], zero between calls
    float *parts;       // [2 pieces][slot]
    int slot;           // floats of a part: rows * (D + 4)
};

// The largest, and the sum, over the four lanes of a column.
__device__ __forceinline__ float column_max(float v) {
    const float2 a = lane_pair32(v), b = lane_pair16(fmaxf(a.x, a.y));
    return fmaxf(b.x, b.y);
}
__device__ __forceinline__ float column_sum(float v) {
    const float2 a = lane_pair32(v), b = lane_pair16(a.x + a.y);
    return b.x + b.y;
}

// The first dimension of the eight that step s of a score's product takes in lane group g; a lane's
// codes lie together, up to 16 bytes.
template <int BITS, int D>
__device__ __forceinline__ constexpr int key_dims(int s, int g) {
    if (BITS == 8) return 64 * (s / 2) + 16 * g + 8 * (s % 2);
    return D == 64 ? 16 * g + 8 * s : 128 * (s / 4) + 32 * g + 8 * (s % 4);
}

// The dimensions of the output's products.  A lane's value codes come as kChunks 16-byte chunks of
// the layout, kIn operands each.  Row c of operand (m, w) is dimension out_dim(c, m, w): with a
// lane's chunks side by side, its dimensions lie in 2 (4 bits) or 1 blocks, and it needs the words of those alone.
template <int BITS, int D>
struct Out {
    static constexpr int kChunks = BITS == 4 ? D / 64 : D / 32;
    static constexpr int kIn = BITS == 4 ? 4 : 2;
    static constexpr int kBlocks = BITS == 4 ? 2 : 1;
    static constexpr int kPer = 16 / kChunks;  // rows of one unit of the layout
    static constexpr int kUnit = BITS == 4 ? 64 : 32;  // dimensions of it

    static __device__ __forceinline__ int unit(int c) { return c / kPer; }
    static __device__ __forceinline__ int chunk(int c, int m) { return c % kPer * kChunks + m; }
    static __device__ __forceinline__ int out_dim(int c, int m, int w) { return unit(c) * kUnit + 16 * w + chunk(c, m); }

    // fn(first dimension, four values) for lane group g's part of a row's sums.
    template <typename Acc, typename Fn>
    static __device__ __forceinline__ void for_each_vec(Acc acc, int g, Fn fn) {
#pragma unroll
        for (int w = 0; w < kIn; ++w) {
            if constexpr (kChunks == 1) {
                fn(out_dim(4 * g, 0, w), acc(0, w));
            } else if constexpr (kChunks == 2) {
#pragma unroll
                for (int r = 0; r < 4; r += 2)
                    fn(out_dim(4 * g + r, 0, w), f32x4{acc(0, w)[r], acc(1, w)[r], acc(0, w)[r + 1], acc(1, w)[r + 1]});
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int m = 0; m < kChunks; m += 4)
                        fn(out_dim(4 * g + r, m, w), f32x4{acc(m, w)[r], acc(m + 1, w)[r], acc(m + 2, w)[r], acc(m + 3, w)[r]});
            }
        }
    }
};

// Scores of 32 tokens: lane (g, c) has row c's of tokens 8 g + 4 i + r in s[i][r].  Those that the row does
// not see (outside [begin, end), t0 the first token) become -inf.
__device__ __forceinline__ void mask_scores(f32x4 (&s)[2], int t0, int g, int begin, int end) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = t0 + 8 * g + 4 * i + r;
            s[i][r] = t >= begin && t < end ? s[i][r] : -INFINITY;
        }
}

__device__ __forceinline__ float largest(const f32x4 (&s)[2]) {
    float most = s[0][0];
#pragma unroll
    for (int e = 1; e < 8; ++e) most = fmaxf(most, s[e >> 2][e & 3]);
    return most;
}

// Codes and words of a lane's keys, and of its values.
template <int BITS, int D>
struct Keys {
    static constexpr int kUnits = BITS == 4 ? (D + 127) / 128 : D / 64;  // loads of a token
    static constexpr int kIn = BITS == 4 ? (D == 64 ? 2 : 4) : 2;        // steps of a load
    u32x4 x[2][kUnits];                                                  // (4 bits, D 64: half of it)
    uint32_t w[kUnits];

    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t tile, uint32_t g, uint32_t c) {
        using T = Tile<BITS, D>;
        const uint32_t t = (c >> 2) * 8 + (c & 3);  // token of half 0
        const uint32_t code = t * T::kRow + g * (BITS == 4 && D == 64 ? 8 : 16);
        const uint32_t word = T::kKeyWords + (c * T::kBlocks + (BITS == 4 && D > 64 ? g : g >> 1)) * 4;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t more = 4 * i * T::kRow + u * 64;
                if (BITS == 4 && D == 64) {
                    const u32x2 v = load2(tile, code, more);
                    x[i][u] = u32x4{v.x, v.y, 0, 0};
                } else {
                    x[i][u] = load4(tile, code, more);
                }
            }
            w[u] = load1(tile, word, u * (BITS == 4 ? 16 : 8));
        }
    }
};

template <int BITS, int D>
struct Values {
    using O = Out<BITS, D>;
    u32x4 x[O::kChunks], w[O::kBlocks];

    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t tile, uint32_t g, uint32_t c) {
        using T = Tile<BITS, D>;
        const uint32_t u = O::unit(c);
        const uint32_t code = T::kValues + ((u * 4 + g) * 16 + O::chunk(c, 0)) * 16;
        const uint32_t word = T::kValueWords + (u * O::kBlocks * 4 + g) * 16;
#pragma unroll
        for (int m = 0; m < O::kChunks; ++m) x[m] = load4(tile, code, m * 16);
#pragma unroll
        for (int b = 0; b < O::kBlocks; ++b) w[b] = load4(tile, word, b * 64);
    }
};

// Which tokens of a tile count: [lo, hi) are there, others' codes may be anything.
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

// A piece: tiles [from, to) of the span of a sequence, for one kv head; piece `index` of `n` of it, whose
// parts are first, first + 1, ..
struct Piece {
    int s, head, index, n;
    int64_t first;
    Rows rows;
    Span span;
};

// Finds piece after piece, in ascending order.
struct Pieces {
    int target, slack;        // tiles of a piece, and how many more are no second one
    int s0 = 0;               // sequences s0 .. s0 + 63 are the lanes'
    int64_t pieces = 0, parts = 0;  // before them
    Rows rows;
    Span span;
    uint32_t count, scan, scan_parts;

    __device__ __forceinline__ uint32_t look(const AttentionArgs &a, int lane) {
        const int s = s0 + lane;
        rows = Rows{0, 0, 0, 0};
        if (s < a.c.sequences) rows = sequence_rows(a.c, s);
        span = span_of(a, rows);
        return static_cast<uint32_t>(span.n);
    }
    __device__ __forceinline__ void divide() {
        count = span.n ? static_cast<uint32_t>(max((span.n - slack + target - 1) / target, 1)) : 0u;
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
                const auto at = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
                out.rows = Rows{at(rows.first), at(rows.n), at(rows.at), at(rows.end)};
                out.span = Span{at(span.first), at(span.n)};
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
            divide();
        }
    }
};

// Waves of a SIMD that the registers allow without a spill (a kernel with scratch memory starts 5 us
// later).
template <int BITS, int D, int NR>
constexpr int kWavesPerSimd = NR == 1 && (D == 64 || (D == 128 && BITS == 4)) ? 3 : 2;

template <int BITS, int D, int NR, int WAVES>
__global__ __launch_bounds__(64 * WAVES, (kWavesPerSimd<BITS, D, NR>)) void few_kernel(FewArgs f) {
    using O = Out<BITS, D>;
    constexpr int kThreads = 64 * WAVES;
    constexpr int kRows = 16 * NR;
    constexpr int kPad = D + 4;
    constexpr int kQuery = NR * (D / 32) * 2 * 64 * 16;  // bytes of the queries' words
    constexpr int kMeet = WAVES * 16 * kPad * 4;         // of the waves' sums, 16 rows at a time
    __shared__ __align__(16) uint8_t shared[kQuery > kMeet ? kQuery : kMeet];
    __shared__ float tops[WAVES][kRows], sums[WAVES][kRows], to_scores[kRows];
    __shared__ uint32_t last;
    half8 *query = reinterpret_cast<half8 *>(shared);
    float *meet = reinterpret_cast<float *>(shared);
    const AttentionArgs &a = f.a;
    const CacheArgs &c = a.c;
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    // How many tiles there are, and so how many make a piece.
    Pieces pieces;
    int64_t total = 0;
    for (; pieces.s0 < c.sequences; pieces.s0 += 64) total += lane_of(wave_scan(pieces.look(a, lane)), 63);
    // (no sequence has more than 2^25 tiles)
    // A large workgroup takes up to half more than a least piece in a turn more at most, and has no parts to join then: 517 tokens
    // (12 waves) 10.4 us with the slack, without it 11.8; 700 tokens (8 waves, up to 128 dimensions) 10.7 to 15.1, without
    // it 11.0 to 15.4. 256 dimensions pay more for the turn: 700 tokens 16.2 (4 bits) and 22.0 (8 bits) with it, 13.9 and 18.4
    // without it. Four waves take a turn more for every four tiles: drafted tokens of 16 sequences 23.8 with it and 22.0.
    pieces.slack = WAVES > 4 && D < 256 ? kMinTiles / 2 : 0;
    pieces.target = static_cast<int>(min(max((total * c.kv_heads + f.pieces - 1) / f.pieces, int64_t(kMinTiles)), int64_t(1) << 26));
    pieces.s0 = 0;
    if (c.sequences > 64) pieces.look(a, lane);
    pieces.divide();

    Piece piece;
    for (int64_t p = blockIdx.x; pieces.find(a, p, lane, piece); p += gridDim.x) {
        const Rows r = piece.rows;
        const Span span = piece.span;
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
            mine = base < to ? min((to - base + WAVES - 1) / WAVES, 64) : 0;
            const int t = span.first + base + lane * WAVES;
            page = -1;
            if (lane < mine && t * kTileTokens < hi) page = c.table[piece.s * c.table_ld + (t >> shift)];
            if (page < 0 || page >= c.pages) page = -1;
        };
        const auto tile_of = [&](int l) {
            const int t = span.first + base + l * WAVES;
            const int64_t pg = max(__builtin_amdgcn_readlane(page, l), 0);  // (none: the pool's first, not looked at)
            return buffer_of(c.data + (((pg * c.kv_heads + head) << shift) + (t & ((1 << shift) - 1))) * Tile<BITS, D>::kBytes,
                             Tile<BITS, D>::kBytes);
        };
        Keys<BITS, D> keys;
        Values<BITS, D> values;
        look_up();
        if (mine) {
            const __amdgpu_buffer_rsrc_t tile = tile_of(0);
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
                half8 *words = query + n * (D / 32) * 128 + lane;
                const auto dims = [&](int s) { return key_dims<BITS, D>(s, g); };
                QueryRow<D / 32> q_row;
                q_row.load(row, dims);
                const float t = query_words<BITS>(q_row, a.scale, column_max, [&](int s, half8 hi, half8 lo) {
                    words[2 * s * 64] = hi, words[(2 * s + 1) * 64] = lo;
                });
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
                const int t0 = (span.first + base + l * WAVES) * kTileTokens;
                const Seen seen = {t0 < all_lo || t0 + kTileTokens > all_hi, t0, lo, hi};
                const bool there = __builtin_amdgcn_readlane(page, l) >= 0;
                const __amdgpu_buffer_rsrc_t next = tile_of(min(l + 1, mine - 1));
                f32x4 z[NR][2];
                if (there) w.scores(keys, query, lane, z);
                keys.load(next, g, col);
                if (there) {
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        if (seen.masked) mask_scores(z[n], t0, g, max(w.begin[n], lo), min(w.end[n], hi));
                        follow_max(largest(z[n]) * w.to_score[n], w.top[n], w.sum[n], column_max, [&](float keep) {
#pragma unroll
                            for (int m = 0; m < O::kChunks; ++m)
#pragma unroll
                                for (int j = 0; j < O::kIn; ++j) w.acc[n][m][j] *= keep;
                        });
                        half2 p[4], q[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) weigh_pair(z[n][0][e], z[n][1][e], w.to_score[n], w.top[n], w.sum[n], p[e], q[e]);
                        w.p_hi[n] = join(p[0], p[1], p[2], p[3]);
                        w.p_lo[n] = join(q[0], q[1], q[2], q[3]);
                    }
                    w.add_values(values, seen, g);
                }
                values.load(next, g, col);
            }
            base += 64 * WAVES;
            look_up();
            if (mine) {
                const __amdgpu_buffer_rsrc_t tile = tile_of(0);
                keys.load(tile, g, col);
                values.load(tile, g, col);
            }
        }

        // The waves' sums meet, 16 rows at a time: all write theirs, every thread adds up some.
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const float all = column_sum(w.sum[n]);
            if (g == 0) tops[wid][n * 16 + col] = w.top[n], sums[wid][n * 16 + col] = all;
        }
        __syncthreads();  // and the queries' words are free
        // parts of a kv head: rows of D sums each, then rows of (maximum, sum)
        const int vecs = rows * (D / 4);  // 16-byte pieces of the rows
        const __amdgpu_buffer_rsrc_t parts = parts_of(f.parts + piece.first * f.slot, piece.n * f.slot);
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            if (n) __syncthreads();
            float top = tops[0][n * 16 + col];
#pragma unroll
            for (int v = 1; v < WAVES; ++v) top = fmaxf(top, tops[v][n * 16 + col]);
            const float scale = exp2_of(w.top[n] - top) * Scales<BITS>::kUp;
            if (n * 16 + col < rows) O::for_each_vec([&](int m, int j) { return w.acc[n][m][j]; }, g, [&](int dim, f32x4 v) {
                *reinterpret_cast<f32x4 *>(meet + (wid * 16 + col) * kPad + dim) = v * scale;
            });
            __syncthreads();
            for (int e = threadIdx.x; e < min(vecs - n * 4 * D, 4 * D); e += kThreads) {
                const int y = e / (D / 4), x = n * 16 + y, dim = e % (D / 4) * 4;
                f32x4 o = *reinterpret_cast<const f32x4 *>(meet + y * kPad + dim);
#pragma unroll
                for (int v = 1; v < WAVES; ++v) o += *reinterpret_cast<const f32x4 *>(meet + (v * 16 + y) * kPad + dim);
                if (piece.n > 1) store_part(parts, piece.index * f.slot + x * D + dim, o);
                if (piece.n == 1 || dim == 0) {
                    float top_x = tops[0][x], sum_x = 0.0f;
#pragma unroll
                    for (int v = 1; v < WAVES; ++v) top_x = fmaxf(top_x, tops[v][x]);
#pragma unroll
                    for (int v = 0; v < WAVES; ++v) sum_x += sums[v][x] * exp2_of(tops[v][x] - top_x);
                    if (piece.n == 1) write_row<D>(a, where(a, r, head, x), dim, o, sum_x, top_x);
                    else store_part(parts, piece.index * f.slot + (vecs + x) * 4, f32x4{top_x, sum_x, 0.f, 0.f});
                }
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
                // Few rows leave threads over: these divide the parts, slice after slice of them.
                const int slices = vecs < kThreads ? kThreads / vecs : 1;
                const int slice = vecs < kThreads ? threadIdx.x / vecs : 0;
                const int i0 = piece.n * slice / slices, i1 = piece.n * (slice + 1) / slices;
                f32x4 *there = reinterpret_cast<f32x4 *>(shared);
                for (int e0 = 0; e0 < vecs; e0 += kThreads) {
                    const int e = vecs < kThreads ? threadIdx.x - slice * vecs : e0 + threadIdx.x;
                    const bool live = slice < slices && e < vecs;
                    const int x = e / (D / 4), dim = e % (D / 4) * 4;
                    Sums all;
                    if (live) {
                        for (int i = i0; i < i1; i += kAhead) {
                            f32x4 o[kAhead], st[kAhead];
#pragma unroll
                            for (int j = 0; j < kAhead; ++j) {
                                // (past the last one: past the buffer, nothing is read)
                                const uint32_t at_part = static_cast<uint32_t>((i + j) * f.slot) | oob_bit(i + j < i1) >> 2;
                                st[j] = load_part(parts, at_part + (vecs + x) * 4);
                                o[j] = load_part(parts, at_part + 4 * e);
                            }
#pragma unroll
                            for (int j = 0; j < kAhead; ++j)
                                if (i + j < i1) all.add(o[j], st[j].x, st[j].y);
                        }
                    }
                    if (slices > 1) {
                        if (live && slice) {
                            there[2 * (threadIdx.x - vecs)] = all.o;
                            there[2 * (threadIdx.x - vecs) + 1] = f32x4{all.top, all.sum, 0.f, 0.f};
                        }
                        __syncthreads();
                        if (live && !slice)
                            for (int v = 1; v < slices; ++v) {
                                const f32x4 st = there[2 * (threadIdx.x + (v - 1) * vecs) + 1];
                                all.add(there[2 * (threadIdx.x + (v - 1) * vecs)], st.x, st.y);
                            }
                    }
                    if (live && !slice) write_row<D>(a, where(a, r, head, x), dim, all.o, all.sum, all.top);
                }
            }
        }
        __syncthreads();  // LDS is free again
    }
}

// Workgroups of 4 waves, as many as a CU holds, overlap one's start and end with another's tiles.  Where
// a kv head is divided over many workgroups anyway, one of all the waves that a CU holds has a third
// or half of the parts to join.
template <int BITS, int D, int NR>
hipError_t run(FewArgs f, hipStream_t stream) {
    constexpr int kPerCu = kWavesPerSimd<BITS, D, NR>;
    const int64_t items = int64_t(f.a.c.sequences) * f.a.c.kv_heads;
    const int cus = device_info().cus;
    if (items * kBigItems <= cus) {
        f.pieces = cus;
        few_kernel<BITS, D, NR, 4 * kPerCu><<<dim3(static_cast<uint32_t>(cus + items)), 256 * kPerCu, 0, stream>>>(f);
    } else {
        f.pieces = cus * kPiecesPerSlot * kPerCu;
        // every piece a workgroup, unless there are very many
        const int64_t most = std::min<int64_t>(f.pieces + items, 32 * int64_t(f.pieces));
        few_kernel<BITS, D, NR, 4><<<dim3(static_cast<uint32_t>(most)), 256, 0, stream>>>(f);
    }
    return hipGetLastError();
}

template <int BITS, int D>
hipError_t run_rows(const FewArgs &f, hipStream_t stream) {
    if constexpr (few_rows(D) > 16)
        if (f.a.c.max_rows * f.a.group > 16) return run<BITS, D, 2>(f, stream);
    return run<BITS, D, 1>(f, stream);
}

int64_t most_pieces() { return int64_t(device_info().cus) * 3 * kPiecesPerSlot; }

}  // namespace

int64_t few_workspace(int dim, const AttentionArgs &a) {
    return attention_counter_bytes() + 2 * most_pieces() * a.c.max_rows * a.group * (dim + 4) * 4;
}

hipError_t launch_few(int bits, int dim, const AttentionArgs &a, void *workspace, hipStream_t stream) {
    FewArgs f = {};
    f.a = a;
    f.arrived = static_cast<uint32_t *>(workspace);
    f.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + attention_counter_bytes());
    f.slot = a.c.max_rows * a.group * (dim + 4);
    if (bits == 4)
        return dim == 64 ? run_rows<4, 64>(f, stream) : dim == 128 ? run_rows<4, 128>(f, stream) : run_rows<4, 256>(f, stream);
    return dim == 64 ? run_rows<8, 64>(f, stream) : dim == 128 ? run_rows<8, 128>(f, stream) : run_rows<8, 256>(f, stream);
}

}  // namespace q8
