// attention_rows.hip -- attention of many rows a sequence and kv head (prompts, chunks of prompts, drafts
// of large groups): bound by the matrix cores.
//
// A workgroup of 4 waves takes a tile of 64 NR query rows of one sequence and kv head (a token's query heads
// side by side), 16 NR a wave, and walks over the tiles of 32 tokens that they see.  Keys and values become
// binary16 once for the workgroup: each wave turns a quarter of a tile's codes into operands of the matrix cores
// and leaves them in LDS in the order in which a wave takes them (no bank conflicts).  A stage makes
//   the weights of tile t from its scores,  the scores of tile t + 1,  the sums of tile t,
//   the operands of tile t + 2's keys and t + 1's values,
// so that the softmax's and the conversion's instructions have products beside them that do not wait for
// them; keys and values have two buffers each and one barrier a stage.
//
// With as many row tiles as the chip holds workgroups, each is taken whole: the longest first, and every second round
// over the CUs in the other order, so that what one CU gets of a causal prompt is about even.  Fewer stand in
// one line, row tile after row tile, of which every workgroup takes an equal part; a row tile that
// several share is joined by the last of them, in the order of the workgroups.
#include <algorithm>

#include "attention.h"
#include "launch.h"

namespace q8 {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kPerCu = 2;
constexpr int kMinTiles = 16;  // tiles of a workgroup's part of the line, at least

// Operands of 16 rows of a wave.
template <int D>
constexpr int kRowTiles = D == 256 ? 1 : 2;

struct RowsArgs {
    AttentionArgs a;
    int cus;
    int workgroups;
    uint32_t *arrived;  // [workgroups], zero between calls
    float *parts;       // [2 workgroups][slot]
};

// Floats of a part: sums of a row tile, then (maximum, sum) of its rows.
constexpr int slot_of(int d) { return (d == 256 ? 64 : 128) * (d + 4); }

// The rows of tile `x` of a sequence's rows.
__device__ __forceinline__ Rows rows_of_tile(const AttentionArgs &a, const Rows &r, int x, int tile_rows) {
    const int64_t from = int64_t(x) * tile_rows / a.group;
    const int64_t to = min((int64_t(x) + 1) * tile_rows + a.group - 1, int64_t(r.n) * a.group) / a.group;
    return {static_cast<int>(r.first + from), static_cast<int>(to - from), static_cast<int>(r.at + from), r.end};
}

// The line of row tiles: sequence after sequence, its last row tile first, kv heads side by side.  A row tile
// is as long as its sequence's last one, the longest; or each is 1 long.
template <int TILE>
struct Line {
    int s0 = 0;  // sequences s0 .. s0 + 63 are the lanes'
    int64_t before = 0;  // the line's place of the first of them
    Rows rows;
    int tiles, length;
    int64_t scan;

    __device__ __forceinline__ void look(const AttentionArgs &a, int lane, bool whole) {
        const int s = s0 + lane;
        rows = Rows{0, 0, 0, 0};
        if (s < a.c.sequences) rows = sequence_rows(a.c, s);
        tiles = static_cast<int>((int64_t(rows.n) * a.group + TILE - 1) / TILE);
        length = tiles ? (whole ? 1 : span_of(a, rows_of_tile(a, rows, tiles - 1, TILE)).n) : 0;
        scan = wave_scan(int64_t(tiles) * length * a.c.kv_heads, lane);
    }
    // All of it.
    __device__ __forceinline__ int64_t measure(const AttentionArgs &a, int lane, bool whole) {
        int64_t all = 0;
        for (s0 = 0; s0 < a.c.sequences; s0 += 64) {
            look(a, lane, whole);
            all += lane_of(scan, 63);
        }
        begin(a, lane, whole);
        return all;
    }
    __device__ __forceinline__ void begin(const AttentionArgs &a, int lane, bool whole) {
        before = 0;
        if (s0 == 64 || s0 == 0) {  // (one round: the lanes have it)
            const bool again = a.c.sequences > 64;
            s0 = 0;
            if (again) look(a, lane, whole);
        } else {
            s0 = 0;
            look(a, lane, whole);
        }
    }
    // The row tile at `at`, which is on the line.
    struct Item {
        int s, tile, head, length;
        int64_t origin;  // its place
        Rows rows;
    };
    __device__ __forceinline__ Item find(const AttentionArgs &a, int64_t at, int lane, bool whole) {
        if (at < before) begin(a, lane, whole);
        uint64_t above;
        while (!(above = __ballot(before + scan > at)) && s0 + 64 < a.c.sequences) {
            before += lane_of(scan, 63);
            s0 += 64;
            look(a, lane, whole);
        }
        const int l = above ? __builtin_ctzll(above) : 63;
        Item it;
        it.s = s0 + l;
        it.length = __builtin_amdgcn_readlane(length, l);
        const int64_t place = before + (l ? lane_of(scan, l - 1) : 0);
        const int64_t item = (at - place) / it.length;
        it.origin = place + item * it.length;
        it.head = static_cast<int>(item % a.c.kv_heads);
        it.tile = __builtin_amdgcn_readlane(tiles, l) - 1 - static_cast<int>(item / a.c.kv_heads);
        it.rows = Rows{__builtin_amdgcn_readlane(rows.first, l), __builtin_amdgcn_readlane(rows.n, l),
                       __builtin_amdgcn_readlane(rows.at, l), __builtin_amdgcn_readlane(rows.end, l)};
        return it;
    }
};

// What a wave turns into operands of a tile: a quarter of the keys' codes, and of the values'.  Wave w takes half
// w % 2 of the dimensions of the keys' 16 tokens w / 2, and D / 64 of the values' D / 16 operands.
template <int BITS, int D>
struct KeyCodes {
    using T = Tile<BITS, D>;
    static constexpr int kOperands = D / 64;
    static constexpr int kDwords = kOperands * BITS / 4;      // a lane
    static constexpr int kWords = BITS == 8 && D == 256 ? 2 : 1;
    uint32_t x[kDwords], w[kWords];

    __device__ __forceinline__ void load(const uint8_t *tile, int wid, uint32_t g, uint32_t c) {
        const uint32_t t = (c >> 2) * 8 + (c & 3), h = wid & 1;
        const uint8_t *p = tile + 4 * (wid >> 1) * T::kRow;
        // 16 bytes of a lane lie together: a quarter, a half or all of them, or two of them
        constexpr bool kApart = BITS == 4 ? D == 256 : D >= 128;  // halves of the dimensions lie apart
        const uint32_t at = t * T::kRow + (BITS == 4 && D == 64 ? g * 8 : g * 16) + h * (kApart ? D * BITS / 16 : 4 * kDwords);
        if constexpr (kDwords == 1) {
            x[0] = *reinterpret_cast<const uint32_t *>(p + at);
        } else if constexpr (kDwords == 2) {
            const u32x2 v = *reinterpret_cast<const u32x2 *>(p + at);
            x[0] = v.x, x[1] = v.y;
        } else {
#pragma unroll
            for (int u = 0; u < kDwords / 4; ++u) {
                const u32x4 v = *reinterpret_cast<const u32x4 *>(p + u * 64 + at);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * u + e] = v[e];
            }
        }
        const uint32_t block = (BITS == 4 && D > 64 ? g : g >> 1) + (kApart ? h * (D / 64) : 0);
#pragma unroll
        for (int u = 0; u < kWords; ++u)
            w[u] = *reinterpret_cast<const uint32_t *>(tile + u * 8 + T::kKeyWords + (c * T::kBlocks + block) * 4);
    }
    // operand e to [half][step][lane]
    __device__ __forceinline__ void store(half8 *keys, int e, int wid, int lane) const {
        Scales<BITS> s;
        s.set(__builtin_amdgcn_perm(w[e * kWords / kOperands], w[e * kWords / kOperands], wid >> 1 ? 0x03020302u : 0x01000100u));
        half8 v;
        if constexpr (BITS == 4) v = values_of(x[e], s, s, s, s);
        else v = values_of(x[2 * e], x[2 * e + 1], s, s, s, s);
        keys[((wid >> 1) * (D / 32) + (wid & 1) * kOperands + e) * 64 + lane] = v;
    }
};

template <int BITS, int D>
struct ValueCodes {
    using T = Tile<BITS, D>;
    using O = Out<BITS, D>;
    static constexpr int kOperands = D / 64;
    static constexpr int kDwords = kOperands * BITS / 4;
    static constexpr int kBlocks = BITS == 4 && D == 256 ? 2 : 1;
    uint32_t x[kDwords];
    u32x4 w[kBlocks];

    __device__ __forceinline__ void load(const uint8_t *tile, int wid, uint32_t g, uint32_t c) {
        // the wave's first operand is number wid * kOperands: (chunk, operand of it)
        const uint32_t first = wid * kOperands, m = first / O::kIn, in = first % O::kIn, u = O::unit(c);
        const uint32_t at = T::kValues + ((u * 4 + g) * 16 + O::chunk(c, 0) + m) * 16 + in * (BITS == 4 ? 4 : 8);
        if constexpr (kDwords == 1) {
            x[0] = *reinterpret_cast<const uint32_t *>(tile + at);
        } else if constexpr (kDwords == 2) {
            const u32x2 v = *reinterpret_cast<const u32x2 *>(tile + at);
            x[0] = v.x, x[1] = v.y;
        } else {
#pragma unroll
            for (int q = 0; q < kDwords / 4; ++q) {
                const u32x4 v = *reinterpret_cast<const u32x4 *>(tile + 16 * q + at);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * q + e] = v[e];
            }
        }
        const uint32_t block = BITS == 4 ? 2 * u + (kBlocks == 1 ? in / 2 : 0) : u;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) w[b] = *reinterpret_cast<const u32x4 *>(tile + b * 64 + T::kValueWords + (block * 4 + g) * 16);
    }
    // operand e to [operand][lane]
    __device__ __forceinline__ void store(half8 *values, int e, int wid, int lane) const {
        Scales<BITS> s[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) s[p].set(w[kBlocks == 2 ? e / 2 : 0][p]);
        half8 v;
        if constexpr (BITS == 4) v = values_of(x[e], s[0], s[1], s[2], s[3]);
        else v = values_of(x[2 * e], x[2 * e + 1], s[0], s[1], s[2], s[3]);
        values[(wid * kOperands + e) * 64 + lane] = v;
    }
};

template <int BITS, int D>
__global__ __launch_bounds__(kThreads, kPerCu) void rows_kernel(RowsArgs f) {
    using O = Out<BITS, D>;
    constexpr int NR = kRowTiles<D>, kTile = 64 * NR, kSteps = D / 32, kSlot = slot_of(D);
    __shared__ half8 keys[2][2 * kSteps * 64], values[2][D / 16 * 64];
    __shared__ uint32_t last;
    const AttentionArgs &a = f.a;
    const CacheArgs &c = a.c;
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    Line<kTile> line;
    int64_t all = line.measure(a, lane, true);
    const bool whole = all >= f.workgroups;
    int64_t chunk = 1;
    if (!whole) {
        line.s0 = 0;
        all = line.measure(a, lane, false);
        chunk = max((all + f.workgroups - 1) / f.workgroups, int64_t(kMinTiles));
    }

    for (int64_t p = blockIdx.x; p * chunk < all; p += gridDim.x) {
        int64_t at = p * chunk, stop = min(at + chunk, all);
        if (whole) {  // every second round over the CUs backwards
            const int64_t round = p / f.cus, size = min(int64_t(f.cus), all - round * f.cus);
            if (round & 1) at = round * f.cus + size - 1 - (p - round * f.cus);
            stop = at + 1;
        }
        while (at < stop) {
            const typename Line<kTile>::Item it = line.find(a, at, lane, whole);
            const Rows r = it.rows, tile_rows = rows_of_tile(a, r, it.tile, kTile);
            const Span span = span_of(a, tile_rows);
            // this workgroup's share of the row tile
            const int64_t share_end = min(stop - it.origin, int64_t(it.length));
            const int from = static_cast<int>(int64_t(span.n) * (at - it.origin) / it.length);
            const int to = static_cast<int>(int64_t(span.n) * share_end / it.length);
            const bool alone = at == it.origin && share_end == it.length, begins = at == it.origin;
            const int first = alone ? 0 : static_cast<int>(it.origin / chunk);
            const int sharers = alone ? 1 : static_cast<int>((it.origin + it.length - 1) / chunk) - first + 1;
            at = it.origin + share_end;
            const int rows = r.n * a.group, row0 = it.tile * kTile, head = it.head;
            // tokens that any row of the tile sees, and those that every one does
            const int lo = a.window ? max(tile_rows.at - a.window + 1, 0) : 0, hi = min(tile_rows.at + tile_rows.n, r.end);
            const int all_lo = a.window ? max(tile_rows.at + tile_rows.n - a.window, 0) : 0, all_hi = min(tile_rows.at + 1, r.end);

            // Pages of the tiles paged .. paged + 63, one a lane (-1: none).
            const int shift = c.page_shift - 5;
            int paged, page;
            const auto look_up = [&](int tile) {
                paged = tile;
                const int t = span.first + tile + lane;
                page = -1;
                if (tile + lane < to && t * kTileTokens < hi) page = c.table[it.s * c.table_ld + (t >> shift)];
                if (page < 0 || page >= c.pages) page = -1;
            };
            const auto page_of = [&](int tile) { return __builtin_amdgcn_readlane(page, tile - paged); };
            const auto tile_in = [&](int tile, int pg) -> const uint8_t * {  // (none: the pool's first, not looked at)
                const int t = span.first + tile;
                return c.data + (((int64_t(max(pg, 0)) * c.kv_heads + head) << shift) + (t & ((1 << shift) - 1))) * Tile<BITS, D>::kBytes;
            };

            KeyCodes<BITS, D> kc;
            ValueCodes<BITS, D> vc;
            // the value words of tokens that are not there are no value's
            const auto clear_words = [&](int tile, int pg) {
                const int t0 = (span.first + tile) * kTileTokens;
                if (pg >= 0 && t0 >= lo && t0 + kTileTokens <= hi) return;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int t = t0 + 8 * g + q;
                    const uint32_t there = (t >= lo && t < hi ? 0xffffu : 0u) | (t + 4 >= lo && t + 4 < hi ? 0xffff0000u : 0u);
#pragma unroll
                    for (auto &w : vc.w) w[q] = pg < 0 ? 0u : w[q] & there;
                }
            };
            look_up(from);
            // pages of tile + 1, tile + 2
            int page1 = page_of(from + 1), page2 = page_of(from + 2);
            const int page0 = page_of(from);
            kc.load(tile_in(from, page0), wid, g, col);
            vc.load(tile_in(from, page0), wid, g, col);

            half8 q_hi[NR][kSteps], q_lo[NR][kSteps];
            float to_score[NR], top[NR], sum[NR];
            f32x4 acc[O::kChunks][O::kIn][NR];  // row operands last
            const int first_row = row0 + wid * 16 * NR;
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                const int x = first_row + n * 16 + col;
                const float *row = nullptr;
                if (x < rows) {
                    const Where q = where(a, r, head, x);
                    row = a.q + q.row * a.q_ld + int64_t(q.head) * D;
                }
                to_score[n] = load_query<BITS, D>(row, a.scale, g, [&](int s, half8 h, half8 l) { q_hi[n][s] = h, q_lo[n][s] = l; });
                top[n] = kNoMax;
                sum[n] = 0.0f;
#pragma unroll
                for (int m = 0; m < O::kChunks; ++m)
#pragma unroll
                    for (int j = 0; j < O::kIn; ++j) acc[m][j][n] = f32x4{0.f, 0.f, 0.f, 0.f};
            }

            const auto scores = [&](int tile, f32x4(&z)[NR][2]) {
                const half8 *k = keys[tile & 1] + lane;
#pragma unroll
                for (int n = 0; n < NR; ++n) z[n][0] = z[n][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    const half8 k0 = k[s * 64], k1 = k[(kSteps + s) * 64];
#pragma unroll
                    for (int n = 0; n < NR; ++n) z[n][0] = mfma(k0, q_hi[n][s], z[n][0]), z[n][1] = mfma(k1, q_hi[n][s], z[n][1]);
#pragma unroll
                    for (int n = 0; n < NR; ++n) z[n][0] = mfma(k0, q_lo[n][s], z[n][0]), z[n][1] = mfma(k1, q_lo[n][s], z[n][1]);
                }
            };
            // What a row does not see of a tile, and the maximum.
            const auto settle = [&](int tile, int pg, f32x4(&z)[NR][2], float (&most)[NR]) {
                const int t0 = (span.first + tile) * kTileTokens;
                if (pg < 0 || t0 < all_lo || t0 + kTileTokens > all_hi) {
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        const int x = first_row + n * 16 + col, t = r.at + x / a.group;
                        const int end = pg < 0 || x >= rows ? 0 : min(t + 1, r.end);
                        mask_scores(z[n], t0, g, a.window ? t - a.window + 1 : 0, end);
                        most[n] = largest(z[n]);
                    }
                }
#pragma unroll
                for (int n = 0; n < NR; ++n) follow_max<O>(most[n] * to_score[n], top[n], sum[n], [&](int m, int j) -> f32x4 & { return acc[m][j][n]; });
            };

            // keys of the first two tiles, values of the first
            constexpr int kMine = D / 64;  // operands of keys, and of values, that a wave makes
            clear_words(from, page0);
#pragma unroll
            for (int e = 0; e < kMine; ++e) kc.store(keys[from & 1], e, wid, lane), vc.store(values[from & 1], e, wid, lane);
            kc.load(tile_in(from + 1, page1), wid, g, col);
            vc.load(tile_in(from + 1, page1), wid, g, col);
#pragma unroll
            for (int e = 0; e < kMine; ++e) kc.store(keys[(from + 1) & 1], e, wid, lane);
            kc.load(tile_in(from + 2, page2), wid, g, col);
            clear_words(from + 1, page1);
            __syncthreads();
            f32x4 z[NR][2];
            float most[NR];
            if (from < to) {
                scores(from, z);
#pragma unroll
                for (int n = 0; n < NR; ++n) most[n] = largest(z[n]);
                settle(from, page0, z, most);
            }
            __syncthreads();
            for (int tile = from; tile < to; ++tile) {
                if (tile + 3 - paged > 63) look_up(tile);
                const int page3 = page_of(tile + 3);
                // The weights of this tile beside the scores of the next.  The order of the steps is kept (the
                // barriers), for the compiler makes all weights and then all products.
                half2 p_hi[NR][4], p_lo[NR][4];
                f32x4 next[NR][2];
#pragma unroll
                for (int n = 0; n < NR; ++n) next[n][0] = next[n][1] = f32x4{0.f, 0.f, 0.f, 0.f};
                const half8 *k = keys[(tile + 1) & 1] + lane, *v = values[tile & 1] + lane;
                half8 k0 = k[0], k1 = k[kSteps * 64], k0_next = k0, k1_next = k1;
                half8 x = v[0], x_next = x;
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int s = 0; s < 2 * kSteps; ++s) {
                    if (s % 2 == 0 && s / 2 + 1 < kSteps) k0_next = k[(s / 2 + 1) * 64], k1_next = k[(kSteps + s / 2 + 1) * 64];
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        const half8 q = s % 2 ? q_lo[n][s / 2] : q_hi[n][s / 2];
                        next[n][0] = mfma(k0, q, next[n][0]);
                        next[n][1] = mfma(k1, q, next[n][1]);
                    }
#pragma unroll
                    for (int i = s * 4 * NR / (2 * kSteps); i < (s + 1) * 4 * NR / (2 * kSteps); ++i)
                        weigh_pair(z[i / 4], i % 4, to_score[i / 4], top[i / 4], sum[i / 4], p_hi[i / 4][i % 4], p_lo[i / 4][i % 4]);
                    if (s % 2) k0 = k0_next, k1 = k1_next;
                    __builtin_amdgcn_sched_barrier(0);
                }
                half8 w_hi[NR], w_lo[NR];
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    w_hi[n] = join(p_hi[n][0], p_hi[n][1], p_hi[n][2], p_hi[n][3]);
                    w_lo[n] = join(p_lo[n][0], p_lo[n][1], p_lo[n][2], p_lo[n][3]);
                    z[n][0] = next[n][0], z[n][1] = next[n][1];
                }
                // The sums of this tile beside the next operands.
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    if (j + 1 < D / 16) x_next = v[(j + 1) * 64];
                    f32x4(&o)[NR] = acc[j / O::kIn][j % O::kIn];
#pragma unroll
                    for (int n = 0; n < NR; ++n) o[n] = mfma(x, w_hi[n], o[n]);
#pragma unroll
                    for (int n = 0; n < NR; ++n) o[n] = mfma(x, w_lo[n], o[n]);
                    constexpr int kWork = 2 * kMine + NR;
#pragma unroll
                    for (int i = j * kWork / (D / 16); i < (j + 1) * kWork / (D / 16); ++i) {
                        if (i < kMine) kc.store(keys[tile & 1], i, wid, lane);
                        if (i == kMine - 1) kc.load(tile_in(tile + 3, page3), wid, g, col);
                        if (i >= kMine && i < 2 * kMine) vc.store(values[(tile + 1) & 1], i - kMine, wid, lane);
                        if (i == 2 * kMine - 1) vc.load(tile_in(tile + 2, page2), wid, g, col);
                        if (i >= 2 * kMine) most[i - 2 * kMine] = largest(z[i - 2 * kMine]);
                    }
                    x = x_next;
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (tile + 1 < to) settle(tile + 1, page1, z, most);
                clear_words(tile + 2, page2);
                page1 = page2, page2 = page3;
                __syncthreads();
            }

            // A part: rows of D sums, then rows of (maximum, sum).  A workgroup has two at most: one that ends
            // a row tile, and one that begins one, of which the second place is.
            const __amdgpu_buffer_rsrc_t parts = parts_of(f.parts, 2 * f.workgroups * kSlot);
            const auto part = [&](int i) { return static_cast<uint32_t>(2 * (first + i) + (i == 0)) * kSlot; };
            const uint32_t mine = (2 * static_cast<uint32_t>(p) + begins) * kSlot;
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                const int x = first_row + n * 16 + col;
                const float total = column_sum(sum[n]);
                if (x >= rows) continue;
                constexpr float kScale = Scales<BITS>::kUp;
                if (alone) {
                    const Where to_row = where(a, r, head, x);
                    O::for_each_vec([&](int m, int j) { return acc[m][j][n]; }, g, [&](int dim, f32x4 o) { write_row<D>(a, to_row, dim, o * kScale, total, top[n]); });
                } else {
                    const int y = x - row0;
                    O::for_each_vec([&](int m, int j) { return acc[m][j][n]; }, g, [&](int dim, f32x4 o) { store_part(parts, mine + y * D + dim, o * kScale); });
                    if (g == 0) store_part(parts, mine + kTile * D + 4 * y, f32x4{top[n], total, 0.f, 0.f});
                }
            }
            if (!alone) {
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                __syncthreads();
                if (threadIdx.x == 0) {
                    uint32_t *counter = f.arrived + first;
                    const uint32_t done = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                    last = done == static_cast<uint32_t>(sharers) - 1;
                    if (last) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                }
                __syncthreads();
                if (last) {
                    const int vecs = min(rows - row0, kTile) * (D / 4);
                    for (int e = threadIdx.x; e < vecs; e += kThreads) {
                        const int y = e / (D / 4), dim = e % (D / 4) * 4;
                        Sums joined;
                        constexpr int kAhead = 4;
                        for (int i = 0; i < sharers; i += kAhead) {
                            f32x4 o[kAhead], st[kAhead];
#pragma unroll
                            for (int j = 0; j < kAhead; ++j) {
                                // (past the last one: past the buffer, nothing is read)
                                const uint32_t place = part(i + j) | oob_bit(i + j < sharers) >> 2;
                                st[j] = load_part(parts, place + kTile * D + 4 * y);
                                o[j] = load_part(parts, place + 4 * e);
                            }
#pragma unroll
                            for (int j = 0; j < kAhead; ++j)
                                if (i + j < sharers) joined.add(o[j], st[j].x, st[j].y);
                        }
                        write_row<D>(a, where(a, r, head, row0 + y), dim, joined.o, joined.sum, joined.top);
                    }
                }
            }
            __syncthreads();  // LDS is free again
        }
    }
}

int rows_workgroups() { return device_info().cus * kPerCu; }

template <int BITS, int D>
hipError_t run(const RowsArgs &f, hipStream_t stream) {
    constexpr int kTile = 64 * kRowTiles<D>;
    // a workgroup for each row tile there may be, unless there are very many
    const int64_t row_tiles = (int64_t(f.a.c.max_rows) * f.a.group + kTile - 1) / kTile;
    const int64_t most = std::max<int64_t>(f.workgroups, f.a.c.sequences * f.a.c.kv_heads * row_tiles);
    const dim3 grid(static_cast<uint32_t>(std::min<int64_t>(most, 16 * int64_t(f.workgroups))));
    rows_kernel<BITS, D><<<grid, kThreads, 0, stream>>>(f);
    return hipGetLastError();
}

}  // namespace

int64_t rows_workspace(int dim) { return attention_counter_bytes() + int64_t(2) * rows_workgroups() * slot_of(dim) * 4; }

hipError_t launch_rows(int bits, int dim, const AttentionArgs &a, void *workspace, hipStream_t stream) {
    RowsArgs f = {};
    f.a = a;
    f.cus = device_info().cus;
    f.workgroups = rows_workgroups();
    f.arrived = static_cast<uint32_t *>(workspace);
    f.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + attention_counter_bytes());
    if (bits == 4) return dim == 64 ? run<4, 64>(f, stream) : dim == 128 ? run<4, 128>(f, stream) : run<4, 256>(f, stream);
    return dim == 64 ? run<8, 64>(f, stream) : dim == 128 ? run<8, 128>(f, stream) : run<8, 256>(f, stream);
}

}  // namespace q8
