// attention_rows.hip -- attention of many rows a sequence and kv head (prompts, chunks of prompts, drafts
// of large groups): bound by the matrix cores.
//
// A workgroup takes a tile of 128 query rows of one sequence and kv head (a token's query heads side by
// side; 64 rows of 256 dimensions, for the registers).  A group of waves, with 32 rows each, walks over the tiles of 32
// tokens that the rows see; a second group over every second of them, with the same rows, and their sums meet in LDS.
// So a SIMD has two waves (256 dimensions: one), one's softmax beside the other's products, and a row tile is
// done in half the time, which is what evens out causal prompts.  Keys and values become binary16 once for a group:
// each wave turns its share of a tile's codes into operands of the matrix cores and leaves them in LDS in the order in
// which a wave takes them (no bank conflicts).  A stage makes
//   the weights of tile t from its scores,  the scores of the tile after it,  the sums of tile t,
//   the operands of the keys two tiles on and the values one tile on,
// so that the softmax's and the conversion's instructions have products beside them that do not wait for
// them; keys and values have two buffers each and one barrier a stage.  The 32 x 32 x 16 products leave
// more room for other instructions beside them than the 16 x 16 x 32 ones, which take twice as many
// operands from the registers for the same work.
//
// Row tiles are taken whole, a prompt's last ones, which see most, first; or they stand in one line, sequence after
// sequence, of which every workgroup takes an equal part, and a row tile that several share is joined by the last
// of them, in the order of the workgroups.  What is estimated to take longer is not taken (Line::measure).
//
// Measured: a prompt of 2048 tokens, 32 heads of 8 kv heads and 128 dimensions, 4 bits: 88 us for 34 GFLOP, 0.78 PFLOP/s of
// binary16 products with both words (a large library product reaches 1.1); two chunks of 512 tokens after 16384: 383 us for 196
// GFLOP, 1.02 PFLOP/s.  A stage takes some 3500 cycles of 1.9 GHz, 2048 of which the matrix cores work; the rest is the issue
// port, which a product takes for half of its time and each weight (an exponential, two words) and code for its own.
// Beside the stages a row tile takes some 12 us: its queries, the first tiles' way through memory, the output.
//
// v_mfma_f32_32x32x16_f16, as its lanes hold it (lane = 32 h + c):
//   A: row c, depth 8 h + e (e = 0 .. 7);  B: column c, depth 8 h + e;
//   C: column c, rows 8 a + 4 h + j in register 4 a + j
// Scores: row 8 a + 4 h + j is token 16 (a / 2) + 8 h + 4 (a % 2) + j of a tile, so that a lane gets row
// c's scores of eight tokens in a row of each half of the tile, and gives their weights to the sums.
#include <algorithm>

#include "attention.h"
#include "launch.h"

namespace q8 {
namespace {

// Tiles of a workgroup's part of the line, at least.  64 rows after 3000 tokens: 44.6 us, at 8 48.0, at 16 47.1; 100 after 9000
// of 256 dimensions: 71.6, at 8 76.9, at 16 77.6.
constexpr int kMinTiles = 12;

constexpr int kGroups = 2;  // of waves
// A group's waves, of 32 query rows each: 256 dimensions take twice the registers for queries and sums.  (One group of four
// waves there: chunks of 700 tokens in a window of 1024 82 us, with two of two 77.)
constexpr int waves_of(int d) { return d == 256 ? 2 : 4; }
constexpr int rows_of(int d) { return 32 * waves_of(d); }  // query rows of a workgroup, a row tile

struct RowsArgs {
    AttentionArgs a;
    int workgroups;     // that the chip holds
    uint32_t *arrived;  // [workgroups], zero between calls
    float *parts;       // [2 workgroups][slot]
};

// Floats of a part: a row tile's sums, and (maximum, sum, -, -) for each lane of a group.
constexpr int slot_of(int d) { return rows_of(d) * (d + 8); }

// The rows of tile `x` of a sequence's rows (rows times heads is below 2^31: the outputs fit in memory).
template <int TILE>
__device__ __forceinline__ Rows rows_of_tile(const AttentionArgs &a, const Rows &r, int x) {
    const uint32_t group = a.group, from = uint32_t(x) * TILE / group;
    const uint32_t to = min((uint32_t(x) + 1) * TILE + group - 1, uint32_t(r.n) * group) / group;
    return {static_cast<int>(r.first + from), static_cast<int>(to - from), static_cast<int>(r.at + from), r.end};
}

// The line of row tiles, sequence after sequence: with `whole` each is 1 long, the last one first and kv heads side
// by side; else a kv head's row tiles follow one another, each about as long as the tiles of tokens that
// it sees, in sixteenths: these grow evenly from the sequence's first row tile to its last.
constexpr int kLinePart = 16;
// What a row tile costs besides its tiles (queries, first tiles and ends of the pipeline, the output), in tiles of
// tokens; a part that does not end there costs as much and a join.  It decides between whole row tiles and parts. us here, and
// at half and (64 and 256 dimensions) one and a half times or (128) twice as much:
//   64 dimensions:  8 heads of 4 kv heads, prompt of 512 tokens 19.1, 27.0, 19.0; of 2048 37.0, 35.1, 44.9;
//                   32 of 8, chunks of 700 in a window of 1024, 8 bits 76.7, 74.7, 85.9
//   128 dimensions: 32 of 8, prompt of 512 26.9, 47.7, 26.9; of 1024 40.4, 55.7, 40.5; 8 of 4, of 512 38.0, 36.7, 26.1;
//                   8 of 4, 100 rows after 4000 tokens 43.2, 43.2, 44.6
//   256 dimensions: 8 of 4, prompt of 512 35.1, 47.0, 35.1; the chunks in a window 84.6, 94.5, 94.4
constexpr int cost_of(int d) { return d == 64 ? 24 : d == 128 ? 12 : 18; }
template <int D>
struct Line {
    static constexpr int TILE = rows_of(D), kCost = cost_of(D), kJoin = 2 * kCost;
    // 64 sequences, a wave's: in LDS, for the registers are the products'
    struct State {
        int rows[4][64], tiles[64], first[64], step[64];
        int64_t scan[64];
    };
    State &state;
    int lane;
    bool whole = true;
    int s0 = 0;          // of sequences s0 .. s0 + 63
    int64_t before = 0;  // the line's place of the first of them

    // Place of a kv head's row tile x, the first one `first` long and each one `step` longer.
    static __device__ __forceinline__ int64_t place(int x, int first, int step) {
        return int64_t(x) * first + (int64_t(x) * (x - 1) >> 1) * step;
    }
    __device__ __forceinline__ void look(const AttentionArgs &a) {
        const int s = s0 + lane;
        Rows rows = {0, 0, 0, 0};
        if (s < a.c.sequences) rows = sequence_rows(a.c, s);
        const int tiles = static_cast<int>((uint32_t(rows.n) * uint32_t(a.group) + TILE - 1) / TILE);
        int first = 0, step = 0;
        if (tiles) {
            first = kLinePart * (span_of(a, rows_of_tile<TILE>(a, rows, 0)).n + kCost);
            step = max((kLinePart * (span_of(a, rows_of_tile<TILE>(a, rows, tiles - 1)).n + kCost) - first) / max(tiles - 1, 1), 0);
        }
        state.rows[0][lane] = rows.first, state.rows[1][lane] = rows.n, state.rows[2][lane] = rows.at, state.rows[3][lane] = rows.end;
        state.tiles[lane] = tiles, state.first[lane] = first, state.step[lane] = step;
    }
    __device__ __forceinline__ int64_t scan(const AttentionArgs &a) {
        const int n = state.tiles[lane];
        const int64_t v = wave_scan(a.c.kv_heads * (whole ? int64_t(n) : place(n, state.first[lane], state.step[lane])));
        state.scan[lane] = v;
        return lane_of(v, 63);
    }
    // How long the line is, and which it is: row tiles are whole if that takes no longer than equal parts, which
    // are joined (or if they are so many that their places would overflow).  A prompt of 512 tokens takes 28 us in whole row
    // tiles and 41 in parts, 1024 tokens 42 and 56, chunks of 900 after 1000 209 and 226; two chunks of 512 after 16384 in
    // whole row tiles 539 and in parts 409.
    __device__ __forceinline__ int64_t measure(const AttentionArgs &a, int workgroups) {
        int64_t items = 0, all = 0;
        float longest = 0.0f, shortest = 3.0e38f;
        for (s0 = 0; s0 < a.c.sequences; s0 += 64) {
            look(a);
            const int n = state.tiles[lane];
            const float first = static_cast<float>(state.first[lane]), last = first + static_cast<float>(state.step[lane]) * static_cast<float>(n - 1);
            longest = fmaxf(longest, wave_max(n ? last : 0.0f));
            shortest = fminf(shortest, -wave_max(n ? -first : -3.0e38f));
            whole = true;
            items += scan(a);
            whole = false;
            all += scan(a);
        }
        // Whole, the longest first: the workgroups that have no row tile in the last round wait for the shortest.
        const float per = static_cast<float>(items) / static_cast<float>(workgroups), part = static_cast<float>(all) / static_cast<float>(workgroups);
        whole = items >= 1 << 16 || fmaxf(longest, part + (ceilf(per) - per) * shortest) <= part + kLinePart * kJoin;
        s0 = 0;
        if (a.c.sequences > 64) look(a);
        scan(a);
        return whole ? items : all;
    }
    // The row tile at `at`, which is on the line and not before the last one found.
    struct Item {
        int s, tile, head;
        int64_t origin, length;
        Rows rows;
    };
    __device__ __forceinline__ Item find(const AttentionArgs &a, int64_t at) {
        uint64_t above;
        while (!(above = __ballot(before + state.scan[lane] > at)) && s0 + 64 < a.c.sequences) {
            before += state.scan[63];
            s0 += 64;
            look(a);
            scan(a);
        }
        const int l = above ? __builtin_ctzll(above) : 63;
        const auto of = [&](const int(&v)[64]) { return __builtin_amdgcn_readfirstlane(v[l]); };
        const int64_t begin = before + (l ? lane_of(state.scan[l - 1], 0) : 0);
        const int n = of(state.tiles);
        Item it;
        it.s = s0 + l;
        it.rows = Rows{of(state.rows[0]), of(state.rows[1]), of(state.rows[2]), of(state.rows[3])};
        if (whole) {
            const uint32_t item = static_cast<uint32_t>(at - begin), x = item / uint32_t(a.c.kv_heads);
            it.head = static_cast<int>(item - x * a.c.kv_heads);
            it.tile = n - 1 - static_cast<int>(x);
            it.origin = at;
            it.length = 1;
            return it;
        }
        const int first = of(state.first), step = of(state.step);
        const int64_t head_length = place(n, first, step);
        it.head = static_cast<int>(static_cast<float>(at - begin) / static_cast<float>(head_length));  // or one beside it
        int64_t rest = at - begin - it.head * head_length;
        if (rest < 0) --it.head, rest += head_length;
        if (rest >= head_length) ++it.head, rest -= head_length;
        for (int x0 = 0;; x0 += 64) {  // the last row tile whose place is not past `rest`
            const uint64_t past = __ballot(x0 + lane + 1 >= n || place(x0 + lane + 1, first, step) > rest);
            if (past) {
                it.tile = x0 + __builtin_ctzll(past);
                break;
            }
        }
        const int64_t p = place(it.tile, first, step);
        it.origin = at - rest + p;
        it.length = first + int64_t(it.tile) * step;
        return it;
    }
};

// What a wave turns into operands of a tile: its group's share of the keys' codes, and of the values'.  An operand of the
// scores is 16 dimensions of the tile's tokens: step s has dimensions D / 2 h + 8 s + e; wave w makes steps
// kMine w + ..
template <int BITS, int D>
struct KeyCodes {
    using T = Tile<BITS, D>;
    static constexpr int kMine = D / 16 / waves_of(D);
    static constexpr int kDwords = kMine * BITS / 4;  // a lane
    static constexpr int kBlocks = (kMine + 3) / 4;
    uint32_t x[kDwords], w[kBlocks];

    // where a lane's codes and word are, and which half of the word's pair is its token's
    struct Place {
        uint32_t code, word, half;
    };
    static __device__ __forceinline__ Place place(uint32_t wid, uint32_t h, uint32_t c) {
        const uint32_t t = 16 * (c >> 4) + 8 * ((c >> 2) & 1) + 4 * ((c >> 3) & 1) + (c & 3);  // row c's token
        const uint32_t block = (h * (D / 2) + wid * 8 * kMine) / 32;
        return {t * T::kRow + h * (T::kRow / 2) + wid * (4 * kDwords),
                T::kKeyWords + 2 * (key_word(t, block, T::kBlocks) & ~1u), (c >> 3) & 1 ? 0x03020302u : 0x01000100u};
    }
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t tile, const Place &p) {
        if constexpr (kDwords == 1) {
            x[0] = load1(tile, p.code, 0);
        } else if constexpr (kDwords == 2) {
            const u32x2 v = load2(tile, p.code, 0);
            x[0] = v.x, x[1] = v.y;
        } else {
#pragma unroll
            for (int u = 0; u < kDwords / 4; ++u) {
                const u32x4 v = load4(tile, p.code, u * 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * u + e] = v[e];
            }
        }
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) w[b] = load1(tile, p.word, 4 * b);
    }
    // operand e to [step][lane]
    __device__ __forceinline__ void store(half8 *keys, int e, int wid, int lane, const Place &p) const {
        Scales<BITS> s;
        s.set(__builtin_amdgcn_perm(w[e / 4], w[e / 4], p.half));
        half8 v;
        if constexpr (BITS == 4) v = values_of(x[e], s, s, s, s);
        else v = values_of(x[2 * e], x[2 * e + 1], s, s, s, s);
        keys[(wid * kMine + e) * 64 + lane] = v;
    }
};

// An operand (u, d) of the sums is 32 dimensions of tokens 16 u + 8 h + e; its row c is dimension
// out_dim(c, d).  Half of a group's waves make operands of u = 0, half of u = 1, kMine each.
template <int BITS, int D>
struct ValueCodes {
    using T = Tile<BITS, D>;
    static constexpr int kMine = D / 16 / waves_of(D), kHalf = waves_of(D) / 2;
    static constexpr int kDwords = kMine * BITS / 4;
    static constexpr int kBlocks = D == 256 ? kMine / 2 : 1;
    // A unit of the layout is 64 (4 bits) or 32 dimensions: 16 chunks of kIn times 16.  The rows' halves are
    // units side by side, or (one unit) dimensions of one.
    static constexpr int kUnit = BITS == 4 ? 64 : 32, kIn = kUnit / 16;
    static constexpr bool kOneUnit = D == kUnit;
    uint32_t x[kDwords];
    u32x4 w[kBlocks];

    static __device__ __forceinline__ constexpr int out_dim(int c, int d) {
        if (kOneUnit) return 32 * d + c;
        return kUnit * (2 * (d / kIn) + c / 16) + 16 * (d % kIn) + c % 16;
    }
    struct Place {
        uint32_t code, word;
    };
    static __device__ __forceinline__ Place place(uint32_t wid, uint32_t h, uint32_t c) {
        const uint32_t a = 2 * (wid / kHalf) + h, d = kMine * (wid % kHalf);
        const uint32_t unit = kOneUnit ? 0 : 2 * (d / kIn) + (c >> 4), in = kOneUnit ? 2 * d + (c >> 4) : d % kIn;
        // blocks of 32 dimensions: two a unit of 4 bits, one of 8
        const uint32_t block = BITS == 4 ? 2 * unit + in / 2 : unit;
        return {T::kValues + ((unit * 4 + a) * 16 + (c & 15)) * 16 + in * (BITS == 4 ? 4 : 8), T::kValueWords + (block * 4 + a) * 16};
    }
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t tile, const Place &p) {
        if constexpr (kDwords == 1) {
            x[0] = load1(tile, p.code, 0);
        } else if constexpr (kDwords == 2) {
            const u32x2 v = load2(tile, p.code, 0);
            x[0] = v.x, x[1] = v.y;
        } else {  // 16 bytes of a unit; a wave's next ones lie two units on
#pragma unroll
            for (int q = 0; q < kDwords / 4; ++q) {
                const u32x4 v = load4(tile, p.code, q * (2 * 4 * 16 * 16));
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * q + e] = v[e];
            }
        }
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) w[b] = load4(tile, p.word, (BITS == 4 ? b / 2 * 4 + b % 2 : 2 * b) * 64);
    }
    // operand e to [u][d][lane]
    __device__ __forceinline__ void store(half8 *values, int e, int wid, int lane) const {
        Scales<BITS> s[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) s[p].set(w[kBlocks > 1 ? e / 2 : 0][p]);
        half8 v;
        if constexpr (BITS == 4) v = values_of(x[e], s[0], s[1], s[2], s[3]);
        else v = values_of(x[2 * e], x[2 * e + 1], s[0], s[1], s[2], s[3]);
        values[(wid / kHalf * (D / 32) + wid % kHalf * kMine + e) * 64 + lane] = v;
    }
};

__device__ __forceinline__ float column_max(float v) {
    const float2 a = lane_pair32(v);
    return fmaxf(a.x, a.y);
}
__device__ __forceinline__ float column_sum(float v) {
    const float2 a = lane_pair32(v);
    return a.x + a.y;
}

__device__ __forceinline__ float largest(const f32x16 &z) {
    float most = z[0];
#pragma unroll
    for (int e = 1; e < 16; ++e) most = fmaxf(most, z[e]);
    return most;
}

template <int BITS, int D>
__global__ __launch_bounds__(64 * waves_of(D) * kGroups, waves_of(D) / 2) void rows_kernel(RowsArgs f) {
    using V = ValueCodes<BITS, D>;
    constexpr int kSteps = D / 16, kDims = D / 32, kSlot = slot_of(D);
    constexpr int kWaves = waves_of(D), kTile = rows_of(D), kMine = V::kMine;
    // A group's operands: keys, keys of the next tile, values, values of the next tile.  As large as the sums of
    // a group's waves, which meet there.
    constexpr int kKeys = kSteps * 64, kValues = 2 * kDims * 64, kOperands = 2 * (kKeys + kValues);
    static_assert(kOperands * kGroups * 16 >= kTile * D * 4);
    __shared__ half8 operands[kGroups][kOperands];
    __shared__ float tops[64 * kWaves], sums[64 * kWaves];
    __shared__ typename Line<D>::State states[kWaves * kGroups];
    __shared__ uint32_t last;
    const AttentionArgs &a = f.a;
    const CacheArgs &c = a.c;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wid = wave % kWaves, group = wave / kWaves;
    half8 *const keys = operands[group], *const values = keys + 2 * kKeys;

    Line<D> line = {states[wave], static_cast<int>(threadIdx.x & 63)};
    const int64_t all = line.measure(a, f.workgroups);
    const int64_t chunk = line.whole ? 1 : max((all + f.workgroups - 1) / f.workgroups, int64_t(kLinePart * kMinTiles));

    for (int64_t p = blockIdx.x; p * chunk < all; p += gridDim.x) {
        int64_t at = p * chunk;
        const int64_t stop = min(at + chunk, all);
        while (at < stop) {
            // (new to the compiler, which else makes what follows from them beforehand and keeps it in registers)
            int lane = threadIdx.x & 63;
            int64_t part_length = chunk;
            asm volatile("" : "+v"(lane), "+s"(part_length));
            const int h = lane >> 5, col = lane & 31;
            const typename Line<D>::Item it = line.find(a, at);
            const Rows r = it.rows, tile_rows = rows_of_tile<kTile>(a, r, it.tile);
            const Span span = span_of(a, tile_rows);
            // this workgroup's share of the row tile
            const int64_t share_end = min(stop - it.origin, it.length);
            // (rounded, but a workgroup's end as the next one's beginning)
            const auto tile_of = [&](int64_t part) {
                return part == it.length ? span.n : min(static_cast<int>(double(span.n) * double(part) / double(it.length)), span.n);
            };
            const int from = tile_of(at - it.origin), to = tile_of(share_end);
            const bool alone = at == it.origin && share_end == it.length, begins = at == it.origin;
            const int first = alone ? 0 : static_cast<int>(uint64_t(it.origin) / uint64_t(part_length));
            const int sharers = alone ? 1 : static_cast<int>((it.origin + it.length - 1) / part_length) - first + 1;
            at = it.origin + share_end;
            const int rows = r.n * a.group, row0 = it.tile * kTile, head = it.head;
            // tokens that any row of the tile sees, and those that every one does
            const int lo = a.window ? max(tile_rows.at - a.window + 1, 0) : 0, hi = min(tile_rows.at + tile_rows.n, r.end);
            const int all_lo = a.window ? max(tile_rows.at + tile_rows.n - a.window, 0) : 0, all_hi = min(tile_rows.at + 1, r.end);

            // the lane's row; past the last one that one's query, whose scores are not looked at
            const int x = row0 + wid * 32 + col;
            const Where of_q = where(a, r, head, min(x, rows - 1));
            QueryRow<kSteps> q_row;
            q_row.load(a.q + of_q.row * a.q_ld + int64_t(of_q.head) * D, [&](int s) { return D / 2 * h + 8 * s; });

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
            const auto tile_in = [&](int tile, int pg) {  // (none: the pool's first, not looked at)
                const int t = span.first + tile;
                return buffer_of(c.data + (((int64_t(max(pg, 0)) * c.kv_heads + head) << shift) + (t & ((1 << shift) - 1))) * Tile<BITS, D>::kBytes, Tile<BITS, D>::kBytes);
            };

            KeyCodes<BITS, D> kc;
            V vc;
            const auto kp = KeyCodes<BITS, D>::place(wid, h, col);
            const auto vp = V::place(wid, h, col);
            // the value words of tokens that are not there are no value's
            const auto clear_words = [&](int tile, int pg) {
                const int t0 = (span.first + tile) * kTileTokens;
                if (pg >= 0 && t0 >= lo && t0 + kTileTokens <= hi) return;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int t = t0 + 16 * (wid / V::kHalf) + 8 * h + q;
                    const uint32_t there = (t >= lo && t < hi ? 0xffffu : 0u) | (t + 4 >= lo && t + 4 < hi ? 0xffff0000u : 0u);
#pragma unroll
                    for (auto &w : vc.w) w[q] = pg < 0 ? 0u : w[q] & there;
                }
            };
            // a group's tiles: begin, begin + kGroups, ..; the pages of the next two
            const int begin = from + group;
            look_up(from);
            const int page0 = page_of(begin);
            int page1 = page_of(begin + kGroups), page2 = page_of(begin + 2 * kGroups);
            kc.load(tile_in(begin, page0), kp);
            vc.load(tile_in(begin, page0), vp);
            KeyCodes<BITS, D> kc1;
            kc1.load(tile_in(begin + kGroups, page1), kp);

            half8 q_hi[kSteps], q_lo[kSteps];
            const float to_score =
                query_words<BITS>(q_row, a.scale, column_max, [&](int s, half8 hi8, half8 lo8) { q_hi[s] = hi8, q_lo[s] = lo8; });
            float top = kNoMax, sum = 0.0f;
            f32x16 acc[kDims];
#pragma unroll
            for (int d = 0; d < kDims; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[d][e] = 0.0f;

            // What the row does not see of a tile, and the maximum.
            const auto settle = [&](int tile, int pg, f32x16 &z, float most) {
                const int t0 = (span.first + tile) * kTileTokens;
                if (pg < 0 || t0 < all_lo || t0 + kTileTokens > all_hi) {
                    const int t = r.at + x / a.group;
                    const int from_token = a.window ? t - a.window + 1 : 0, end = pg < 0 || x >= rows ? 0 : min(t + 1, r.end);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int token = t0 + 16 * (e >> 3) + 8 * h + (e & 7);
                        z[e] = token >= from_token && token < end ? z[e] : -INFINITY;
                    }
                    most = largest(z);
                }
                follow_max(most * to_score, top, sum, column_max, [&](float keep) {
#pragma unroll
                    for (int d = 0; d < kDims; ++d) acc[d] *= keep;
                });
            };

            // keys of the first two tiles, values of the first
            clear_words(begin, page0);
#pragma unroll
            for (int e = 0; e < kMine; ++e) kc.store(keys, e, wid, lane, kp), vc.store(values, e, wid, lane);
            kc.load(tile_in(begin + 2 * kGroups, page2), kp);
            vc.load(tile_in(begin + kGroups, page1), vp);
#pragma unroll
            for (int e = 0; e < kMine; ++e) kc1.store(keys + kKeys, e, wid, lane, kp);
            clear_words(begin + kGroups, page1);
            __syncthreads();
            f32x16 z;
#pragma unroll
            for (int e = 0; e < 16; ++e) z[e] = 0.0f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) z = mfma(keys[s * 64 + lane], q_hi[s], z), z = mfma(keys[s * 64 + lane], q_lo[s], z);
            settle(begin, page0, z, largest(z));
            __syncthreads();
            // Past the last tile a group's page is none: its weights there are zeros.
            for (int tile = begin, odd = 0; tile - group < to; tile += kGroups, odd ^= 1) {
                if (tile + 3 * kGroups - paged > 63) look_up(tile);
                const int page3 = page_of(tile + 3 * kGroups);
                // The weights of this tile beside the scores of the next.  The order of the steps is kept (the
                // barriers), for the compiler makes all weights and then all products.
                half2 p_hi[2][4], p_lo[2][4];
                f32x16 next;
#pragma unroll
                for (int e = 0; e < 16; ++e) next[e] = 0.0f;
                half8 *const now_keys = keys + (odd ? kKeys : 0), *const now_values = values + (odd ? kValues : 0);
                const half8 *k = keys + (odd ? 0 : kKeys) + lane, *v = now_values + lane;
                half8 *const next_values = values + (odd ? 0 : kValues);
                half8 operand = k[0], after = operand;
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    after = s + 1 < kSteps ? k[(s + 1) * 64] : v[0];
                    next = mfma(operand, q_hi[s], next);
                    next = mfma(operand, q_lo[s], next);
#pragma unroll
                    for (int i = s * 8 / kSteps; i < (s + 1) * 8 / kSteps; ++i) {
                        const int u = i / 4, p = i % 4;
                        weigh_pair(z[8 * u + p], z[8 * u + 4 + p], to_score, top, sum, p_hi[u][p], p_lo[u][p]);
                    }
                    operand = after;
                    __builtin_amdgcn_sched_barrier(0);
                }
                z = next;
                // The sums of this tile beside the next operands.
                float most = kNoMax;
#pragma unroll
                for (int j = 0; j < 2 * kDims; ++j) {
                    const int u = j / kDims, d = j % kDims;
                    if (j + 1 < 2 * kDims) after = v[(j + 1) * 64];
                    acc[d] = mfma(operand, join(p_hi[u][0], p_hi[u][1], p_hi[u][2], p_hi[u][3]), acc[d]);
                    acc[d] = mfma(operand, join(p_lo[u][0], p_lo[u][1], p_lo[u][2], p_lo[u][3]), acc[d]);
                    constexpr int kWork = 2 * kMine + 1;
#pragma unroll
                    for (int i = j * kWork / (2 * kDims); i < (j + 1) * kWork / (2 * kDims); ++i) {
                        if (i < kMine) kc.store(now_keys, i, wid, lane, kp);
                        if (i == kMine - 1) kc.load(tile_in(tile + 3 * kGroups, page3), kp);
                        if (i >= kMine && i < 2 * kMine) vc.store(next_values, i - kMine, wid, lane);
                        if (i == 2 * kMine - 1) vc.load(tile_in(tile + 2 * kGroups, page2), vp);
                        if (i == 2 * kMine) most = largest(z);
                    }
                    operand = after;
                    __builtin_amdgcn_sched_barrier(0);
                }
                settle(tile + kGroups, page1, z, most);
                clear_words(tile + 2 * kGroups, page2);
                page1 = page2, page2 = page3;
                __syncthreads();
            }

            {  // the other group's sums, lane by lane
                f32x4 *meet = reinterpret_cast<f32x4 *>(&operands[0][0]) + wid * (kDims * 4 * 64) + lane;
                if (group == 1) {
#pragma unroll
                    for (int d = 0; d < kDims; ++d)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            meet[(d * 4 + e) * 64] = f32x4{acc[d][4 * e], acc[d][4 * e + 1], acc[d][4 * e + 2], acc[d][4 * e + 3]};
                    tops[wid * 64 + lane] = top;
                    sums[wid * 64 + lane] = sum;
                }
                __syncthreads();
                if (group == 0) {
                    const float other = tops[wid * 64 + lane], now = fmaxf(top, other);
                    const float keep = exp2_of(top - now), more = exp2_of(other - now);
                    top = now;
                    sum = sum * keep + sums[wid * 64 + lane] * more;
#pragma unroll
                    for (int d = 0; d < kDims; ++d)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const f32x4 o = meet[(d * 4 + e) * 64];
#pragma unroll
                            for (int j = 0; j < 4; ++j) acc[d][4 * e + j] = acc[d][4 * e + j] * keep + o[j] * more;
                        }
                }
            }

            sum = column_sum(sum);
            if (!alone) {
                // A part: a wave's sums as its lanes hold them, then the rows' (maximum, sum), lane by lane.  A
                // workgroup has two at most: one that ends a row tile, and one that begins one, of which the second
                // place is.
                const __amdgpu_buffer_rsrc_t parts = parts_of(f.parts, 2 * f.workgroups * kSlot);
                const auto part = [&](int i, bool begins) {
                    return static_cast<uint32_t>(2 * i + begins) * kSlot + wid * (kSlot / kWaves) + 4 * lane;
                };
                if (group == 0) {
                    const uint32_t mine = part(static_cast<int>(p), begins);
#pragma unroll
                    for (int d = 0; d < kDims; ++d)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            store_part(parts, mine + (4 * d + e) * 256, f32x4{acc[d][4 * e], acc[d][4 * e + 1], acc[d][4 * e + 2], acc[d][4 * e + 3]});
                    store_part(parts, mine + kDims * 1024, f32x4{top, sum, 0.f, 0.f});
                    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                }
                __syncthreads();
                if (threadIdx.x == 0) {
                    uint32_t *counter = f.arrived + first;
                    const uint32_t done = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                    last = done == static_cast<uint32_t>(sharers) - 1;
                    if (last) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                }
                __syncthreads();
                if (last) {  // all of them, in the workgroups' order: half of the dimensions a group, the next part under way
                    constexpr int kHalf = kDims / 2, kLoads = kHalf * 4;
                    f32x4 o[kLoads], next[kLoads], st, next_st;
                    const auto load = [&](int i, f32x4(&to)[kLoads], f32x4 &to_st) {
                        const uint32_t from_part = part(first + i, i == 0);
                        to_st = load_part(parts, from_part + kDims * 1024);
#pragma unroll
                        for (int e = 0; e < kLoads; ++e) to[e] = load_part(parts, from_part + (group * kLoads + e) * 256);
                    };
                    load(0, o, st);
                    top = kNoMax;
                    sum = 0.0f;
#pragma unroll
                    for (int d = 0; d < kHalf; ++d)
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[d][e] = 0.0f;
                    for (int i = 0; i < sharers; ++i) {
                        load(min(i + 1, sharers - 1), next, next_st);
                        const float now = fmaxf(top, st.x), keep = exp2_of(top - now), more = exp2_of(st.x - now);
                        top = now;
                        sum = sum * keep + st.y * more;
#pragma unroll
                        for (int d = 0; d < kHalf; ++d)
#pragma unroll
                            for (int e = 0; e < 16; ++e) acc[d][e] = acc[d][e] * keep + o[4 * d + e / 4][e % 4] * more;
#pragma unroll
                        for (int e = 0; e < kLoads; ++e) o[e] = next[e];
                        st = next_st;
                    }
                }
            }
            // (what the wave has: all dimensions or its group's half)
            const int from_d = alone ? 0 : group * (kDims / 2), end_d = alone ? kDims : kDims / 2;
            if (x < rows && (alone ? group == 0 : last != 0)) {
                constexpr float kScale = Scales<BITS>::kUp;
                const Where to_row = where(a, r, head, x);
#pragma unroll
                for (int d = 0; d < kDims; ++d) {
                    if (d >= end_d) break;
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        write_row<D>(a, to_row, V::out_dim(2 * e + 4 * h, from_d + d),
                                     f32x4{acc[d][e], acc[d][e + 1], acc[d][e + 2], acc[d][e + 3]} * kScale, sum, top);
                }
            }
            __syncthreads();  // LDS is free again
        }
    }
}

int rows_workgroups() { return device_info().cus; }

template <int BITS, int D>
hipError_t run(const RowsArgs &f, hipStream_t stream) {
    // a workgroup for each row tile there may be, unless there are very many
    const int64_t row_tiles = (int64_t(f.a.c.max_rows) * f.a.group + rows_of(D) - 1) / rows_of(D);
    const int64_t most = std::max<int64_t>(f.workgroups, f.a.c.sequences * f.a.c.kv_heads * row_tiles);
    const dim3 grid(static_cast<uint32_t>(std::min<int64_t>(most, 32 * int64_t(f.workgroups))));
    rows_kernel<BITS, D><<<grid, 64 * waves_of(D) * kGroups, 0, stream>>>(f);
    return hipGetLastError();
}

}  // namespace

int64_t rows_workspace(int dim) { return attention_counter_bytes() + int64_t(2) * rows_workgroups() * slot_of(dim) * 4; }

hipError_t launch_rows(int bits, int dim, const AttentionArgs &a, void *workspace, hipStream_t stream) {
    RowsArgs f = {};
    f.a = a;
    f.workgroups = rows_workgroups();
    f.arrived = static_cast<uint32_t *>(workspace);
    f.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + attention_counter_bytes());
    if (bits == 4) return dim == 64 ? run<4, 64>(f, stream) : dim == 128 ? run<4, 128>(f, stream) : run<4, 256>(f, stream);
    return dim == 64 ? run<8, 64>(f, stream) : dim == 128 ? run<8, 128>(f, stream) : run<8, 256>(f, stream);
}

}  // namespace q8
